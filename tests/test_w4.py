"""thl.gemm_w4 against the plain fp64 product, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import tile_hierarchy_linear_amd as thl
from oracle import operators as ref

pytestmark = pytest.mark.gpu
F = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _make(m, n, k, type_w="u4", group=128, x="bf16", ts=None, seed=0, pitch=0, offset=0):
    """Weights, scales, zeros and x; rows pitched and starting off 16 bytes where asked."""
    g = torch.Generator().manual_seed(seed)
    kb, groups = (k + 1) // 2, max(1, -(-k // group))
    w = torch.randint(0, 256, (offset + m * (kb + pitch),), generator=g).to(torch.uint8).cuda()
    w = w[offset:].view(m, kb + pitch)[:, :kb]
    zeros = None
    if type_w == "e2m1":
        scales = torch.randint(110, 135, (m, groups + pitch), generator=g).to(torch.uint8).cuda()[:, :groups]
    else:
        scales = (torch.rand(m, groups + pitch, generator=g) * 0.02 - 0.002).to(F[ts or x]).cuda()[:, :groups]
        if type_w == "u4":
            zeros = torch.randint(0, 16, (m, groups + pitch), generator=g).to(torch.uint8).cuda()[:, :groups]
    xt = torch.zeros(n, k + pitch, dtype=F[x], device="cuda")[:, :k]
    xt.copy_(torch.randn(n, k, generator=g))
    return w, scales, zeros, xt


def _check(got, want, bound, what=""):
    d = (ref.f64(got) - want).abs()
    assert not bool((d > bound).any()), (what, float((d / bound.clamp(min=1e-300)).max()))


def _run(m, n, k, type_w="u4", group=128, x="bf16", d=None, **kw):
    w, scales, zeros, xt = _make(m, n, k, type_w, group, x, **kw)
    out = torch.full((n, m + 3), float("nan"), dtype=F[d or x], device="cuda")
    thl.gemm_w4(w, xt, out[:, :m], scales=scales, group=group, type_w=type_w, zeros=zeros)
    torch.cuda.synchronize()
    want, bound = ref.gemm_w4(w, type_w, scales, group, zeros, xt, k)
    _check(out[:, :m], want, bound + ref.half_step(want, out.dtype) * 1.001, (m, n, k, type_w, group))
    assert bool(torch.isnan(out[:, m:]).all())
    return w, scales, zeros, xt, out[:, :m]


@pytest.mark.parametrize("type_w,group", [("u4", 32), ("u4", 64), ("u4", 128), ("u4", 256), ("u4", 1024), ("u4", 100000),
                                          ("i4", 32), ("i4", 64), ("i4", 128), ("i4", 512), ("e2m1", 32)])
@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_groups(type_w, group, x):
    for n in (1, 19, 40):
        _run(70, n, 1536, type_w, group, x, d="f32", seed=n)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 130])
@pytest.mark.parametrize("type_w", ["u4", "e2m1"])
def test_token_counts(n, type_w):
    _run(83, n, 640, type_w, 32, d="f32", seed=n)
    _run(83, n, 640, type_w, 32, x="f16", seed=n)


@pytest.mark.parametrize("k", [1, 2, 7, 31, 32, 33, 64, 100, 255, 256, 257, 511, 1024, 1500, 2049, 8192])
@pytest.mark.parametrize("type_w,group", [("i4", 32), ("u4", 64), ("i4", 128), ("u4", 4096), ("e2m1", 32)])
def test_lengths(k, type_w, group):
    for n in (1, 21):
        _run(33, n, k, type_w, group, d="f32", seed=k)


@pytest.mark.parametrize("m", [1, 15, 16, 17, 31, 33, 100, 1003, 4096])
def test_features(m):
    for n in (1, 40):
        _run(m, n, 768, "u4", 128, seed=m)


@pytest.mark.parametrize("ts", ["f16", "bf16"])
def test_scale_types_and_pitched_rows_at_byte_offsets(ts):
    for offset in (0, 1, 5):
        for k in (512, 700):
            _run(50, 3, k, "u4", 64, "f16", d="f32", ts=ts, pitch=3, offset=offset)
            _run(50, 35, k, "i4", 32, "bf16", d="f32", ts=ts, pitch=5, offset=offset)


@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
@pytest.mark.parametrize("types", [("bf16", "bf16", "f32"), ("f32", "f16", "f16"), ("f16", "f32", "bf16")])
def test_epilogue(act, types):
    tc, td, tb = types
    m, n, k = 90, 6, 512
    w, scales, zeros, xt = _make(m, n, k)
    g = torch.Generator().manual_seed(7)
    c = torch.randn(n, m, generator=g).to(F[tc]).cuda()
    bias = torch.randn(m, generator=g).to(F[tb]).cuda()
    d = c if tc == td else torch.empty(n, m, dtype=F[td], device="cuda")  # d over c where they may be one
    c64 = ref.f64(c)
    thl.gemm_w4(w, xt, d, scales=scales, group=128, zeros=zeros, c=c, alpha=0.5, beta=2.0, bias=bias, act=act)
    torch.cuda.synchronize()
    y, b = ref.gemm_w4(w, "u4", scales, 128, zeros, xt, k)
    want = 0.5 * y + 2.0 * c64 + ref.f64(bias)
    size = 0.5 * y.abs() + 2.0 * c64.abs() + ref.f64(bias).abs()
    bound = 0.5 * b + 4 * ref.U * size
    if act == "relu":
        want = want.clamp(min=0)
    elif act == "gelu":
        # |gelu'| <= 1.13; erff within 2 ulp of 1 times |x| / 2, three products
        bound = 1.13 * bound + 8 * ref.U * want.abs()
        want = 0.5 * want * (1 + torch.erf(want / 2 ** 0.5))
    _check(d, want, bound + ref.half_step(want, d.dtype) * 1.001)


def test_every_code_and_zero_point():
    # feature i's codes are all i % 16; one nonzero activation per group: d = (q - z) s x, exact in fp32
    m, k = 64, 512
    q = torch.arange(m) % 16
    w = (q | (q << 4)).to(torch.uint8)[:, None].expand(m, k // 2).contiguous().cuda()
    scales = torch.full((m, 16), 0.5, dtype=torch.float16, device="cuda")
    zeros = (torch.arange(16)[None, :] + torch.arange(m)[:, None]).remainder(16).to(torch.uint8).cuda()
    for x in ("bf16", "f16"):
        xt = torch.zeros(16, k, dtype=F[x], device="cuda")
        for g in range(16):
            xt[g, 32 * g + g] = 2.0
        d = torch.empty(16, m, device="cuda")
        thl.gemm_w4(w, xt, d, scales=scales, group=32, zeros=zeros)
        torch.cuda.synchronize()
        assert torch.equal(d.cpu(), (q[:, None] - zeros.cpu().long()).t().float())
        s = torch.where(q >= 8, q - 16, q)
        thl.gemm_w4(w, xt, d, scales=scales, group=32, type_w="i4")
        torch.cuda.synchronize()
        assert torch.equal(d.cpu(), s.float()[None, :].expand(16, m))
        codes = torch.arange(120, 136).to(torch.uint8)[None, :].expand(m, 16).contiguous().cuda()
        thl.gemm_w4(w, xt, d, scales=codes, group=32, type_w="e2m1")
        torch.cuda.synchronize()
        v = torch.tensor(ref.E2M1 + [-e for e in ref.E2M1])[q]
        assert torch.equal(d.cpu(), v[None, :] * torch.pow(2.0, codes[0].cpu().float() - 126)[:, None])


def test_extreme_block_scales():
    m, k = 16, 64
    w = torch.full((m, k // 2), 0x22, dtype=torch.uint8, device="cuda")  # 1.0
    x = torch.zeros(2, k, dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[1, 40] = 1.0, 2.0 ** -20
    sf = torch.zeros(m, 2, dtype=torch.uint8, device="cuda")
    sf[:, 1] = 254
    sf[3, 0] = 255
    d = torch.empty(2, m, device="cuda")
    thl.gemm_w4(w, x, d, scales=sf, group=32, type_w="e2m1")
    torch.cuda.synchronize()
    keep = torch.arange(m) != 3
    assert bool((d[0].cpu()[keep] == 2.0 ** -127).all()) and bool((d[1].cpu()[keep] == 2.0 ** 107).all())
    assert bool(torch.isnan(d[:, 3]).all())


@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 2, 3, 20, 50])
def test_block_scales_of_the_whole_range(n, x):
    # feature i has code 1 + i % 7 under every scale byte in turn, and token t one
    # nonzero activation, in block t: products that are exact in fp32 wherever they are
    # in its range, also where the weight itself is none of bf16's numbers
    m, k = 130, 32 * 64
    blocks = [0, 1, 2, 3, 4, 5, 124, 127, 130, 250, 251, 252, 253, 254, 9]
    q = 1 + torch.arange(m) % 7
    w = (q | (q << 4)).to(torch.uint8)[:, None].expand(m, k // 2).contiguous().cuda()
    v = torch.tensor(ref.E2M1, dtype=torch.float64)[q]
    sf = torch.full((m, 64), 127, dtype=torch.uint8)
    xt = torch.zeros(n, k, dtype=F[x])
    want = torch.empty(n, m, dtype=torch.float64)
    for t in range(n):
        b, code = (3 * t) % 64, blocks[t % len(blocks)]
        sf[:, b] = code
        xt[t, 32 * b + 5] = 2.0 ** (-12 if code > 127 else 6)
        want[t] = v * float(xt[t, 32 * b + 5]) * 2.0 ** (code - 127)
    d = torch.empty(n, m, device="cuda")
    thl.gemm_w4(w, xt.cuda(), d, scales=sf.cuda(), group=32, type_w="e2m1")
    torch.cuda.synchronize()
    assert torch.equal(d.cpu().double(), want)
    sf[3, 40] = 255
    thl.gemm_w4(w, xt.cuda(), d, scales=sf.cuda(), group=32, type_w="e2m1")
    torch.cuda.synchronize()
    keep = torch.arange(m) != 3
    assert torch.equal(d.cpu().double()[:, keep], want[:, keep]) and bool(torch.isnan(d[:, 3]).all())


def test_infinities_stay_in_their_token():
    w, scales, zeros, xt = _make(40, 5, 300, "u4", 64)
    xt[1, 7], xt[3, 299] = float("inf"), float("nan")
    d = torch.empty(5, 40, device="cuda")
    thl.gemm_w4(w, xt, d, scales=scales, group=64, zeros=zeros)
    torch.cuda.synchronize()
    assert bool(torch.isnan(d[1]).all()) and bool(torch.isnan(d[3]).all())
    rest = [0, 2, 4]
    want, bound = ref.gemm_w4(w, "u4", scales, 64, zeros, xt[rest], 300)
    _check(d[rest], want, bound + ref.half_step(want, torch.float32))


def test_k_zero_is_the_epilogue():
    bias = torch.randn(20, device="cuda")
    d = torch.empty(3, 20, device="cuda")
    e = torch.empty(3, 0, dtype=torch.bfloat16, device="cuda")
    thl.gemm_w4(torch.empty(20, 0, dtype=torch.uint8, device="cuda"), e, d, scales=torch.empty(20, 0, dtype=torch.float16, device="cuda"),
                group=32, type_w="i4", bias=bias, act="relu")
    torch.cuda.synchronize()
    assert torch.equal(d, bias.clamp(min=0).expand(3, 20))


def test_offsets_past_32_bits():
    # feature rows 2^26 bytes apart: the last of 70 lies past 2^32 bytes
    m, k, pitch = 70, 512, 1 << 26
    big = torch.empty(m * pitch, dtype=torch.uint8, device="cuda").view(m, pitch)
    w = big[:, :k // 2]
    w0, scales, zeros, xt = _make(m, 2, k)
    w.copy_(w0)
    d = torch.empty(2, m, device="cuda")
    thl.gemm_w4(w, xt, d, scales=scales, group=128, zeros=zeros)
    torch.cuda.synchronize()
    want, bound = ref.gemm_w4(w0, "u4", scales, 128, zeros, xt, k)
    _check(d, want, bound + ref.half_step(want, torch.float32))


def test_results_do_not_depend_on_timing():
    w, scales, zeros, xt, d = _run(1000, 7, 4096)
    for _ in range(3):
        d2 = torch.empty_like(d)
        thl.gemm_w4(w, xt, d2, scales=scales, group=128, zeros=zeros)
        torch.cuda.synchronize()
        assert torch.equal(d, d2)


@pytest.mark.parametrize("bad", ["shape", "zeros", "scales", "type", "beta"])
def test_torch_form_refusals(bad):
    w, scales, zeros, xt = _make(32, 2, 256)
    d = torch.empty(2, 32, device="cuda")
    kw = dict(scales=scales, group=128, zeros=zeros)
    with pytest.raises((ValueError, thl.ThlError)):
        if bad == "shape":
            thl.gemm_w4(w[:, :100], xt, d, **kw)
        elif bad == "zeros":
            thl.gemm_w4(w, xt, d, scales=scales, group=128)
        elif bad == "scales":
            thl.gemm_w4(w, xt, d, scales=scales[:, :1], group=128, zeros=zeros)
        elif bad == "type":
            thl.gemm_w4(w, xt.float(), d, **kw)
        else:
            thl.gemm_w4(w, xt, d, beta=1.0, **kw)


@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 2, 3, 40])
@pytest.mark.parametrize("type_w,group", [("u4", 32), ("i4", 128), ("e2m1", 32)])
def test_subnormal_activations(type_w, group, x, n):
    # one nonzero activation a token, below the format's normal numbers: exact in fp32
    m, k = 40, 1024
    w, _, zeros, _ = _make(m, n, k, type_w, group, x)
    scales = torch.full((m, k // group), 127 if type_w == "e2m1" else 1.0,
                        dtype=torch.uint8 if type_w == "e2m1" else F[x], device="cuda")
    xt = torch.zeros(n, k, dtype=F[x])
    for t in range(n):
        xt[t, (37 * t + 5) % k] = (3 + t) * (2.0 ** -24 if x == "f16" else 2.0 ** -133)
    assert bool((xt.abs().amax(dim=1) < torch.finfo(F[x]).tiny).all()) and bool((xt.abs().amax(dim=1) > 0).all())
    up = 2.0 ** 20  # the sums themselves stay normal in fp32
    d = torch.empty(n, m, device="cuda")
    thl.gemm_w4(w, xt.cuda(), d, scales=scales, group=group, type_w=type_w, zeros=zeros, alpha=up)
    torch.cuda.synchronize()
    want, _ = ref.gemm_w4(w, type_w, scales, group, zeros, xt.cuda(), k)
    assert torch.equal(d.double().cpu(), want.cpu() * up)


@pytest.mark.parametrize("type_w", ["u4", "i4", "e2m1"])
@pytest.mark.parametrize("n", [1, 2, 3, 20])
def test_large_finite_activations(type_w, n):
    """The largest activations that the sums before a group's scale leave finite: their magnitudes, times 31 (271 with
    the largest zero point, 6 for E2M1), stay below 2^128.  One activation a token, of 2^123 (2^119, 2^125); the
    products are exact, and so is a result that is small or zero."""
    m, k = 48, 512
    group = 32 if type_w == "e2m1" else 128
    w, _, _, _ = _make(m, n, k, type_w, group)
    for z, size in {"u4": ((15, 2.0 ** 123), (255, 2.0 ** 119)), "i4": ((0, 2.0 ** 123),),
                    "e2m1": ((0, 2.0 ** 125),)}[type_w]:
        zeros = torch.full((m, k // group), z, dtype=torch.uint8, device="cuda") if type_w == "u4" else None
        scales = (torch.full((m, k // group), 117, dtype=torch.uint8, device="cuda") if type_w == "e2m1" else
                  torch.full((m, k // group), 2.0 ** -10, dtype=torch.bfloat16, device="cuda"))
        xt = torch.zeros(n, k, dtype=torch.bfloat16)
        for t in range(n):
            xt[t, (41 * t + 9) % k] = size * (1 if t % 2 else -1)
        d = torch.empty(n, m, device="cuda")
        thl.gemm_w4(w, xt.cuda(), d, scales=scales, group=group, type_w=type_w, zeros=zeros)
        torch.cuda.synchronize()
        want, _ = ref.gemm_w4(w, type_w, scales, group, zeros, xt, k)
        assert torch.equal(d.double().cpu(), want)
        assert type_w != "u4" or z != 15 or bool((want == 0).any())  # some code is the zero point


@pytest.mark.parametrize("n", [1, 2, 3, 20])
def test_activations_as_large_as_bf16_sums_allow(n):
    # every activation at 4e33 and the largest zero point: 256 of them times 271 are finite, and so is every result
    m, k, group = 40, 1024, 256
    w, _, _, _ = _make(m, n, k, "u4", group)
    zeros = torch.full((m, k // group), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((m, k // group), 2.0 ** -4, dtype=torch.bfloat16, device="cuda")
    xt = torch.full((n, k), 4e33, dtype=torch.bfloat16, device="cuda")
    d = torch.empty(n, m, device="cuda")
    thl.gemm_w4(w, xt, d, scales=scales, group=group, zeros=zeros)
    torch.cuda.synchronize()
    want, bound = ref.gemm_w4(w, "u4", scales, group, zeros, xt, k)
    # the oracle's bound counts terms of up to 31 |x|; here the zero point's are up to 271 |x|
    _check(d, want, bound * 271 / 31 + ref.half_step(want, torch.float32))


def _exact(m, n, k, type_w, group, x, seed=0):
    """Small whole activations, scales that are powers of two: every product and sum is a multiple of 1/8 (a scale of
    1/4 times a step of 1/2) below 2^20, so exact in fp32, in any order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    groups = -(-k // group)
    assert k * 3 * (31 + 15) < 2 ** 22  # |x| <= 3 times 16 + q and 16 + z, in steps of 1/4
    w = torch.randint(0, 256, (m, (k + 1) // 2), generator=g, device="cuda").to(torch.uint8)
    xt = torch.randint(-3, 4, (n, k), generator=g, device="cuda").to(F[x])
    e = torch.randint(-2, 1, (m, groups), generator=g, device="cuda")
    zeros = torch.randint(0, 16, (m, groups), generator=g, device="cuda").to(torch.uint8) if type_w == "u4" else None
    scales = (127 + e).to(torch.uint8) if type_w == "e2m1" else torch.pow(2.0, e.float()).to(F[x])
    d = torch.full((n, m), float("nan"), device="cuda")
    thl.gemm_w4(w, xt, d, scales=scales, group=group, type_w=type_w, zeros=zeros)
    torch.cuda.synchronize()
    values = torch.tensor(ref.E2M1 + [-v for v in ref.E2M1] if type_w == "e2m1" else
                          [float(q if q < 8 or type_w == "u4" else q - 16) for q in range(16)], dtype=torch.float64,
                          device="cuda")
    x64 = xt.double().t().contiguous()
    at = (torch.arange(k, device="cuda") // group)
    for a in range(0, m, 4096):  # pieces of the fp64 form
        c = slice(a, min(m, a + 4096))
        v = values[torch.stack([w[c] & 15, w[c] >> 4], dim=2).reshape(w[c].shape[0], -1)[:, :k].int()]
        if zeros is not None:
            v -= zeros[c].double()[:, at]
        v *= torch.pow(2.0, e[c].double())[:, at]
        want = (v @ x64).t()
        assert torch.equal(d[:, c].double(), want), (a, int((d[:, c].double() != want).sum()))


# one and two tokens: K over 1 to 8 wavefronts, several slices each, a part of a piece at its end, and several
# blocks of rows a workgroup
@pytest.mark.parametrize("m,k", [(40000, 1536), (4200, 2048), (4200, 4096), (4200, 6144), (28672, 8192), (4200, 10240),
                                 (4200, 12288), (4200, 14336), (9000, 16384), (9000, 20493), (4200, 27000)])
@pytest.mark.parametrize("type_w,group", [("u4", 128), ("i4", 64), ("e2m1", 32), ("u4", 1 << 20)])
def test_down_the_rows(m, k, type_w, group):
    for n in (1, 2):
        _exact(m, n, k, type_w, group, "bf16" if n == 1 else "f16", seed=k)


# more tokens: so many features that K is not split, and a workgroup goes through sixteen units and a part of one
@pytest.mark.parametrize("type_w,group", [("u4", 32), ("u4", 64), ("u4", 128), ("u4", 256), ("u4", 1 << 20), ("i4", 32),
                                          ("i4", 64), ("i4", 128), ("i4", 1024), ("e2m1", 32)])
@pytest.mark.parametrize("n", [3, 12, 20, 40, 64, 100])
def test_along_k(type_w, group, n):
    _exact(33000, n, 4166, type_w, group, "bf16", seed=n)
    _exact(28672, n, 4096, type_w, group, "f16", seed=n)


# and so few that it is split, with several sets of units a workgroup
@pytest.mark.parametrize("type_w,group", [("u4", 128), ("i4", 32), ("e2m1", 32)])
@pytest.mark.parametrize("n", [8, 24, 48, 64])
def test_along_split_k(type_w, group, n):
    assert thl.thl_gemm_w4_workspace(8192, n, 8192) > 0
    _exact(8192, n, 8192, type_w, group, "bf16", seed=n)
    _exact(5000, n, 20493, type_w, group, "f16", seed=n)


@pytest.mark.parametrize("m,n,k", [(1 << 26, 1, 32), (1 << 26, 3, 40), (130, 1 << 21, 70)])
def test_most_features_and_most_tokens(m, n, k):
    _exact(m, n, k, "i4", 32, "bf16", seed=n)
