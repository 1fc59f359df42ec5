"""thl.rmsnorm and its gradient against the plain fp64 forms, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import tile_hierarchy_linear_amd as thl
from oracle import operators as ref

pytestmark = pytest.mark.gpu
F = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
     "e5m2": torch.float8_e5m2}
EPS = 1e-5


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _rand(seed, *shape, dtype="f32", scale=1.0, pitch=0, offset=0):
    """A (n, m) tensor on the GPU, rows `pitch` elements past m apart, starting `offset` elements in."""
    g = torch.Generator().manual_seed(seed)
    v = (torch.randn(*shape, generator=g) * scale).to(F[dtype])
    if v.dim() == 2 and (pitch or offset):
        n, m = shape
        big = torch.zeros(offset + n * (m + pitch), dtype=F[dtype], device="cuda")
        view = big[offset:].view(n, m + pitch)[:, :m]
        view.copy_(v)
        return view
    return v.cuda()


def _check(got, want, bound, what):
    d = (ref.f64(got) - want).abs()
    over = d > bound
    assert not bool(over.any()), (what, int(over.sum()), float((d / bound.clamp(min=1e-300)).max()))


def _check_float(got, want, rel, what):
    _check(got, want, rel * want.abs() + ref.half_step(want, got.dtype) * (1 + 2 * rel), what)


def _check_narrow(values, want, kind, err):
    """values (before the block scale) of a narrow format against unrounded ones with absolute error err."""
    top = ref.TOP[kind]
    c = torch.clamp(want, -top, top)
    _check(values, c, ref.narrow_half_step(c, kind) * 1.0 + 2 * err, kind)


def _run(n, m, x="bf16", res=None, w=None, y="bf16", mx=False, scale=1.0, pitch=0, offset=0, seed=0, xt=None,
         keep_sum=True):
    xt = _rand(seed, n, m, dtype=x, pitch=pitch, offset=offset) if xt is None else xt
    rt = _rand(seed + 1, n, m, dtype=res, scale=3.0, pitch=pitch, offset=offset) if res else None
    wt = (1 + 0.3 * _rand(seed + 2, m)).to(F[w or x])
    st = torch.full_like(rt, float("nan")) if res and keep_sum else None
    if y == "e2m1":
        yt = torch.full((n, (m + 1) // 2 + pitch), 0xEE, dtype=torch.uint8, device="cuda")[:, :(m + 1) // 2]
    elif y in ref.TOP:
        yt = torch.full((n, m + pitch), 0xEE, dtype=torch.uint8, device="cuda")[:, :m].view(F[y])
    else:
        yt = torch.full((n, m + pitch), float("nan"), dtype=F[y], device="cuda")[:, :m]
    nb = (m + 31) // 32
    sf = torch.full((n, nb + 3), 0xEE, dtype=torch.uint8, device="cuda") if mx else None
    before = (xt.clone(), None if rt is None else rt.clone())
    thl.rmsnorm(xt, wt, yt, eps=EPS, residual=rt, residual_out=st, scale=scale, sf=sf)
    torch.cuda.synchronize()
    assert torch.equal(before[0].view(torch.uint8), xt.contiguous().view(torch.uint8)) if m else True
    s, want, rel = ref.rmsnorm(xt, rt, wt, EPS)
    if st is not None:
        _check(st, s, ref.half_step(s, st.dtype) + ref.U * s.abs(), "sum")
    if mx:
        kind = y
        code = sf.cpu()[:, :nb].to(torch.int64)
        assert bool((sf[:, nb:] == 0xEE).all())  # scale padding untouched
        pad = torch.nn.functional.pad(want, (0, 32 * nb - m)).reshape(n, nb, 32)
        amax = pad.abs().amax(dim=2)
        # the code is that of some value within the fp32 error of the maximum
        lo = torch.floor(torch.log2((amax * (1 - rel)).clamp(min=1e-300)))
        hi = torch.floor(torch.log2((amax * (1 + rel)).clamp(min=1e-300)))
        lo, hi = ((v - ref.EMAX[kind]).clamp(-127, 127) + 127 for v in (lo, hi))
        lo, hi = torch.where(amax > 0, lo, 0.0), torch.where(amax > 0, hi, 0.0)
        assert bool(((code >= lo) & (code <= hi)).all())
        x2 = torch.pow(2.0, code.double() - 127)
        each = x2.repeat_interleave(32, dim=1)[:, :m]
        values = ref.e2m1_values(yt, m) if kind == "e2m1" else ref.f64(yt)
        _check_narrow(values, want / each, kind, rel * want.abs() / each)
    elif y in ref.TOP:
        _check_narrow(ref.f64(yt), want / scale, y, (rel + ref.U) * want.abs() / scale)
    else:
        _check_float(yt, want, rel, "y")
    return xt, rt, st, yt, sf


# 512 and 16,384: the last features of a variant; 16,385 on: the token read twice
@pytest.mark.parametrize("m", [1, 7, 31, 33, 100, 512, 513, 1024, 1500, 2048, 2049, 4099, 8192, 8200, 16384, 16385,
                               20011])
@pytest.mark.parametrize("n", [1, 3])
def test_widths(n, m):
    _run(n, m, res="bf16", seed=m)


@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("res", [None, "same", "f32"])
@pytest.mark.parametrize("y", ["bf16", "f16", "f32"])
def test_types(x, res, y):
    _run(5, 777, x=x, res=x if res == "same" else res, y=y, w="f32" if y == "f16" else None)
    _run(2, 16999, x=x, res=x if res == "same" else res, y=y)


@pytest.mark.parametrize("y", ["e4m3", "e5m2"])
@pytest.mark.parametrize("scale", [1.0, 0.0123, 0.001])  # the last clamps part of them
@pytest.mark.parametrize("m", [40, 1001, 5003, 17000])
def test_one_scale(y, scale, m):
    _run(4, m, y=y, scale=scale, res="f32", pitch=5)


@pytest.mark.parametrize("y", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("m", [1, 32, 33, 63, 64, 1000, 2047, 4096, 8224, 16390, 20000])
def test_mx_blocks(y, m):
    _run(3, m, y=y, mx=True, res="bf16", seed=m)


@pytest.mark.parametrize("m", [65, 4099, 16411])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_pitched_rows_at_element_offsets(m, offset):
    for x in ("f16", "f32"):
        _run(6, m, x=x, res=x, y="f32", pitch=3, offset=offset)


def test_many_tokens_walk_the_grid():
    _run(40000, 72, res="bf16")
    _run(9000, 2100, y="e4m3", mx=True)


def test_in_place():
    # the residual stream updated in place and the output over the input: the same bits as out of place
    for m in (600, 4096, 16500):
        x, r, s, y, _ = _run(5, m, res="bf16")
        w = (1 + 0.3 * _rand(2, m)).to(F["bf16"])
        thl.rmsnorm(x, w, x, eps=EPS, residual=r, residual_out=r)
        torch.cuda.synchronize()
        assert torch.equal(x, y) and torch.equal(r, s)
        x, r, s, y, _ = _run(5, m, res="bf16", y="f32")
        y2 = torch.empty_like(y)
        thl.rmsnorm(x, w, y2, eps=EPS, residual=r, residual_out=x)  # the sum over x
        torch.cuda.synchronize()
        assert torch.equal(x, s) and torch.equal(y, y2)


def test_sum_not_kept_and_padding_untouched():
    _run(4, 100, res="f32", keep_sum=False)
    y = torch.full((4, 128), 7.0, device="cuda")
    thl.rmsnorm(_rand(0, 4, 100), _rand(1, 100), y[:, :100], eps=EPS)
    torch.cuda.synchronize()
    assert bool((y[:, 100:] == 7.0).all())


def test_zero_tokens_infinities_and_nan():
    x = _rand(0, 5, 300, dtype="bf16")
    x[0] = 0.0
    x[1, 7] = float("inf")
    x[2, 299] = float("nan")
    w = torch.ones(300, device="cuda")
    y = torch.empty(5, 300, device="cuda")
    thl.rmsnorm(x, w, y, eps=EPS)
    torch.cuda.synchronize()
    assert bool((y[0] == 0).all())
    assert bool(torch.isnan(y[1, 7])) and bool((y[1, :7] == 0).all())  # inf * 0, and finite / inf
    assert bool(torch.isnan(y[2]).all())
    _, want, rel = ref.rmsnorm(x[3:], None, w, EPS)
    _check_float(y[3:], want, rel, "the other tokens")
    thl.rmsnorm(x, w, y, eps=0.0)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[0]).all())  # 0 / 0
    q = torch.empty(5, 300, dtype=torch.float8_e4m3fn, device="cuda")
    sf = torch.zeros(5, 16, dtype=torch.uint8, device="cuda")
    thl.rmsnorm(x, w, q, eps=EPS, sf=sf)
    torch.cuda.synchronize()
    assert bool((sf[0, :10] == 0).all()) and bool((q[0].float() == 0).all())
    assert bool(torch.isnan(q[2].float()).all())


def test_empty():
    w = torch.ones(8, device="cuda")
    thl.rmsnorm(torch.empty(0, 8, device="cuda"), w, torch.empty(0, 8, device="cuda"))
    thl.rmsnorm(torch.empty(3, 0, device="cuda"), w[:0], torch.empty(3, 0, device="cuda"))
    dw = torch.full((8,), 5.0, device="cuda")
    e = torch.empty(0, 8, device="cuda")
    thl.rmsnorm_backward(e, e, w, torch.empty_like(e), dw)
    torch.cuda.synchronize()
    assert bool((dw == 0).all())


def test_offsets_past_32_bits():
    # rows 2^20 elements apart: token 4,200's features lie past 2^32 elements
    n, m, pitch = 4200, 64, 1 << 20
    big = torch.zeros(n * pitch, dtype=torch.bfloat16, device="cuda")
    x = big.view(n, pitch)[:, :m]
    x.copy_(_rand(0, n, m, dtype="bf16"))
    w, y = torch.ones(m, device="cuda"), torch.empty(n, m, device="cuda")
    thl.rmsnorm(x, w, y, eps=EPS)
    torch.cuda.synchronize()
    _, want, rel = ref.rmsnorm(x, None, w, EPS)
    _check_float(y, want, rel, "y")


# ------------------------------------------------------------------ gradient

def _grad(n, m, s="bf16", g="bf16", w=None, dres=True, dw="f32", pitch=0, seed=0):
    st = _rand(seed, n, m, dtype=s, scale=2.0, pitch=pitch)
    dy = _rand(seed + 1, n, m, dtype=g, pitch=pitch)
    dr = _rand(seed + 2, n, m, dtype=g, pitch=pitch) if dres else None
    wt = (1 + 0.3 * _rand(seed + 3, m)).to(F[w or s])
    dx = torch.full((n, m + pitch), float("nan"), dtype=F[g], device="cuda")[:, :m]
    dwt = torch.full((m,), float("nan"), dtype=F[dw], device="cuda") if dw else None
    thl.rmsnorm_backward(st, dy, wt, dx, dwt, eps=EPS, dres=dr)
    torch.cuda.synchronize()
    want_x, want_w, bx, bw = ref.rmsnorm_backward(st, dy, wt, dr, EPS)
    _check(dx, want_x, bx + ref.half_step(want_x, dx.dtype) * 1.001, "dx")
    if dw:
        _check(dwt, want_w, bw + ref.half_step(want_w, dwt.dtype) * 1.001, "dw")
    return st, dy, dr, wt, dx, dwt


@pytest.mark.parametrize("m", [1, 9, 500, 513, 2048, 2050, 4096, 5003, 8193, 16384, 16390])
@pytest.mark.parametrize("n", [1, 40])
def test_backward_widths(n, m):
    _grad(n, m, seed=m)


@pytest.mark.parametrize("s", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("g", ["bf16", "f16", "f32"])
def test_backward_types(s, g):
    _grad(37, 1203, s=s, g=g, dres=False, pitch=1)
    _grad(3, 17001, s=s, g=g, w="f32")
    _grad(3, 12000, s=s, g=g, dw=s if s != "f32" else "f32")


def test_backward_many_tokens():
    _grad(3000, 136, s="f32", g="f32")
    _grad(1500, 16392, dres=False)  # several tokens a workgroup on the path that reads twice


@pytest.mark.parametrize("n,m", [(4099, 227), (5000, 600), (4200, 1500), (600, 5003), (520, 8192), (300, 9001), (270, 16384)])
@pytest.mark.parametrize("g", ["bf16", "f32"])
def test_backward_more_tokens_than_workgroups(n, m, g):
    _grad(n, m, s="f32" if g == "f32" else "bf16", g=g, seed=n)


@pytest.mark.parametrize("n,m", [(300, 9001), (2, 6000)])
def test_backward_long_tokens_in_place(n, m):
    st, dy, dr, w, dx, dw = _grad(n, m, seed=5)
    for out in (dy, dr, st):
        keep, dw2 = out.clone(), torch.empty_like(dw)
        thl.rmsnorm_backward(st, dy, w, out, dw2, eps=EPS, dres=dr)
        torch.cuda.synchronize()
        assert torch.equal(out, dx) and torch.equal(dw2, dw)
        out.copy_(keep)


def test_backward_without_dw_and_in_place():
    st, dy, dr, w, dx, _ = _grad(600, 1000)
    thl.rmsnorm_backward(st, dy, w, dy, None, eps=EPS, dres=dr)  # dx over dy
    torch.cuda.synchronize()
    assert torch.equal(dy, dx)
    for m in (700, 16600):
        st, dy, dr, w, dx, dw = _grad(600, m, seed=5)
        dw2 = torch.empty_like(dw)
        thl.rmsnorm_backward(st, dy, w, st, dw2, eps=EPS, dres=dr)  # dx over s
        torch.cuda.synchronize()
        assert torch.equal(st, dx) and torch.equal(dw, dw2)


def test_backward_against_differences():
    """The directional derivative of the fp64 norm by central differences.  With step h the difference is off by
    h^2 / 6 times a third derivative of order one times the function's scale: 1e-8 relative at h = 1e-4, far below
    the kernel's own fp32 error, 1e-5 of the sum of magnitudes."""
    n, m, h = 6, 90, 1e-4
    x, dy, w = _rand(0, n, m), _rand(1, n, m), 1 + 0.3 * _rand(2, m)
    dx, dw = torch.empty_like(x), torch.empty(m, device="cuda")
    thl.rmsnorm_backward(x, dy, w, dx, dw, eps=EPS)
    torch.cuda.synchronize()
    dirs = torch.randn(n, m, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    wdir = torch.randn(m, generator=torch.Generator().manual_seed(4), dtype=torch.float64)
    X, DY, W = ref.f64(x), ref.f64(dy), ref.f64(w)

    def loss(a, b):
        return float((ref.rmsnorm(a, None, b, EPS)[1] * DY).sum())

    num = (loss(X + h * dirs, W) - loss(X - h * dirs, W)) / (2 * h)
    got = ref.f64(dx) * dirs
    assert abs(num - float(got.sum())) <= 1e-5 * float(got.abs().sum())
    num = (loss(X, W + h * wdir) - loss(X, W - h * wdir)) / (2 * h)
    got = ref.f64(dw) * wdir
    assert abs(num - float(got.sum())) <= 1e-5 * float(got.abs().sum())


def test_results_do_not_depend_on_timing():
    a = _grad(2000, 1024, seed=9)
    for _ in range(3):
        dw = torch.empty_like(a[5])
        thl.rmsnorm_backward(a[0], a[1], a[3], torch.empty_like(a[4]), dw, eps=EPS, dres=a[2])
        torch.cuda.synchronize()
        assert torch.equal(dw, a[5])


@pytest.mark.parametrize("bad", ["shape", "stride", "type", "device", "sum", "grads"])
def test_torch_form_refusals(bad):
    x, w, y = _rand(0, 4, 64), _rand(1, 64), torch.empty(4, 64, device="cuda")
    with pytest.raises((ValueError, thl.ThlError)):
        if bad == "shape":
            thl.rmsnorm(x, w, y[:3])
        elif bad == "stride":
            thl.rmsnorm(x, w, torch.empty(64, 4, device="cuda").t())
        elif bad == "type":
            thl.rmsnorm(x.double(), w, y)
        elif bad == "device":
            thl.rmsnorm(x, w.cpu(), y)
        elif bad == "sum":
            thl.rmsnorm(x, w, y, residual_out=y)
        else:
            thl.rmsnorm_backward(x, x, w, torch.empty(4, 64, device="cuda", dtype=torch.float16))


@pytest.mark.parametrize("y", ["e4m3", "e5m2"])
@pytest.mark.parametrize("m", [1024, 1003, 16500])  # 1003: a ragged row; 16,500: the token read twice
def test_one_scale_is_a_product_with_its_reciprocal(y, m):
    """x all ones and eps = 0: the norm of ones is exactly w, so y is w * (1 / scale) in fp32, rounded once more.  The
    weights are where the quotient lies on or next to a midpoint of two codes, which a division would now and then
    leave to the other side."""
    top = ref.TOP[y]
    codes = torch.arange(1, 256, dtype=torch.uint8).view(F[y]).float()
    codes = torch.sort(codes[torch.isfinite(codes) & (codes > 0)]).values
    mids = (codes[1:].double() + codes[:-1].double()) / 2
    x, differ = torch.ones(2, m, device="cuda"), 0  # codes that a division gives otherwise
    for scale in (0.02, 0.0123, 0.7, 3.0, 1.7e-30, 3.1e29):
        s = torch.tensor(scale, dtype=torch.float32)
        near = (mids * s.double()).float()
        w = torch.cat([near, torch.nextafter(near, torch.tensor(0.0)), -torch.nextafter(near, torch.tensor(torch.inf)),
                       torch.tensor([0.0, -0.0, 3e38, -3e38, torch.inf, 1e-45, 1e-38])])
        w = w.repeat(-(-m // w.numel()))[:m]
        q = w * (1 / s)  # both rounded in fp32
        want = q.clamp(-top, top).to(F[y]).view(torch.uint8)
        differ += int(((w / s).clamp(-top, top).to(F[y]).view(torch.uint8) != want).sum())
        got = torch.empty(2, m, dtype=F[y], device="cuda")
        thl.rmsnorm(x, w.cuda(), got, eps=0.0, scale=float(s))
        torch.cuda.synchronize()
        got = got.view(torch.uint8).cpu()
        assert torch.equal(got[0], want) and torch.equal(got[1], want), scale
    assert differ > 0  # a division is something else


def test_one_scale_keeps_nan():
    w = torch.ones(64, device="cuda")
    w[5] = float("nan")
    y = torch.empty(1, 64, dtype=torch.float8_e4m3fn, device="cuda")
    thl.rmsnorm(torch.ones(1, 64, device="cuda"), w, y, eps=0.0, scale=0.3)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[0, 5].float())) and not bool(torch.isnan(y.float()[0, torch.arange(64) != 5]).any())


@pytest.mark.parametrize("m", [64, 1003, 17000])
def test_range_of_the_squares(m):
    # every feature +-2^e: sums of squares m 2^(2e), inside fp32's range up to e = 56 and past it from 64 on
    sign = torch.where(torch.arange(m) % 3 == 0, -1.0, 1.0)
    w, y = torch.ones(m, device="cuda"), torch.empty(1, m, device="cuda")
    rel = ref.rmsnorm(torch.ones(1, m), None, torch.ones(m), 0.0)[2]
    for e in (-56, -1, 0, 56):
        thl.rmsnorm((sign * 2.0 ** e).cuda().reshape(1, m), w, y, eps=0.0)
        torch.cuda.synchronize()
        _check_float(y, sign.double().reshape(1, m), rel, e)
    thl.rmsnorm((sign * 2.0 ** 64).cuda().reshape(1, m), w, y, eps=EPS)
    torch.cuda.synchronize()
    assert bool((y == 0).all())
    thl.rmsnorm((sign * 2.0 ** -80).cuda().reshape(1, m), w, y, eps=0.0)
    torch.cuda.synchronize()
    assert bool(torch.isinf(y).all())


def _plain64(x, r, w):
    """(s, y) in fp64 on the GPU."""
    s = x.double() if r is None else x.double() + r.double()
    return s, s * torch.rsqrt(s.square().mean(dim=1, keepdim=True) + EPS) * w.double()


def _near(got, want, bound):
    return bool(((got.double() - want).abs() <= bound).all())


# more tokens than workgroups (8,192 of four wavefronts, 2,048 of sixteen), for every width from 1,025 on, whole and ragged
@pytest.mark.parametrize("n,m", [(1100, 4104), (1100, 6000), (1100, 6152), (1100, 8192), (8300, 1800), (8300, 2050),
                                 (8300, 4096), (8300, 4099), (8300, 6144), (8300, 6147), (8300, 8192), (2100, 8195),
                                 (2100, 16384), (2100, 16411)])
@pytest.mark.parametrize("x,res,y", [("bf16", "bf16", "bf16"), ("f16", "f32", "f32")])
def test_more_tokens_than_workgroups(n, m, x, res, y):
    g = torch.Generator(device="cuda").manual_seed(m)
    xt = torch.randn(n, m, generator=g, device="cuda").to(F[x])
    rt = (3 * torch.randn(n, m, generator=g, device="cuda")).to(F[res])
    wt = (1 + 0.3 * torch.randn(m, generator=g, device="cuda")).to(F[x])
    st, yt = torch.full_like(rt, float("nan")), torch.full((n, m), float("nan"), dtype=F[y], device="cuda")
    thl.rmsnorm(xt, wt, yt, eps=EPS, residual=rt, residual_out=st)
    torch.cuda.synchronize()
    rel = ref.rmsnorm(xt[:1], rt[:1], wt, EPS)[2]
    for a in range(0, n, 1024):  # pieces of the fp64 form
        c = slice(a, min(n, a + 1024))
        s, want = _plain64(xt[c], rt[c], wt)
        assert _near(st[c], s, ref.half_step(s, st.dtype) + ref.U * s.abs())
        assert _near(yt[c], want, rel * want.abs() + ref.half_step(want, yt.dtype) * (1 + 2 * rel))


# widths off eight: the last two runs of a row overlap, and every lane has to read before any stores
@pytest.mark.parametrize("m", [9, 65, 777, 1025, 2049, 4099, 6147, 8195, 12001, 16411])
@pytest.mark.parametrize("n", [5, 1100])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_ragged_rows_in_place(m, n, x):
    g = torch.Generator(device="cuda").manual_seed(m)
    xt = torch.randn(n, m, generator=g, device="cuda").to(F[x])
    rt = (3 * torch.randn(n, m, generator=g, device="cuda")).to(F[x])
    wt = (1 + 0.3 * torch.randn(m, generator=g, device="cuda")).to(F[x])
    st, yt = torch.empty_like(xt), torch.empty_like(xt)
    thl.rmsnorm(xt, wt, yt, eps=EPS, residual=rt, residual_out=st)
    for over in ("s over r, y over x", "s over x", "y over x"):
        x2, r2, s2, y2 = xt.clone(), rt.clone(), torch.empty_like(xt), torch.empty_like(xt)
        s2 = r2 if over.startswith("s over r") else x2 if over == "s over x" else s2
        y2 = x2 if "y over x" in over else y2
        thl.rmsnorm(x2, wt, y2, eps=EPS, residual=r2, residual_out=s2)
        torch.cuda.synchronize()
        assert torch.equal(s2, st) and torch.equal(y2, yt), over


@pytest.mark.parametrize("n,m", [(700, 2056), (600, 3001), (1300, 4096), (5000, 1024), (4500, 513), (4200, 2048),
                                 (1100, 6000), (600, 12288)])
@pytest.mark.parametrize("g", ["bf16", "f32"])
def test_backward_sums_dw_over_tokens_of_a_workgroup(n, m, g):
    _grad(n, m, s="f32" if g == "f32" else "bf16", g=g, seed=n)


def test_longest_tokens():
    # 2^26 features, the most that a call takes: sums, gradients and dw against fp64 on the GPU
    m = 1 << 26
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, m, generator=g, device="cuda").bfloat16()
    dy = torch.randn(1, m, generator=g, device="cuda").bfloat16()
    w = (1 + 0.3 * torch.randn(m, generator=g, device="cuda")).bfloat16()
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(m, device="cuda")
    thl.rmsnorm(x, w, y, eps=EPS)
    thl.rmsnorm_backward(x, dy, w, dx, dw, eps=EPS)
    torch.cuda.synchronize()
    X, G, W = x.double(), dy.double(), w.double()
    rho = torch.rsqrt(X.square().mean(dim=1, keepdim=True) + EPS)
    terms = 64 + m / 8192 + 22  # as the oracle counts them
    rel = (terms / 2 + 8) * ref.U
    want = X * rho * W
    assert _near(y, want, rel * want.abs() + ref.half_step(want, y.dtype) * (1 + 2 * rel))
    h, t = rho * X, W * G
    want = rho * (t - h * (t * h).mean(dim=1, keepdim=True))
    c = 3 * (terms + 8) * ref.U
    bound = c * rho * (t.abs() + h.abs() * (t * h).abs().mean(dim=1, keepdim=True))
    assert _near(dx, want, bound + ref.half_step(want, dx.dtype) * 1.001)
    want = (G * h)[0]
    assert _near(dw, want, (rel + 4 * ref.U) * want.abs() + ref.half_step(want, dw.dtype))


@pytest.mark.parametrize("m", [40, 300, 2050, 16400])
def test_nan_in_fp4_blocks(m):
    """A block of E2M1 that holds a NaN has the scale NaN: its elements have no code for one."""
    x = _rand(m, 4, m, dtype="bf16")
    x[1, 3] = float("nan")
    w = torch.ones(m, device="cuda")
    want = [torch.full((4, (m + 1) // 2), 0xEE, dtype=torch.uint8, device="cuda"), torch.full((4, -(-m // 32)), 0xEE, dtype=torch.uint8, device="cuda")]
    thl.rmsnorm(x, w, want[0], eps=EPS, sf=want[1])
    got = [torch.full_like(v, 0xEE) for v in want]
    w[m - 2] = float("nan")
    thl.rmsnorm(x, w, got[0], eps=EPS, sf=got[1])
    torch.cuda.synchronize()
    assert bool((got[1][1] == 255).all()) and bool((got[0][1] == 0).all())
    block = (m - 2) // 32
    assert bool((got[1][:, block] == 255).all()) and bool((got[0][:, 16 * block:16 * block + 16] == 0).all())
    for j in (0, 2, 3):
        assert torch.equal(got[1][j, :block], want[1][j, :block])
        assert torch.equal(got[0][j, :16 * block], want[0][j, :16 * block])
