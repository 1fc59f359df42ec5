"""thl.moe_layer against the plain fp64 form, on the GPU; most of it on inputs whose sums are exact, bit for bit."""
import pytest

torch = pytest.importorskip("torch")

import tile_hierarchy_linear_amd as thl
from oracle import operators as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def _give_back():
    """What lives on (a library's workspace, say) is not cut from these tests' large blocks."""
    yield
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _matrix(g, kind, experts, rows, k, exact, pad=0, scales=None):
    """(stored weights, block scales, fp64 values).  exact: small whole numbers under scales of 1/2 and 1 (the given
    ones otherwise)."""
    blocks = -(-k // 32)
    if kind in ("bf16", "f16"):
        v = torch.randint(-2, 3, (experts, rows, k), generator=g).float() if exact else torch.randn(experts, rows, k, generator=g) / k ** 0.5
        w = torch.zeros(experts, rows, k + pad, dtype=F[kind], device=DEV)[:, :, :k]
        w.copy_(v)
        return w, None, ref.f64(w)
    lo, hi = scales or ((126, 128) if exact else (122, 126))
    sf = torch.randint(lo, hi, (experts, rows, blocks), generator=g).to(torch.uint8)
    if kind == "e2m1":
        codes = torch.randint(0, 256, (experts, rows, (k + 1) // 2), generator=g).to(torch.uint8)
        if exact:  # 0, 1 and 2 of either sign
            codes = torch.tensor([0, 2, 4, 10, 12, 2, 10, 0], dtype=torch.uint8)[codes.long() & 7] | \
                (torch.tensor([0, 2, 4, 10, 12, 2, 10, 0], dtype=torch.uint8)[codes.long() >> 5] << 4)
        w = torch.zeros(experts, rows, (k + 1) // 2 + pad, dtype=torch.uint8, device=DEV)[:, :, :(k + 1) // 2]
        w.copy_(codes)
        v = ref.e2m1_values(codes.reshape(-1, (k + 1) // 2), k).reshape(experts, rows, k)
    else:
        v = torch.randint(-2, 3, (experts, rows, k), generator=g).float() if exact else torch.randn(experts, rows, k, generator=g)
        w = torch.zeros(experts, rows, k + pad, dtype=torch.uint8, device=DEV)[:, :, :k].view(F["e4m3"])
        w.view(torch.uint8).copy_(v.to(F["e4m3"]).view(torch.uint8))
        v = ref.f64(w)
    s = torch.pow(2.0, sf.double() - 127).repeat_interleave(32, dim=2)[:, :, :k]
    big = torch.full((experts, rows, blocks + 3), 0xFF, dtype=torch.uint8, device=DEV)[:, :, :blocks]
    big.copy_(sf)
    return w, big, v * s


def _sums_are_exact(x, ids, wt, v1, v2, gated, act, b1, b2):
    """Every sum of the layer is a whole number of steps that fit 24 bits, and u splits into two bf16 numbers."""
    x = ref.f64(x)
    hidden = v2.shape[2]
    y = torch.zeros(x.shape, dtype=torch.float64)
    for j in range(x.shape[0]):
        for t in range(ids.shape[1]):
            e = int(ids[j, t])
            if not 0 <= e < v1.shape[0]:
                continue
            u = v1[e] @ x[j] + (0 if b1 is None else ref.f64(b1[e]))
            a = v1[e].abs() @ x[j].abs() + 4
            assert float(a.max()) < 2 ** 22  # steps of 1/2 at the smallest
            u = (torch.relu(u[:hidden]) if act == "relu" else u[:hidden]) * (u[hidden:] if gated else 1.0)
            hi = u.float().bfloat16().double()
            lo = (u - hi).float().bfloat16().double()
            assert bool((hi + lo == u).all())
            y[j] += float(wt[j, t]) * (v2[e].abs() @ u.abs() + 4)
    # steps of 1, or of 1/8 with scales of 1/2, times weights of 1/4 or more: 23 bits
    assert float(y.max()) < (2 ** 21 if bool((v1 == v1.round()).all() and (v2 == v2.round()).all()) else 2 ** 18)


def _layer(n, m, hidden, experts, topk, w="bf16", x=None, gated=True, act="none", bias=False, exact=True, y="f32", seed=0,
           ids=None, pad=0, ids_type=torch.int32, scales=None):
    g = torch.Generator().manual_seed(seed)
    x = x or (w if w in ("bf16", "f16") else "bf16")
    xv = torch.randint(-1, 2, (n, m), generator=g).float() if exact else torch.randn(n, m, generator=g)
    xt = torch.zeros(n, m + pad, dtype=F[x], device=DEV)[:, :m]
    xt.copy_(xv)
    w1, sf1, v1 = _matrix(g, w, experts, 2 * hidden if gated else hidden, m, exact, 2 * pad, scales)
    w2, sf2, v2 = _matrix(g, w, experts, m, hidden, exact, 2 * pad, scales)
    b1 = b2 = None
    if bias:
        b1 = torch.randint(-3, 4, (experts, v1.shape[1]), generator=g).to(F[x]).to(DEV)
        b2 = torch.randint(-3, 4, (experts, m), generator=g).float().to(DEV)
    if ids is None:
        ids = torch.randint(-1, experts + 1, (n, topk), generator=g)  # some outside
    ids = ids.to(ids_type)
    wt = torch.pow(2.0, -torch.randint(0, 3, (n, topk), generator=g).float()) if exact else torch.rand(n, topk, generator=g)
    wt = torch.where((ids < 0) | (ids >= experts), float("nan"), wt)  # of no account
    yt = torch.full((n, m + pad), float("nan"), dtype=F[y], device=DEV)[:, :m]
    call = dict(gated=gated, act=act, sf1=sf1, sf2=sf2, b1=b1, b2=b2)
    thl.moe_layer(xt, ids.to(DEV), wt.to(DEV), w1, w2, yt, **call)
    torch.cuda.synchronize()
    want, bound = ref.moe_layer(xt, ids, torch.nan_to_num(wt), v1, v2, gated, act, b1, b2)
    if exact:
        _sums_are_exact(xt, ids, wt, v1, v2, gated, act, b1, b2)
        assert torch.equal(yt.cpu(), want.to(F[y]))
    else:
        d = (ref.f64(yt) - want).abs()
        assert bool((d <= bound + ref.half_step(want.abs() + bound, yt.dtype)).all()), float((d / bound.clamp(min=1e-300)).max())
    if pad:
        assert bool(torch.isnan(torch.as_strided(yt, (n, pad), (m + pad, 1), yt.storage_offset() + m)).all())
    return xt, ids.to(DEV), wt.to(DEV), w1, w2, yt, call


KINDS = ["bf16", "f16", "e4m3", "e2m1"]


@pytest.mark.parametrize("w", KINDS)
@pytest.mark.parametrize("n,m,hidden,experts,topk", [
    (1, 1, 1, 1, 1), (1, 7, 5, 3, 2), (1, 64, 32, 8, 2), (2, 33, 17, 4, 2), (3, 128, 64, 16, 3), (5, 130, 100, 2, 2),
    (1, 256, 256, 128, 8), (17, 96, 48, 4, 2), (40, 70, 34, 3, 2), (64, 64, 40, 2, 1), (9, 258, 300, 20, 4)])
@pytest.mark.parametrize("gated", [True, False])
def test_exact_sums(w, n, m, hidden, experts, topk, gated):
    _layer(n, m, hidden, experts, topk, w=w, gated=gated, act="none" if gated else "relu", bias=n % 2 == 1, seed=n + m)


@pytest.mark.parametrize("w", ["e4m3", "e2m1"])
@pytest.mark.parametrize("gated", [True, False])
def test_fp16_activations_on_mx_weights(w, gated):
    _layer(6, 300, 70, 4, 2, w=w, x="f16", gated=gated)
    _layer(3, 512, 200, 8, 2, w=w, x="f16", gated=gated, act="gelu", exact=False)


@pytest.mark.parametrize("w", KINDS)
@pytest.mark.parametrize("k", [31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 320, 511, 512, 513])
def test_ends_of_k(w, k):
    _layer(2, k, 16, 2, 1, w=w, gated=False, seed=k)
    _layer(2, 16, k, 2, 1, w=w, gated=False, seed=k)


@pytest.mark.parametrize("w", KINDS)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_activations(w, act):
    for gated in (True, False):
        _layer(4, 200, 96, 5, 2, w=w, act=act, gated=gated, exact=False, bias=gated)


@pytest.mark.parametrize("w", KINDS)
def test_larger(w):
    _layer(3, 1000, 600, 6, 2, w=w, act="silu", exact=False, y="bf16")
    _layer(20, 640, 512, 4, 2, w=w, act="silu", exact=False, y="f16")


@pytest.mark.parametrize("w", KINDS)
def test_pitched_rows(w):
    for pad in (1, 3, 8):
        _layer(5, 100, 60, 4, 2, w=w, pad=pad)


@pytest.mark.parametrize("y", ["f32", "f16", "bf16"])
def test_output_types(y):
    _layer(3, 90, 40, 4, 2, y=y)


@pytest.mark.parametrize("w", ["bf16", "e2m1"])
@pytest.mark.parametrize("many", [1, 15, 16, 17, 33, 64, 200])
def test_choices_of_one_expert(w, many):
    # all tokens on one expert of few, and of more experts than choices; every token the same expert twice
    _layer(many, 48, 40, 3, 1, w=w, ids=torch.full((many, 1), 1), seed=many)
    _layer(many, 48, 40, 2 * many + 5, 2, w=w, ids=torch.full((many, 2), 2 * many), seed=many)


def test_the_most_choices():
    _layer(1024, 40, 20, 7, 1)
    _layer(128, 40, 20, 300, 8)
    _layer(16, 40, 20, 1100, 64)  # a workgroup for each choice


def test_int64_ids_and_ids_outside():
    _layer(4, 64, 32, 8, 2, ids_type=torch.int64)
    ids = torch.tensor([[-1, 1 << 40], [-(1 << 40), 3], [8, -1]])
    got = _layer(3, 64, 32, 8, 2, ids=ids, ids_type=torch.int64)
    assert bool((got[5][0] == 0).all()) and bool((got[5][2] == 0).all())
    big = torch.zeros(4, 9, dtype=torch.int32, device=DEV)  # pitched ids
    xt, ids, wt, w1, w2, yt, call = _layer(4, 64, 32, 8, 2)
    big[:, 3:5] = ids
    y2 = torch.empty_like(yt)
    thl.moe_layer(xt, big[:, 3:5], wt, w1, w2, y2, **call)
    torch.cuda.synchronize()
    assert torch.equal(y2, yt)


@pytest.mark.parametrize("w", ["e2m1", "e4m3"])
@pytest.mark.parametrize("lo,hi", [(0, 3), (8, 12), (1, 130), (120, 135), (244, 249)])
def test_scales_beyond_normal_bf16(w, lo, hi):
    """One expert's first matrix under extreme scales; what the second makes of it is scaled back by its own."""
    g = torch.Generator().manual_seed(lo)
    n, m, hidden = 3, 200, 64
    w1, sf1, v1 = _matrix(g, w, 2, hidden, m, True, scales=(lo, hi))
    back = 254 - (lo + hi) // 2
    w2, sf2, v2 = _matrix(g, w, 2, m, hidden, True, scales=(min(back, 254), min(back, 254) + 1))
    x = torch.randint(-2, 3, (n, m), generator=g).float().to(F["bf16"]).to(DEV)
    ids, wt = torch.tensor([[0], [1], [0]], dtype=torch.int32), torch.ones(n, 1)
    y = torch.empty(n, m, device=DEV)
    thl.moe_layer(x, ids.to(DEV), wt.to(DEV), w1, w2, y, gated=False, act="none", sf1=sf1, sf2=sf2)
    torch.cuda.synchronize()
    want, bound = ref.moe_layer(x, ids, wt, v1, v2, False, "none")
    # (fp32 drops what lies below its subnormals, 2^-149, of u's planes 2^-133, times the second matrix's values)
    floor = 2.0 ** -132 * v2[ids[:, 0].long()].abs().sum(dim=2)
    assert bool(((ref.f64(y) - want).abs() <= bound + floor + ref.half_step(want, torch.float32)).all())


@pytest.mark.parametrize("w", ["e2m1", "e4m3"])
@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("lo,hi", [(60, 66), (98, 112), (104, 127), (120, 140), (190, 196)])
def test_every_code_under_every_scale(w, x, lo, hi):
    """One value in each token, and a second matrix that passes u on: the elements themselves, bit for bit."""
    g = torch.Generator().manual_seed(hi)
    for m, hidden in ((256, 64), (150, 96)):
        sf = torch.randint(lo, hi, (1, hidden, -(-m // 32)), generator=g).to(torch.uint8)
        if w == "e2m1":
            codes = torch.randint(0, 256, (hidden, m // 2), generator=g).to(torch.uint8)
            v1, w1 = ref.e2m1_values(codes, m), codes[None]
            w2 = torch.zeros(1, m, hidden, dtype=torch.uint8)
            w2[0, torch.arange(hidden), torch.arange(hidden)] = 2  # 1
            w2 = w2[:, :, 0::2] | (w2[:, :, 1::2] << 4)
        else:
            codes = torch.randint(0, 256, (hidden, m), generator=g).to(torch.uint8)
            codes[(codes & 0x7F) == 0x7F] = 1  # no NaN; the smallest
            w1 = codes[None].view(F["e4m3"])
            v1 = ref.f64(w1)[0]
            w2 = torch.zeros(1, m, hidden)
            w2[0, torch.arange(hidden), torch.arange(hidden)] = 1.0
            w2 = w2.to(F["e4m3"])
        v1 = v1 * torch.pow(2.0, sf[0].double() - 127).repeat_interleave(32, dim=1)[:, :m]
        xt = torch.diag(torch.tensor([1.0, -2.0, 0.5]).repeat(m)[:m]).to(F[x])
        y = torch.full((m, m), float("nan"), device=DEV)
        thl.moe_layer(xt.to(DEV), torch.zeros(m, 1, dtype=torch.int32, device=DEV), torch.ones(m, 1, device=DEV),
                      w1.to(DEV), w2.to(DEV), y, gated=False, act="none", sf1=sf.to(DEV),
                      sf2=torch.full((1, m, -(-hidden // 32)), 127, dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()
        want = torch.zeros(m, m, dtype=torch.float64)
        want[:, :hidden] = xt.double() @ v1.T
        assert torch.equal(y.cpu().double(), want)


@pytest.mark.parametrize("w", ["e2m1", "e4m3"])
@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("rare", [3, 250])
@pytest.mark.parametrize("m", [100, 256, 300])
def test_infinities_next_to_extreme_scales(w, x, rare, m):
    # every weight 1 or 2^(rare - 127), one activation infinite, the others 0: every sum is that infinity
    hidden = 32
    one = {"e2m1": 0x22, "e4m3": 0x38}[w]
    w1, w2 = (torch.full((1, r, k // 2 if w == "e2m1" else k), one, dtype=torch.uint8, device=DEV)
              for r, k in ((hidden, m), (m, hidden)))
    if w == "e4m3":
        w1, w2 = w1.view(F["e4m3"]), w2.view(F["e4m3"])
    xt = torch.zeros(3, m, dtype=F[x], device=DEV)
    xt[0, 5], xt[1, m - 1] = float("inf"), float("-inf")
    for block in range(-(-m // 32)):
        sf1 = torch.full((1, hidden, -(-m // 32)), 127, dtype=torch.uint8, device=DEV)
        sf1[:, :, block] = rare
        y = torch.empty(3, m, device=DEV)
        thl.moe_layer(xt, torch.zeros(3, 1, dtype=torch.int32, device=DEV), torch.ones(3, 1, device=DEV), w1, w2, y,
                      gated=False, act="none", sf1=sf1,
                      sf2=torch.full((1, m, 1), 127, dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()
        assert bool((y[0] == float("inf")).all()) and bool((y[1] == float("-inf")).all()) and bool((y[2] == 0).all())


@pytest.mark.parametrize("w", ["e2m1", "e4m3"])
def test_a_nan_scale(w):
    xt, ids, wt, w1, w2, yt, call = _layer(3, 300, 64, 2, 1, w=w, ids=torch.tensor([[0], [1], [0]]))
    sf1 = call["sf1"].clone()
    sf1[1, 5, 2] = 255
    y = torch.empty_like(yt)
    thl.moe_layer(xt, ids, wt, w1, w2, y, **{**call, "sf1": sf1})
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[1]).all()) and torch.equal(y[[0, 2]], yt[[0, 2]])


def test_infinities_stay_with_their_token():
    for w in KINDS:
        xt, ids, wt, w1, w2, yt, call = _layer(5, 160, 64, 2, 1, w=w, ids=torch.ones(5, 1))
        x = xt.clone()
        x[2, 7], x[3, 159] = float("inf"), float("nan")
        y = torch.empty_like(yt)
        thl.moe_layer(x, ids, wt, w1, w2, y, **call)
        torch.cuda.synchronize()
        assert not bool(torch.isfinite(y[2:4]).any()) and torch.equal(y[[0, 1, 4]], yt[[0, 1, 4]])


def test_large_u_of_fp16_activations():
    # u = 2^18, past fp16's range, comes back exactly
    n, m, hidden = 2, 64, 32
    x = torch.full((n, m), 64.0, dtype=torch.float16, device=DEV)
    w1 = torch.full((1, hidden, m), 64.0, dtype=torch.float16, device=DEV)
    w2 = torch.full((1, m, hidden), 2.0 ** -14, dtype=torch.float16, device=DEV)
    y = torch.empty(n, m, dtype=torch.float16, device=DEV)
    thl.moe_layer(x, torch.zeros(n, 1, dtype=torch.int32, device=DEV), torch.ones(n, 1, device=DEV), w1, w2, y,
                  gated=False, act="none")
    torch.cuda.synchronize()
    assert bool((y == 512.0).all())


def test_empty():
    xt, ids, wt, w1, w2, yt, call = _layer(3, 64, 32, 4, 2)
    thl.moe_layer(xt[:0], ids[:0], wt[:0], w1, w2, yt[:0], **call)
    with pytest.raises(thl.ThlError):
        thl.moe_layer(xt, ids[:, :0].contiguous(), wt[:, :0].contiguous(), w1, w2, yt, **call)


def test_offsets_past_32_bits():
    # expert 2's matrices start past 2^32 elements
    g = torch.Generator().manual_seed(0)
    n, m, hidden, far = 2, 96, 48, (1 << 31) + 64
    v1, v2 = (torch.randint(-2, 3, s, generator=g).float() for s in ((3, hidden, m), (3, m, hidden)))
    big = torch.zeros(2 * far + 2 * m * hidden, dtype=torch.bfloat16, device=DEV)
    w1 = torch.as_strided(big, (3, hidden, m), (far, m, 1))
    w2 = torch.as_strided(big, (3, m, hidden), (far, hidden, 1), m * hidden)
    w1.copy_(v1)
    w2.copy_(v2)
    x = torch.randint(-2, 3, (n, m), generator=g).to(torch.bfloat16).to(DEV)
    ids, wt = torch.tensor([[2, 1], [0, 2]], dtype=torch.int32), torch.ones(n, 2)
    y = torch.empty(n, m, device=DEV)
    thl.moe_layer(x, ids.to(DEV), wt.to(DEV), w1, w2, y, gated=False, act="relu")
    torch.cuda.synchronize()
    assert torch.equal(ref.f64(y), ref.moe_layer(x, ids, wt, v1.double(), v2.double(), False, "relu")[0])


def test_results_do_not_depend_on_timing():
    xt, ids, wt, w1, w2, yt, call = _layer(30, 700, 333, 6, 3, act="silu", exact=False)
    for _ in range(3):
        y = torch.empty_like(yt)
        thl.moe_layer(xt, ids, wt, w1, w2, y, **call)
        torch.cuda.synchronize()
        assert torch.equal(y, yt)


@pytest.mark.parametrize("bad", ["ids", "w1", "w2", "weights", "act", "scales", "type", "device", "rows", "many"])
def test_torch_form_refusals(bad):
    xt, ids, wt, w1, w2, yt, call = _layer(3, 64, 32, 4, 2)
    with pytest.raises((ValueError, thl.ThlError)):
        if bad == "ids":
            thl.moe_layer(xt, ids.float(), wt, w1, w2, yt, **call)
        elif bad == "w1":
            thl.moe_layer(xt, ids, wt, w1[:, :63], w2, yt, **call)
        elif bad == "w2":
            thl.moe_layer(xt, ids, wt, w1, w2[:3], yt, **call)
        elif bad == "weights":
            thl.moe_layer(xt, ids, wt.half(), w1, w2, yt, **call)
        elif bad == "act":
            thl.moe_layer(xt, ids, wt, w1, w2, yt, **{**call, "act": "tanh"})
        elif bad == "scales":
            thl.moe_layer(xt, ids, wt, w1, w2, yt, **{**call, "sf1": torch.zeros(4, 64, 2, dtype=torch.uint8, device=DEV)})
        elif bad == "type":
            thl.moe_layer(xt.half(), ids, wt, w1, w2, yt, **call)
        elif bad == "device":
            thl.moe_layer(xt, ids, wt, w1.cpu(), w2, yt, **call)
        elif bad == "rows":
            thl.moe_layer(xt, ids, wt, w1.transpose(1, 2), w2, yt, **call)
        else:
            thl.moe_layer(xt[:1].expand(1025, 64), ids[:1, :1].expand(1025, 1), torch.ones(1025, 1, device=DEV), w1, w2,
                          torch.empty(1025, 64, device=DEV), **call)


def _unit(w, k):
    """The matrix that passes k values on, as stored, with its scales."""
    one = torch.eye(k)
    if w == "e2m1":
        codes = (2 * one).to(torch.uint8)  # code 2 is 1
        return (codes[:, 0::2] | (codes[:, 1::2] << 4))[None].to(DEV), torch.full((1, k, -(-k // 32)), 127, dtype=torch.uint8, device=DEV)
    if w == "e4m3":
        return one.to(F["e4m3"])[None].to(DEV), torch.full((1, k, -(-k // 32)), 127, dtype=torch.uint8, device=DEV)
    return one.to(F[w])[None].to(DEV), None


@pytest.mark.parametrize("w", KINDS)
@pytest.mark.parametrize("k", [34, 64, 300, 520])
@pytest.mark.parametrize("n", [1, 3, 4, 5, 9, 17, 40])
def test_u_has_the_bits_of_fp32(w, k, n):
    """u = gate * up of two numbers of 17 bits, rounded to fp32 once, passed on by the second matrix: bit for bit."""
    g = torch.Generator().manual_seed(k + n)
    x = torch.zeros(n, k)
    x[:, :4] = torch.tensor([1.0, 2.0 ** -4, 2.0 ** -8, 2.0 ** -12]) * (1.0 - 2.0 * torch.randint(0, 2, (n, 4), generator=g))
    w2, sf2 = _unit(w, k)
    if w == "e2m1":
        w1 = torch.randint(0, 256, (1, 2 * k, k // 2), generator=g).to(torch.uint8)
        v1 = ref.e2m1_values(w1[0], k)
    else:
        v1 = torch.randint(-15, 16, (2 * k, k), generator=g).double() / 8
        w1 = v1.float()[None].to(F[w])
    sf1 = None if sf2 is None else torch.full((1, 2 * k, sf2.shape[2]), 127, dtype=torch.uint8, device=DEV)
    y = torch.full((n, k), float("nan"), device=DEV)
    thl.moe_layer(x.to(F["f16" if w == "f16" else "bf16"]).to(DEV), torch.zeros(n, 1, dtype=torch.int32, device=DEV),
                  torch.ones(n, 1, device=DEV), w1.to(DEV), w2, y, act="none", sf1=sf1, sf2=sf2)
    torch.cuda.synchronize()
    pre = x.double() @ v1.t()
    assert bool((pre.float().double() == pre).all())  # multiples of 2^-15 below 8
    want = pre[:, :k].float() * pre[:, k:].float()
    assert torch.equal(y.cpu(), want), float(((y.cpu() - want).abs() / want.abs().clamp(min=1e-30)).max())


def test_u_of_the_whole_range_of_fp32():
    # between bf16's largest number and fp32's
    n, k = 3, 64
    x = torch.zeros(n, k, dtype=torch.bfloat16, device=DEV)
    x[:, 0], x[:, 1] = 2.0 ** 64, 2.0 ** 50
    x[1] = -x[1]
    w1 = torch.zeros(1, k, k, dtype=torch.bfloat16, device=DEV)
    w1[:, :, 0] = torch.finfo(torch.bfloat16).max / 2.0 ** 64
    w1[:, :, 1] = 1.5 * 2.0 ** (119 - 50)  # three quarters of a step of bf16
    w2, _ = _unit("bf16", k)
    y = torch.empty(n, k, device=DEV)
    thl.moe_layer(x, torch.zeros(n, 1, dtype=torch.int32, device=DEV), torch.ones(n, 1, device=DEV), w1, w2, y, gated=False,
                  act="none")
    torch.cuda.synchronize()
    want = (ref.f64(x) @ ref.f64(w1[0]).t()).float()
    assert bool(torch.isfinite(want).all()) and float(want.max()) > torch.finfo(torch.bfloat16).max * (1 + 2.0 ** -9)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("w", KINDS)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("gated", [False, True])
def test_nan_goes_through_every_activation(w, act, gated):
    xt, ids, wt, w1, w2, yt, call = _layer(5, 160, 64, 2, 1, w=w, ids=torch.ones(5, 1), act=act, gated=gated, exact=False)
    x, y = xt.clone(), torch.empty_like(yt)
    x[3, 159] = float("nan")
    thl.moe_layer(x, ids, wt, w1, w2, y, **call)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[3]).all()) and torch.equal(y[[0, 1, 2, 4]], yt[[0, 1, 2, 4]])
    # one row of the first matrix: every token of the expert
    bad, call = w1.clone(), dict(call)
    if w in ("e4m3", "e2m1"):
        call["sf1"] = call["sf1"].clone()
        call["sf1"][1, 5, 2] = 255
    else:
        bad[1, 5, 70] = float("nan")
    thl.moe_layer(xt, ids, wt, bad, w2, y, **call)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y).all())
    ids = torch.tensor([[1], [0], [1], [0], [-1]], dtype=torch.int32, device=DEV)
    thl.moe_layer(xt, ids, wt, w1, w2, yt, **call)  # (call: the scales with the NaN, the weights without)
    thl.moe_layer(xt, ids, wt, bad, w2, y, **call)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[[0, 2]]).all()) and bool(torch.isfinite(y[[1, 3, 4]]).all())
    assert torch.equal(y[[1, 3, 4]], yt[[1, 3, 4]])


@pytest.mark.parametrize("w", ["bf16", "f16"])
@pytest.mark.parametrize("n,experts", [(1, 3), (4, 1), (9, 2), (40, 2)])
def test_an_infinite_weight_of_the_second_matrix(w, n, experts):
    xt, ids, wt, w1, w2, yt, call = _layer(n, 70, 40, experts, 1, w=w, gated=False, ids=torch.zeros(n, 1))
    u = ref.f64(xt) @ ref.f64(w1[0]).t()
    c = int(u.abs().amin(dim=0).argmax())
    bad, y = w2.clone(), torch.empty_like(yt)
    bad[0, 3, c], bad[0, 69, c] = float("inf"), -float("inf")
    thl.moe_layer(xt, ids, wt, w1, bad, y, **call)
    torch.cuda.synchronize()
    assert bool(u[:, c].ne(0).any())
    for row, sign in ((3, 1), (69, -1)):
        want = torch.where(u[:, c] == 0, torch.nan, sign * torch.copysign(torch.full((), torch.inf).double(), u[:, c]))
        assert torch.equal(y[:, row].cpu().double().nan_to_num(nan=7.0, posinf=1.0, neginf=-1.0),
                           want.nan_to_num(nan=7.0, posinf=1.0, neginf=-1.0))
    rest = [i for i in range(70) if i not in (3, 69)]
    assert torch.equal(y[:, rest], yt[:, rest])


@pytest.mark.parametrize("w", ["bf16", "e2m1"])
@pytest.mark.parametrize("n,experts,topk", [(1, 12, 4), (3, 40, 2), (40, 6, 3)])
def test_what_the_workspace_held_does_not_matter(w, n, experts, topk):
    """Through the C entry point, which takes the workspace, with choices that do not count."""
    xt, ids, wt, w1, w2, yt, call = _layer(n, 96, 40, experts, topk, w=w)
    need = thl.thl_moe_layer_workspace(96, 40, n, topk)
    up, down = (thl.thl_expert_matrix(v.data_ptr(), code * v.stride(1), code * v.stride(0), s.data_ptr() if s is not None else None,
                                      s.stride(1) if s is not None else 0, s.stride(0) if s is not None else 0, None, 0,
                                      thl.DTYPES[w], thl.DTYPES["none"])
                for code in [2 if w == "e2m1" else 1] for v, s in ((w1, call["sf1"]), (w2, call["sf2"])))
    for byte in (0x00, 0x7F, 0xFF):  # zeros, large numbers, NaN
        ws = torch.full((need,), byte, dtype=torch.uint8, device=DEV)
        y = torch.empty_like(yt)
        stream = torch.cuda.current_stream().cuda_stream
        assert thl.thl_moe_layer(96, 40, n, topk, experts, xt.data_ptr(), xt.stride(0), ids.data_ptr(), ids.stride(0), 4,
                                 wt.data_ptr(), up, down, thl.THL_MOE_GATED, y.data_ptr(), 96, "bf16", "f32", ws.data_ptr(),
                                 need, stream) == thl.THL_OK
        torch.cuda.synchronize()
        assert torch.equal(y, yt), byte


@pytest.mark.parametrize("w", ["e2m1", "e4m3"])
@pytest.mark.parametrize("k", [32, 150, 256, 520])
@pytest.mark.parametrize("n", [3, 6, 20, 50])
def test_large_scales_of_the_second_matrix(w, k, n):
    """u times powers of two up to 2^127, also past the fast range: bit for bit, of few choices and of many."""
    g = torch.Generator().manual_seed(k + n)
    x = torch.zeros(n, k, dtype=torch.float64)
    x[:, :4] = torch.tensor([2.0 ** -8, 2.0 ** -12, 2.0 ** -16, 2.0 ** -20], dtype=torch.float64)
    x *= 1.0 - 2.0 * torch.randint(0, 2, (n, k), generator=g)
    v1 = torch.randint(-6, 7, (k, k), generator=g).double() / 2
    if w == "e2m1":
        v1 = torch.where(v1.abs() == 2.5, 2.0, v1)  # (no code for 2.5; 0.5 to 3 by halves otherwise)
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
        codes = (v1.abs()[:, :, None] == grid).to(torch.uint8).argmax(dim=2).to(torch.uint8) + 8 * (v1 < 0).to(torch.uint8)
        w1 = (codes[:, 0::2] | (codes[:, 1::2] << 4))[None]
    else:
        w1 = v1.float()[None].to(F["e4m3"])
    w2, sf2 = _unit(w, k)
    sf2 = torch.randint(120, 255, sf2.shape, generator=g).to(torch.uint8)
    y = torch.full((n, k), float("nan"), device=DEV)
    thl.moe_layer(x.to(torch.bfloat16).to(DEV), torch.zeros(n, 1, dtype=torch.int32, device=DEV),
                  torch.ones(n, 1, device=DEV), w1.to(DEV), w2, y, gated=False, act="none",
                  sf1=torch.full((1, k, sf2.shape[2]), 127, dtype=torch.uint8, device=DEV), sf2=sf2.to(DEV))
    torch.cuda.synchronize()
    u = x @ v1.t()
    own = sf2[0, torch.arange(k), torch.arange(k) // 32].double()
    assert torch.equal(y.cpu().double(), u * torch.pow(2.0, own - 127))
