"""thl.layernorm and its gradient against the plain fp64 forms, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import tile_hierarchy_linear_amd as thl
from oracle import operators as ref

pytestmark = pytest.mark.gpu
F = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
     "e5m2": torch.float8_e5m2}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _give_back():
    """What lives on (a library's workspace, say) is not cut from these tests' large blocks."""
    yield
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _rand(seed, *shape, dtype="f32", scale=1.0, shift=0.0, pitch=0, offset=0):
    """A (n, m) tensor on the GPU, rows `pitch` elements past m apart, starting `offset` elements in."""
    g = torch.Generator().manual_seed(seed)
    v = (torch.randn(*shape, generator=g) * scale + shift).to(F[dtype])
    if v.dim() == 2 and (pitch or offset):
        n, m = shape
        big = torch.zeros(offset + n * (m + pitch), dtype=F[dtype], device="cuda")
        view = big[offset:].view(n, m + pitch)[:, :m]
        view.copy_(v)
        return view
    return v.cuda()


def _check(got, want, bound, what):
    d = (ref.f64(got) - want).abs()
    over = ~(d <= bound)
    assert not bool(over.any()), (what, int(over.sum()), float((d / bound.clamp(min=1e-300)).max()))


def _check_float(got, want, err, what):
    _check(got, want, err + ref.half_step(want.abs() + err, got.dtype), what)


def _run(n, m, x="bf16", res=None, w=True, b=True, vec=None, y="bf16", mx=False, scale=1.0, pitch=0, offset=0, seed=0,
         shift=0.5, xt=None, keep_sum=True):
    xt = _rand(seed, n, m, dtype=x, shift=shift, pitch=pitch, offset=offset) if xt is None else xt
    rt = _rand(seed + 1, n, m, dtype=res, scale=3.0, pitch=pitch, offset=offset) if res else None
    wt = (1 + 0.3 * _rand(seed + 2, m)).to(F[vec or x]) if w else None
    bt = _rand(seed + 3, m, dtype=vec or x, scale=0.3) if b else None
    st = torch.full_like(rt, float("nan")) if res and keep_sum else None
    if y == "e2m1":
        yt = torch.full((n, (m + 1) // 2 + pitch), 0xEE, dtype=torch.uint8, device="cuda")[:, :(m + 1) // 2]
    elif y in ref.TOP:
        yt = torch.full((n, m + pitch), 0xEE, dtype=torch.uint8, device="cuda")[:, :m].view(F[y])
    else:
        yt = torch.full((n, m + pitch), float("nan"), dtype=F[y], device="cuda")[:, :m]
    nb = (m + 31) // 32
    sf = torch.full((n, nb + 3), 0xEE, dtype=torch.uint8, device="cuda") if mx else None
    thl.layernorm(xt, wt, bt, yt, eps=EPS, residual=rt, residual_out=st, scale=scale, sf=sf)
    torch.cuda.synchronize()
    s, want, err = ref.layernorm(xt, rt, wt, bt, EPS)
    if st is not None:
        _check(st, s, ref.half_step(s, st.dtype) + ref.U * s.abs(), "sum")
    if mx:
        code = sf.cpu()[:, :nb].to(torch.int64)
        assert bool((sf[:, nb:] == 0xEE).all())  # scale padding untouched
        pad, perr = (torch.nn.functional.pad(v, (0, 32 * nb - m)).reshape(n, nb, 32) for v in (want, err))
        # the code is that of some value within the fp32 error of the maximum
        lo = (pad.abs() - perr).amax(dim=2).clamp(min=1e-300)
        hi = (pad.abs() + perr).amax(dim=2).clamp(min=1e-300)
        lo, hi = ((torch.floor(torch.log2(v)) - ref.EMAX[y]).clamp(-127, 127) + 127 for v in (lo, hi))
        assert bool(((code >= lo) & (code <= hi)).all())
        each = torch.pow(2.0, code.double() - 127).repeat_interleave(32, dim=1)[:, :m]
        values = ref.e2m1_values(yt, m) if y == "e2m1" else ref.f64(yt)
        c = (want / each).clamp(-ref.TOP[y], ref.TOP[y])
        _check(values, c, ref.narrow_half_step(c, y) + 2 * err / each, y)
    elif y in ref.TOP:
        c = (want / scale).clamp(-ref.TOP[y], ref.TOP[y])
        _check(ref.f64(yt), c, ref.narrow_half_step(c, y) + 2 * (err + 2 * ref.U * want.abs()) / scale, y)
    else:
        _check_float(yt, want, err, "y")
    return xt, rt, st, yt, wt, bt


# 512 and 16,384: the last features of a variant; 16,385 on: the token read several times
@pytest.mark.parametrize("m", [1, 7, 9, 31, 100, 512, 513, 1024, 1500, 2048, 2049, 4099, 6144, 8192, 8200, 16384, 16385,
                               20011])
@pytest.mark.parametrize("n", [1, 3])
def test_widths(n, m):
    _run(n, m, res="bf16", seed=m)


@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("res", [None, "same", "f32"])
@pytest.mark.parametrize("y", ["bf16", "f16", "f32"])
def test_types(x, res, y):
    _run(5, 777, x=x, res=x if res == "same" else res, y=y, vec="f32" if y == "f16" else None)
    _run(2, 16999, x=x, res=x if res == "same" else res, y=y)


@pytest.mark.parametrize("w,b", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("m", [5, 640, 4099, 16500])
def test_without_weight_or_bias(w, b, m):
    _run(3, m, w=w, b=b, res="f32")


@pytest.mark.parametrize("y", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("m", [1, 33, 64, 1000, 4096, 16390])
def test_narrow_outputs(y, m):
    _run(3, m, y=y, mx=True, res="bf16", seed=m)
    if y != "e2m1":
        _run(4, m, y=y, scale=0.0123, res="f32", pitch=5)


@pytest.mark.parametrize("m", [65, 4099, 16411])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_pitched_rows_at_element_offsets(m, offset):
    for x in ("f16", "f32"):
        _run(6, m, x=x, res=x, y="f32", pitch=3, offset=offset)


@pytest.mark.parametrize("m", [300, 2050, 8192, 16400])
@pytest.mark.parametrize("shift", [100.0, -3e4])
def test_a_mean_far_from_zero(m, shift):
    # the variance is 1 beside squares of up to 1e9: a difference of sums would lose it
    _run(3, m, x="f32", y="f32", shift=shift)


def test_equal_features():
    for m in (1, 40, 5000, 17000):
        x = torch.full((2, m), 3.0, device="cuda")
        w, b, y = torch.full((m,), 2.0, device="cuda"), torch.full((m,), 0.25, device="cuda"), torch.empty(2, m, device="cuda")
        thl.layernorm(x, w, b, y, eps=EPS)
        torch.cuda.synchronize()
        assert bool((y == 0.25).all())  # sums of threes are exact
        thl.layernorm(x, w, b, y, eps=0.0)
        torch.cuda.synchronize()
        assert bool(torch.isnan(y).all())  # 0 / 0


def test_many_tokens_walk_the_grid():
    _run(40000, 72, res="bf16")
    _run(9000, 2100, y="e4m3", mx=True)
    _run(1100, 8192, x="f32", y="f32")
    _run(2100, 8195)


def test_in_place():
    for m in (600, 1025, 4096, 4099, 16500):
        x, r, s, y, w, b = _run(5, m, res="bf16")
        x2, r2 = x.clone(), r.clone()
        thl.layernorm(x2, w, b, x2, eps=EPS, residual=r2, residual_out=r2)
        torch.cuda.synchronize()
        assert torch.equal(x2, y) and torch.equal(r2, s)
        x2, y2 = x.clone(), torch.empty_like(y)
        thl.layernorm(x2, w, b, y2, eps=EPS, residual=r, residual_out=x2)  # the sum over x
        torch.cuda.synchronize()
        assert torch.equal(x2, s) and torch.equal(y, y2)


def test_infinities_nan_and_empty():
    x = _rand(0, 4, 300, dtype="bf16")
    x[1, 7] = float("inf")
    x[2, 299] = float("nan")
    w, b, y = torch.ones(300, device="cuda"), torch.zeros(300, device="cuda"), torch.empty(4, 300, device="cuda")
    thl.layernorm(x, w, b, y, eps=EPS)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[1:3]).all())
    for k in (0, 3):
        _, want, err = ref.layernorm(x[k:k + 1], None, w, b, EPS)
        _check_float(y[k:k + 1], want, err, "the other tokens")
    e = torch.empty(0, 300, device="cuda")
    thl.layernorm(e, w, b, e.clone())
    dw, db = (torch.full((300,), 5.0, device="cuda") for _ in range(2))
    thl.layernorm_backward(e, e, w, torch.empty_like(e), dw, db)
    torch.cuda.synchronize()
    assert bool((dw == 0).all()) and bool((db == 0).all())
    thl.layernorm(torch.empty(3, 0, device="cuda"), None, None, torch.empty(3, 0, device="cuda"))


def test_offsets_past_32_bits():
    n, m, pitch = 4200, 64, 1 << 20
    big = torch.zeros(n * pitch, dtype=torch.bfloat16, device="cuda")
    x = big.view(n, pitch)[:, :m]
    x.copy_(_rand(0, n, m, dtype="bf16"))
    y = torch.empty(n, m, device="cuda")
    thl.layernorm(x, None, None, y, eps=EPS)
    torch.cuda.synchronize()
    _, want, err = ref.layernorm(x, None, None, None, EPS)
    _check_float(y, want, err, "y")


# ------------------------------------------------------------------ gradient

def _grad(n, m, s="bf16", g="bf16", w=True, vec=None, dres=True, dw="f32", db=True, pitch=0, seed=0, shift=0.5):
    st = _rand(seed, n, m, dtype=s, scale=2.0, shift=shift, pitch=pitch)
    dy = _rand(seed + 1, n, m, dtype=g, shift=0.1, pitch=pitch)
    dr = _rand(seed + 2, n, m, dtype=g, pitch=pitch) if dres else None
    wt = (1 + 0.3 * _rand(seed + 3, m)).to(F[vec or s]) if w else None
    dx = torch.full((n, m + pitch), float("nan"), dtype=F[g], device="cuda")[:, :m]
    dwt = torch.full((m,), float("nan"), dtype=F[dw], device="cuda") if dw else None
    dbt = torch.full((m,), float("nan"), dtype=F[dw or "f32"], device="cuda") if db else None
    thl.layernorm_backward(st, dy, wt, dx, dwt, dbt, eps=EPS, dres=dr)
    torch.cuda.synchronize()
    want_x, want_w, want_b, bx, bw, bb = ref.layernorm_backward(st, dy, wt, dr, EPS)
    _check_float(dx, want_x, bx, "dx")
    if dw:
        _check_float(dwt, want_w, bw, "dw")
    if db:
        _check_float(dbt, want_b, bb, "db")
    return st, dy, dr, wt, dx, dwt, dbt


@pytest.mark.parametrize("m", [1, 7, 9, 500, 513, 1001, 2048, 2050, 4096, 5003, 8193, 16384, 16390])
@pytest.mark.parametrize("n", [1, 40])
def test_backward_widths(n, m):
    _grad(n, m, seed=m)


@pytest.mark.parametrize("s", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("g", ["bf16", "f16", "f32"])
def test_backward_types(s, g):
    _grad(37, 1203, s=s, g=g, dres=False, pitch=1)
    _grad(3, 17001, s=s, g=g, vec="f32")
    _grad(3, 12000, s=s, g=g, dw=s)


@pytest.mark.parametrize("w,dw,db", [(False, "f32", True), (True, None, True), (True, "f32", False), (False, None, False)])
@pytest.mark.parametrize("m", [300, 5000, 16400])
def test_backward_without_some(w, dw, db, m):
    _grad(700, m, w=w, dw=dw, db=db)


@pytest.mark.parametrize("n,m", [(4099, 227), (5000, 600), (4200, 1500), (600, 5003), (520, 8192), (300, 9001), (270, 16384),
                                 (1500, 16392), (3000, 136)])
@pytest.mark.parametrize("g", ["bf16", "f32"])
def test_backward_more_tokens_than_workgroups(n, m, g):
    _grad(n, m, s="f32" if g == "f32" else "bf16", g=g, seed=n, dres=g == "f32")


@pytest.mark.parametrize("s", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("g", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m", [8200, 12291])
def test_backward_of_long_tokens(s, g, m):
    # two runs a lane on sixteen wavefronts, several tokens a workgroup
    _grad(520, m, s=s, g=g, seed=m, dres=True)


def test_backward_with_a_mean_far_from_zero():
    for m in (300, 8192, 16400):
        _grad(30, m, s="f32", g="f32", shift=300.0)


@pytest.mark.parametrize("n,m", [(600, 700), (600, 1001), (300, 9001), (2, 6000), (600, 16600)])
def test_backward_in_place(n, m):
    st, dy, dr, w, dx, dw, db = _grad(n, m, seed=5)
    for out in (dy, dr, st):
        keep, dw2, db2 = out.clone(), torch.empty_like(dw), torch.empty_like(db)
        thl.layernorm_backward(st, dy, w, out, dw2, db2, eps=EPS, dres=dr)
        torch.cuda.synchronize()
        assert torch.equal(out, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
        out.copy_(keep)


def test_backward_against_differences():
    """The directional derivative of the fp64 norm by central differences: with step h off by h^2 / 6 times a third
    derivative of order one, 1e-8 relative at h = 1e-4, far below the kernel's own fp32 error, 1e-5 of the sum of
    magnitudes."""
    n, m, h = 6, 90, 1e-4
    x, dy, w, b = _rand(0, n, m, shift=1.0), _rand(1, n, m), 1 + 0.3 * _rand(2, m), _rand(5, m)
    dx, dw, db = torch.empty_like(x), torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    thl.layernorm_backward(x, dy, w, dx, dw, db, eps=EPS)
    torch.cuda.synchronize()
    g = torch.Generator().manual_seed(3)
    dirs = torch.randn(n, m, generator=g, dtype=torch.float64)
    wdir, bdir = (torch.randn(m, generator=g, dtype=torch.float64) for _ in range(2))
    X, DY, W, B = ref.f64(x), ref.f64(dy), ref.f64(w), ref.f64(b)

    def loss(a, v, c):
        return float((ref.layernorm(a, None, v, c, EPS)[1] * DY).sum())

    for got, up, down in ((dx, (X + h * dirs, W, B), (X - h * dirs, W, B)), (dw, (X, W + h * wdir, B), (X, W - h * wdir, B)),
                          (db, (X, W, B + h * bdir), (X, W, B - h * bdir))):
        num = (loss(*up) - loss(*down)) / (2 * h)
        along = ref.f64(got) * (dirs if got is dx else wdir if got is dw else bdir)
        assert abs(num - float(along.sum())) <= 1e-5 * float(along.abs().sum())


def test_results_do_not_depend_on_timing():
    a = _grad(2000, 1024, seed=9)
    for _ in range(3):
        dw, db = torch.empty_like(a[5]), torch.empty_like(a[6])
        thl.layernorm_backward(a[0], a[1], a[3], torch.empty_like(a[4]), dw, db, eps=EPS, dres=a[2])
        torch.cuda.synchronize()
        assert torch.equal(dw, a[5]) and torch.equal(db, a[6])


@pytest.mark.parametrize("bad", ["shape", "stride", "type", "device", "sum", "grads", "bias", "sums"])
def test_torch_form_refusals(bad):
    x, w, y = _rand(0, 4, 64), _rand(1, 64), torch.empty(4, 64, device="cuda")
    with pytest.raises((ValueError, thl.ThlError)):
        if bad == "shape":
            thl.layernorm(x, w, w, y[:3])
        elif bad == "stride":
            thl.layernorm(x, w, w, torch.empty(64, 4, device="cuda").t())
        elif bad == "type":
            thl.layernorm(x.double(), w, w, y)
        elif bad == "device":
            thl.layernorm(x, w.cpu(), w, y)
        elif bad == "sum":
            thl.layernorm(x, w, w, y, residual_out=y)
        elif bad == "bias":
            thl.layernorm(x, w, w.half(), y)
        elif bad == "sums":
            thl.layernorm_backward(x, x, w, y, torch.empty(64, device="cuda"), torch.empty(64, device="cuda").half())
        else:
            thl.layernorm_backward(x, x, w, torch.empty(4, 64, device="cuda", dtype=torch.float16))


def test_longest_tokens():
    # 2^26 features, the most that a call takes, against fp64 on the GPU
    m = 1 << 26
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (0.5 + torch.randn(1, m, generator=g, device="cuda")).bfloat16()
    dy = torch.randn(1, m, generator=g, device="cuda").bfloat16()
    w = (1 + 0.3 * torch.randn(m, generator=g, device="cuda")).bfloat16()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    thl.layernorm(x, w, w, y, eps=EPS)
    thl.layernorm_backward(x, dy, w, dx, dw, db, eps=EPS)
    torch.cuda.synchronize()
    X, G, W = x.double(), dy.double(), w.double()
    d = X - X.mean(dim=1, keepdim=True)
    rho = torch.rsqrt(d.square().mean(dim=1, keepdim=True) + EPS)
    h, t = d * rho, W * G
    c = (64 + m / 8192 + 22 + 8) * ref.U  # as the oracle counts them; |s| and |d| are 1 on average, rho 1
    e_h = c * (2 + 2 * h.abs())
    want = h * W + W
    assert bool(((y.double() - want).abs() <= 2 * e_h * W.abs() + 8 * ref.U * want.abs() + ref.half_step(want, y.dtype) * 1.01).all())
    want = rho * (t - t.mean(dim=1, keepdim=True) - h * (t * h).mean(dim=1, keepdim=True))
    bound = 4 * c * rho * (t.abs() + t.abs().mean() + h.abs() * (t * h).abs().mean() + t.abs().mean())
    assert bool(((dx.double() - want).abs() <= bound + ref.half_step(want, dx.dtype) * 1.01).all())
    assert bool(((dw.double() - (G * h)[0]).abs() <= 2 * G[0].abs() * e_h[0] + 4 * ref.U * (G * h)[0].abs()).all())
    assert torch.equal(db, dy[0].float())


@pytest.mark.parametrize("kind", ["e2m1", "e4m3", "e5m2"])
@pytest.mark.parametrize("m", [33, 300, 2050, 5000, 16400])
@pytest.mark.parametrize("eps", [EPS, 0.0])
def test_nan_in_mx_blocks(kind, m, eps):
    """The blocks of the norm are thl.mx_quantize's of its fp32 output: scale 255 (NaN) where one holds a NaN."""
    x = _rand(m, 6, m, dtype="bf16", shift=0.5)
    x[1, 7], x[2, m - 1], x[4] = float("inf"), float("nan"), 3.0  # (equal features: 0 / 0 with eps = 0)
    w, b = 1 + 0.2 * _rand(1, m), _rand(2, m)
    w[m // 2], b[m - 1] = float("inf"), float("nan")
    full = torch.empty(6, m, device="cuda")
    thl.layernorm(x, w, b, full, eps=eps)
    got, want = ([torch.full((6, (m + 1) // 2 if kind == "e2m1" else m), 0xEE, dtype=torch.uint8, device="cuda"),
                  torch.full((6, (m + 31) // 32), 0xEE, dtype=torch.uint8, device="cuda")] for _ in range(2))
    typed = [v if kind == "e2m1" else v.view(F[kind]) for v in (got[0], want[0])]
    thl.layernorm(x, w, b, typed[0], eps=eps, sf=got[1])
    thl.mx_quantize(full, typed[1], want[1])
    torch.cuda.synchronize()
    assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0])
    gone = [1, 2] + ([4] if eps == 0.0 else [])
    assert bool((got[1][gone] == 255).all()) and bool((got[0][gone] == 0).all())
    assert bool((got[1][:, -1] == 255).all())  # the bias's NaN
    last = torch.tensor([0, 3, 5])
    assert bool((got[1][last, :(m - 1) // 32] < 255).all()) and bool((got[0][last, :16] != 0).any())


@pytest.mark.parametrize("m", [64, 1001, 5000, 16400])
def test_features_at_the_end_of_fp32(m):
    # squares past fp32's range give the bias, a sum of features past it NaN
    x = _rand(m, 3, m)
    x[1] *= 1e30
    x[2] = 3e38
    w, b, y = 1 + 0.2 * _rand(1, m), _rand(2, m), torch.empty(3, m, device="cuda")
    thl.layernorm(x, w, b, y, eps=EPS)
    torch.cuda.synchronize()
    assert torch.equal(y[1], b) and bool(torch.isnan(y[2]).all())
    _, want, err = ref.layernorm(x[:1], None, w, b, EPS)
    _check_float(y[:1], want, err, "the other token")
