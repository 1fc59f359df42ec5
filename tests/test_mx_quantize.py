"""thl.mx_quantize against the exact fp64 rule, on the GPU: codes and scales bit for bit."""
import pytest

torch = pytest.importorskip("torch")

import tile_hierarchy_linear_amd as thl
from oracle import operators as ref

pytestmark = pytest.mark.gpu
F = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
     "e5m2": torch.float8_e5m2}


@pytest.fixture(scope="module", autouse=True)
def _give_back():
    """What lives on (a library's workspace, say) is not cut from these tests' large blocks."""
    yield
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _empty(n, m, kind, pad, fill=0xEE):
    """A pitched (n, m) output with the array behind it."""
    cols = (m + 1) // 2 if kind == "e2m1" else m
    whole = torch.full((n, cols + pad), fill, dtype=torch.uint8, device="cuda")
    return whole, whole[:, :cols] if kind == "e2m1" else whole[:, :cols].view(F[kind])


def _same(whole, sf, x, kind, cols):
    """`whole` and `sf` hold x's blocks, and nothing else of them was written."""
    values, codes = ref.mx_quantize(x, kind)
    n, m = x.shape
    nb = (m + 31) // 32
    assert torch.equal(sf.cpu()[:, :nb], codes) and bool((sf[:, nb:] == 0xEE).all())
    assert bool((whole[:, cols:] == 0xEE).all())
    got = whole[:, :cols].cpu()
    if kind == "e2m1":
        v = ref.e2m1_values(got, m)
        if m % 2:
            assert bool((got[:, -1] >> 4 == 0).all())
        sign = torch.signbit(v) == torch.signbit(values)
        assert torch.equal(v, values)
    else:
        v = ref.f64(got.view(F[kind]))
        sign = torch.signbit(v) == torch.signbit(values)
        assert torch.equal(v, values)
    assert bool((sign | (codes == 255).repeat_interleave(32, dim=1)[:, :m]).all())


def _run(x, kind, rows=True, cols=True, pad=0, sf_pad=2):
    n, m = x.shape
    out = {}
    if rows:
        whole, y = _empty(n, m, kind, pad)
        sf = torch.full((n, (m + 31) // 32 + sf_pad), 0xEE, dtype=torch.uint8, device="cuda")
        out["rows"] = (whole, y, sf)
    if cols:
        whole, y = _empty(m, n, kind, pad)
        sf = torch.full((m, (n + 31) // 32 + sf_pad), 0xEE, dtype=torch.uint8, device="cuda")
        out["cols"] = (whole, y, sf)
    r, c = out.get("rows", (None,) * 3), out.get("cols", (None,) * 3)
    thl.mx_quantize(x, r[1], r[2], y_t=c[1], sf_t=c[2])
    torch.cuda.synchronize()
    if rows:
        _same(r[0], r[2], x, kind, r[1].shape[1])
    if cols:
        _same(c[0], c[2], x.t(), kind, c[1].shape[1])
    return out


def _rand(seed, n, m, dtype):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(n, m, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g)) * torch.exp(torch.randn(1, m, generator=g))
    return v.to(F[dtype]).cuda()


@pytest.mark.parametrize("kind", ["e2m1", "e4m3", "e5m2"])
@pytest.mark.parametrize("n,m", [(1, 1), (1, 31), (1, 64), (3, 33), (31, 7), (32, 32), (33, 129), (64, 512), (130, 1000),
                                 (257, 640), (5, 4100), (300, 3), (128, 128), (129, 257)])
def test_sizes(kind, n, m):
    for dtype in ("bf16", "f16", "f32"):
        x = _rand(n + m, n, m, dtype)
        _run(x, kind)
        _run(x, kind, cols=False, pad=3)
        _run(x, kind, rows=False, pad=5)


@pytest.mark.parametrize("kind", ["e2m1", "e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_pitched_at_element_offsets(kind, dtype):
    for offset in (0, 1, 3):
        big = torch.zeros(offset + 70 * 205, dtype=F[dtype], device="cuda")
        x = big[offset:].view(70, 205)[:, :200]
        x.copy_(_rand(7, 70, 200, dtype))
        _run(x, kind, pad=1)


@pytest.mark.parametrize("kind", ["e2m1", "e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_16_bit_value(kind, dtype):
    # each value of the type in a block whose largest it is, and under a largest magnitude 2^0 .. 2^8 above it
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(F[dtype])
    lead = torch.tensor([0.0, 1.0, 3.0, 6.0, 24.0, 100.0, 300.0, 1000.0], dtype=F[dtype])
    block = torch.zeros(8, 1 << 16, 2, dtype=F[dtype])
    block[:, :, 0], block[:, :, 1] = x, lead[:, None]
    x = torch.nn.functional.pad(block.reshape(-1, 2), (0, 30)).reshape(4096, -1).cuda()
    _run(x, kind, cols=False)
    _run(x[:, :512].t().contiguous(), kind, rows=False)


@pytest.mark.parametrize("kind", ["e2m1", "e4m3", "e5m2"])
def test_midpoints_and_scales(kind):
    # under every scale from fp32's smallest to its largest: the elements, the midpoints between them and their neighbours
    top = ref.TOP[kind]
    if kind == "e2m1":
        codes = torch.tensor(ref.E2M1, dtype=torch.float32)
    else:
        codes = torch.arange(256, dtype=torch.uint8).view(F[kind]).float()
        codes = torch.sort(codes[torch.isfinite(codes) & (codes >= 0)]).values
    mids = (codes[1:] + codes[:-1]) / 2
    v = torch.cat([codes, mids, torch.nextafter(mids, torch.tensor(0.0)), torch.nextafter(mids, torch.tensor(1e9))])
    v = torch.cat([v, -v])
    v = torch.nn.functional.pad(v, (0, -v.numel() % 31)).reshape(-1, 31)
    v = torch.cat([torch.full((v.shape[0], 1), top), v], dim=1)  # the block's largest
    for e in list(range(-149, -120)) + [-64, -3, 0, 5, 77] + list(range(104, 126)):
        x = torch.ldexp(v.double(), torch.tensor(float(e), dtype=torch.float64)).float()
        x = torch.where(torch.isinf(x), torch.finfo(torch.float32).max, x)
        _run(x.cuda(), kind, cols=False)
        _run(x.t().contiguous().cuda(), kind, rows=False)


@pytest.mark.parametrize("kind", ["e2m1", "e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_nan_infinities_and_zeros(kind, dtype):
    x = _rand(1, 96, 128, dtype)
    x[0, :32] = 0.0
    x[1, 32:64] = -0.0
    x[2, 5] = float("nan")
    x[3, 40], x[3, 41] = float("inf"), -float("inf")
    x[4, 70], x[4, 71] = float("nan"), float("inf")
    x[5] = torch.finfo(F[dtype]).max
    x[6] = torch.finfo(F[dtype]).tiny
    x[7, 0] = -torch.finfo(F[dtype]).max
    out = _run(x, kind)
    _, y, sf = out["rows"]
    assert int(sf[2, 0]) == 255 and int(sf[2, 1]) != 255 and int(sf[0, 0]) == 0
    # the infinities are ones again under their scale
    if kind != "e2m1":
        v = y[3].float() * torch.pow(2.0, sf[3, :4].float() - 127).repeat_interleave(32)
        assert v[40] == float("inf") and v[41] == -float("inf") and bool(torch.isfinite(v[:32]).all())


def test_many_tiles():
    _run(_rand(3, 1030, 4200, "bf16"), "e2m1")
    _run(_rand(3, 9000, 40, "f32"), "e4m3")


def test_offsets_past_32_bits():
    n, m, pitch = 4200, 64, 1 << 20
    big = torch.zeros(n * pitch, dtype=torch.bfloat16, device="cuda")
    x = big.view(n, pitch)[:, :m]
    x.copy_(_rand(0, n, m, "bf16"))
    _run(x, "e2m1")
    del big, x
    x = _rand(0, 4200, 64, "bf16")  # and of the outputs
    whole = torch.full((4200, pitch + 32), 0xEE, dtype=torch.uint8, device="cuda")
    sf = torch.full((4200, pitch), 0xEE, dtype=torch.uint8, device="cuda")
    thl.mx_quantize(x, whole[:, :64].view(F["e4m3"]), sf[:, :2])
    torch.cuda.synchronize()
    _same(whole[:, :80], sf[:, :4], x, "e4m3", 64)


@pytest.mark.parametrize("bad", ["pair", "types", "shape", "none", "device", "input"])
def test_torch_form_refusals(bad):
    x, u = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 32, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(4, 2, dtype=torch.uint8, device="cuda")
    with pytest.raises((ValueError, thl.ThlError)):
        if bad == "pair":
            thl.mx_quantize(x, u)
        elif bad == "types":
            thl.mx_quantize(x, u, sf, y_t=torch.zeros(64, 4, device="cuda").to(F["e4m3"]), sf_t=torch.zeros(64, 1, dtype=torch.uint8, device="cuda"))
        elif bad == "shape":
            thl.mx_quantize(x, u[:, :31], sf)
        elif bad == "none":
            thl.mx_quantize(x)
        elif bad == "device":
            thl.mx_quantize(x, u, sf.cpu())
        else:
            thl.mx_quantize(x.double(), u, sf)
