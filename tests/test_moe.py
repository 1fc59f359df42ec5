"""Tokens sorted by expert and back, against plain loops and fp64, on the GPU."""
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


def _ids(n, topk, experts, seed=0, lo=0, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, experts, (n, topk), generator=g).to(dtype)


def _sort(ids, experts):
    d = ids.cuda()
    n, topk = ids.shape
    rows = torch.full((n, topk), -7, dtype=torch.int32, device="cuda")
    offsets = torch.full((experts + 1,), -7, dtype=torch.int32, device="cuda")
    order = torch.full((n * topk,), -7, dtype=torch.int32, device="cuda")
    thl.moe_sort(d, experts, rows, offsets, order=order)
    torch.cuda.synchronize()
    return rows, offsets, order


def _check_sort(ids, experts):
    rows, offsets, order = _sort(ids, experts)
    want = ref.moe_sort(ids, experts)
    assert torch.equal(rows.cpu(), want[0])
    assert torch.equal(offsets.cpu(), want[1])
    kept = int(want[1][-1])
    assert torch.equal(order.cpu()[:kept], want[2])
    assert bool((order[kept:] == -7).all())  # entries past the last place
    return rows, offsets, order


@pytest.mark.parametrize("n,topk,experts", [
    (1, 1, 1), (1, 8, 128), (5, 3, 7), (24, 8, 128), (63, 1, 64), (64, 1, 3), (65, 2, 2), (512, 8, 1024),
    (513, 8, 1024), (4096, 1, 60), (4097, 1, 60), (3000, 6, 255), (20000, 8, 64), (131072, 2, 1000), (200000, 8, 17),
])
def test_sort(n, topk, experts):
    _check_sort(_ids(n, topk, experts, seed=n), experts)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort_drops_what_is_no_expert(dtype):
    for n in (50, 5000):
        ids = _ids(n, 4, 12, seed=1, lo=-3, dtype=dtype)
        ids[3, 1] = 12
        ids[4, 0] = 2 ** 31 - 1
        if dtype == torch.int64:
            ids[5, 0] = 2 ** 32 + 3  # 3 in its low half
        _check_sort(ids, 12)
        _check_sort(torch.full_like(ids, -1), 12)  # nothing kept


def test_sort_one_expert_takes_all_and_twice():
    for n in (100, 6000):
        _check_sort(torch.full((n, 2), 5, dtype=torch.int64), 9)


def test_sort_pitched_ids_and_no_order():
    ids = _ids(700, 9, 33, seed=2)
    d = ids.cuda()[:, :5]
    rows, offsets = torch.empty(700, 5, dtype=torch.int32, device="cuda"), torch.empty(34, dtype=torch.int32,
                                                                                      device="cuda")
    thl.moe_sort(d, 33, rows, offsets)
    torch.cuda.synchronize()
    want = ref.moe_sort(ids[:, :5], 33)
    assert torch.equal(rows.cpu(), want[0]) and torch.equal(offsets.cpu(), want[1])


def test_sort_of_nothing():
    for shape in ((0, 4), (4, 0)):
        _, offsets, _ = _sort(torch.zeros(*shape, dtype=torch.int64), 6)
        assert bool((offsets == 0).all())


def _gather(n, topk, m, dtype, experts=8, pitch=0, sf=False, lo=-1, short=0, seed=0, type_x=None):
    ids = _ids(n, topk, experts, seed=seed, lo=lo)
    rows, offsets, _ = _sort(ids, experts)
    g = torch.Generator().manual_seed(seed)
    size = torch.empty(0, dtype=dtype).element_size()
    bits = torch.randint(0, 256, (n, (m + pitch) * size), generator=g).to(torch.uint8).cuda()
    x = bits.view(dtype)[:, :m]
    total = n * topk - short
    y = torch.full((total, (m + pitch) * size), 0xEE, dtype=torch.uint8, device="cuda").view(dtype)[:, :m]
    features = 2 * m if type_x == "e2m1" else m
    nb = (features + 31) // 32
    sfx = torch.randint(0, 256, (n, nb + 2), generator=g).to(torch.uint8).cuda() if sf else None
    sfy = torch.full((total, nb + 5), 0xEE, dtype=torch.uint8, device="cuda") if sf else None
    thl.moe_gather(x, rows, y, sf=sfx, sf_y=sfy, type_x=type_x)
    torch.cuda.synchronize()
    want = torch.full((total, m * size), 0xEE, dtype=torch.uint8)
    want_sf = torch.full((total, nb + 5), 0xEE, dtype=torch.uint8)
    xb = x.contiguous().view(torch.uint8).cpu().reshape(n, m * size)
    for j, places in enumerate(rows.cpu().tolist()):
        for p in places:
            if 0 <= p < total:
                want[p] = xb[j]
                if sf:
                    want_sf[p, :nb] = sfx[j, :nb].cpu()
    whole = y._base if y._base is not None else y
    assert torch.equal(y.contiguous().view(torch.uint8).cpu().reshape(total, m * size), want)
    rest = whole.view(torch.uint8).reshape(total, (m + pitch) * size)[:, m * size:]
    assert bool((rest == 0xEE).all())  # padding of the rows
    if sf:
        assert torch.equal(sfy.cpu(), want_sf)


@pytest.mark.parametrize("m", [1, 3, 8, 100, 1000, 4097])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float8_e4m3fn])
def test_gather(m, dtype):
    _gather(13, 3, m, dtype, sf=True, seed=m)
    _gather(9, 8, m, dtype, pitch=3, lo=0, seed=m + 1)


def test_gather_many_tokens_and_short_rows():
    _gather(30000, 2, 4, torch.bfloat16)
    _gather(700, 6, 640, torch.float8_e5m2, sf=True, pitch=16)


def test_gather_packed_and_into_fewer_rows():
    _gather(20, 4, 96, torch.uint8, sf=True, type_x="e2m1")
    _gather(20, 4, 64, torch.float16, short=11, lo=0)  # places past the array are left out


def _setup(n, topk, m, x, seed=0, lo=-1, experts=8, pitch=0):
    rows, _, _ = _sort(_ids(n, topk, experts, seed=seed, lo=lo), experts)
    g = torch.Generator().manual_seed(seed)
    xt = torch.zeros(n * topk, m + pitch, dtype=F[x], device="cuda")[:, :m]
    xt.copy_(torch.randn(n * topk, m, generator=g))
    weights = torch.rand(n, topk, generator=g).cuda()
    dy = torch.randn(n, m, generator=g)
    return rows, xt, weights, dy


def _check(got, want, bound):
    d = (ref.f64(got) - want).abs()
    assert not bool((d > bound).any()), float((d / bound.clamp(min=1e-300)).max())


@pytest.mark.parametrize("m", [1, 7, 64, 777, 2048, 5000])
@pytest.mark.parametrize("topk", [1, 2, 5, 8, 9])
def test_combine(m, topk):
    for x, y in (("bf16", "bf16"), ("f16", "f32"), ("f32", "f16")):
        rows, xt, weights, _ = _setup(17, topk, m, x, seed=m, pitch=1)
        for w in (weights, None):
            yt = torch.full((17, m + 2), float("nan"), dtype=F[y], device="cuda")
            thl.moe_combine(xt, rows, yt[:, :m], weights=w)
            torch.cuda.synchronize()
            want, bound = ref.moe_combine(xt, rows, None if w is None else w.cpu(), 17, m)
            _check(yt[:, :m], want, bound + ref.half_step(want, F[y]) * 1.001)
            assert bool(torch.isnan(yt[:, m:]).all())


def test_combine_tokens_without_a_row():
    rows, xt, weights, _ = _setup(6, 3, 130, "bf16", lo=0)
    xt[int(rows[1, 0])] = float("nan")
    rows[1, 0] = -1  # dropped: neither its row nor its weight is read
    weights[1, 0] = float("nan")
    rows[2] = -1
    rows[3, 1] = 10 ** 9  # no row of the array
    y = torch.full((6, 130), float("nan"), device="cuda")
    thl.moe_combine(xt, rows, y, weights=weights)
    torch.cuda.synchronize()
    want, bound = ref.moe_combine(xt, rows, weights.cpu(), 6, 130)
    assert bool((y[2] == 0).all())
    _check(y, want, bound + ref.half_step(want, torch.float32) * 1.001)


def test_combine_many_tokens():
    rows, xt, weights, _ = _setup(3000, 4, 72, "bf16", seed=3)
    y = torch.empty(3000, 72, dtype=torch.bfloat16, device="cuda")
    thl.moe_combine(xt, rows, y, weights=weights)
    torch.cuda.synchronize()
    want, bound = ref.moe_combine(xt, rows, weights.cpu(), 3000, 72)
    _check(y, want, bound + ref.half_step(want, torch.bfloat16) * 1.001)


def test_combine_without_weights_is_the_gradient_of_gather():
    # <gather(x), g> = <x, combine(g)> for every x and g: sums of the same products, in exact small integers
    n, topk, m = 40, 3, 50
    rows, _, _, _ = _setup(n, topk, m, "f32", seed=4)
    g = torch.Generator().manual_seed(5)
    x = torch.randint(-8, 9, (n, m), generator=g).float().cuda()
    gy = torch.randint(-8, 9, (n * topk, m), generator=g).float().cuda()
    y, gx = torch.zeros_like(gy), torch.empty_like(x)
    thl.moe_gather(x, rows, y)
    thl.moe_combine(gy, rows, gx)
    torch.cuda.synchronize()
    assert float((y.double() * gy.double()).sum()) == float((x.double() * gx.double()).sum())


@pytest.mark.parametrize("m", [1, 9, 512, 1024, 1030, 4096, 5126])
@pytest.mark.parametrize("topk", [1, 2, 3, 8, 11])
def test_combine_backward(m, topk):
    for x, d in (("bf16", "bf16"), ("f32", "f32"), ("f16", "f32"), ("f32", "bf16")):
        n = 9
        rows, xt, weights, dy = _setup(n, topk, m, x, seed=m, pitch=2)
        dyt = dy.to(F[d]).cuda()
        dx = torch.full((n * topk, m + 1), 7.0, dtype=F[x], device="cuda")[:, :m]
        dw = torch.full((n, topk), float("nan"), device="cuda")
        thl.moe_combine_backward(dyt, xt, rows, weights, dx, dw)
        torch.cuda.synchronize()
        want, want_w, bw = ref.moe_combine_backward(dyt, xt, rows.cpu(), weights.cpu())
        _check(dw, want_w, bw)
        full = torch.full((n * topk, m), 7.0, dtype=torch.float64)  # rows without a choice are left as they were
        for p, v in want.items():
            full[p] = v
        _check(dx, full, (ref.U * full.abs() + ref.half_step(full, F[x])) * 1.001)


def test_combine_backward_parts():
    rows, xt, weights, dy = _setup(30, 2, 640, "bf16", seed=6)
    dyt = dy.to(torch.bfloat16).cuda()
    dx, dw = torch.zeros(60, 640, dtype=torch.bfloat16, device="cuda"), torch.empty(30, 2, device="cuda")
    thl.moe_combine_backward(dyt, xt, rows, weights, dx, dw)
    dx1, dw1 = torch.zeros_like(dx), torch.empty_like(dw)
    thl.moe_combine_backward(dyt, None, rows, weights, dx1)
    thl.moe_combine_backward(dyt, xt, rows, None, None, dw1)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx1) and torch.equal(dw, dw1)


def test_combine_backward_against_differences():
    """combine is linear in x and in the weights, so a difference of the fp64 form is exact but for its own
    rounding; the kernel's fp32 products and sums stay within 1e-5 of the magnitudes."""
    n, topk, m = 7, 3, 60
    rows, xt, weights, dy = _setup(n, topk, m, "f32", seed=8, lo=0)
    dyt = dy.cuda()
    dx, dw = torch.zeros_like(xt), torch.empty_like(weights)
    thl.moe_combine_backward(dyt, xt, rows, weights, dx, dw)
    torch.cuda.synchronize()
    g = torch.Generator().manual_seed(9)
    a, b = torch.randn(n * topk, m, generator=g, dtype=torch.float64), torch.randn(n, topk, generator=g).double()

    def loss(x, w):
        return float((ref.moe_combine(x, rows, w, n, m)[0] * dy.double()).sum())

    X, W = ref.f64(xt), ref.f64(weights)
    for got, num in ((ref.f64(dx) * a, (loss(X + a, W) - loss(X - a, W)) / 2),
                     (ref.f64(dw) * b, (loss(X, W + b) - loss(X, W - b)) / 2)):
        assert abs(float(got.sum()) - num) <= 1e-5 * float(got.abs().sum())


def test_empty():
    x, i = torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    thl.moe_gather(x, i, torch.empty(0, 8, device="cuda"))
    thl.moe_combine(x, i, torch.empty(0, 8, device="cuda"))
    y = torch.full((3, 8), 5.0, device="cuda")
    thl.moe_combine(x, torch.empty(3, 0, dtype=torch.int32, device="cuda"), y)  # no choices: zeros
    torch.cuda.synchronize()
    assert bool((y == 0).all())
    dw = torch.full((3, 2), 5.0, device="cuda")  # no rows: nothing has a place
    rows = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    y.fill_(5.0)
    thl.moe_combine(x, rows, y)
    thl.moe_combine_backward(torch.ones(3, 8, device="cuda"), x, rows, None, None, dw)
    torch.cuda.synchronize()
    assert bool((dw == 0).all()) and bool((y == 0).all())


def test_offsets_past_32_bits():
    # the last row of an array of more than 2^32 bytes
    n, m, rows_y = 2, 4096, 1 << 20
    y = torch.zeros(rows_y, m + 1024, dtype=torch.float8_e4m3fn, device="cuda")[:, :m]
    x = torch.randint(0, 120, (n, m), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    rows = torch.tensor([[rows_y - 1], [0]], dtype=torch.int32, device="cuda")
    thl.moe_gather(x, rows, y)
    torch.cuda.synchronize()
    assert torch.equal(y[rows_y - 1].view(torch.uint8), x[0].view(torch.uint8))
    assert torch.equal(y[0].view(torch.uint8), x[1].view(torch.uint8))
    z = torch.zeros(rows_y, m + 1024, dtype=torch.bfloat16, device="cuda")[:, :m]
    z[rows_y - 1] = 3.0
    out = torch.empty(1, m, device="cuda")
    thl.moe_combine(z, rows[:1], out)
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())


def test_gather_of_the_longest_token():
    m = 1 << 26  # of four bytes: more pieces than a grid has rows of workgroups
    x = torch.arange(m, dtype=torch.int32, device="cuda").view(1, m).view(torch.float32)
    y = torch.zeros(2, m, device="cuda")
    thl.moe_gather(x, torch.tensor([[1]], dtype=torch.int32, device="cuda"), y)
    assert torch.equal(y[1:].view(torch.int32), x.view(torch.int32)) and not bool(y[0].any())


# rows of packed codes: bytes a row of m elements, and elements a unit of whole bytes
PACKED = {"e2m1": (lambda m: (m + 1) // 2, 2, 1), "i4": (lambda m: (m + 1) // 2, 2, 1),
          "u4": (lambda m: (m + 1) // 2, 2, 1), "e2m3": (lambda m: (6 * m + 7) // 8, 4, 3),
          "e3m2": (lambda m: (6 * m + 7) // 8, 4, 3), "i8": (lambda m: m, 1, 1), "i32": (lambda m: 4 * m, 1, 4),
          "e8m0": (lambda m: m, 1, 1)}


@pytest.mark.parametrize("fmt", sorted(PACKED))
@pytest.mark.parametrize("m", [1, 5, 31, 33, 100, 1001, 4096])
def test_gather_of_packed_rows(fmt, m):
    size, per, unit = PACKED[fmt]
    n, topk, experts = 21, 3, 5
    rows, _, _ = _sort(_ids(n, topk, experts, seed=m, lo=-1), experts)
    whole = -(-m // per) + 2  # units of whole bytes a row, two of them padding
    g = torch.Generator().manual_seed(m)
    x = torch.randint(0, 256, (n, whole * unit), generator=g).to(torch.uint8).cuda()
    y = torch.full((n * topk, whole * unit), 0xEE, dtype=torch.uint8, device="cuda")
    nb = (m + 31) // 32
    sfx = torch.randint(0, 256, (n, nb + 1), generator=g).to(torch.uint8).cuda()
    sfy = torch.full((n * topk, nb + 2), 0xEE, dtype=torch.uint8, device="cuda")
    st = thl.thl_moe_gather(m, n, topk, x.data_ptr(), whole * per, sfx.data_ptr(), nb + 1, rows.data_ptr(), n * topk,
                            y.data_ptr(), whole * per, sfy.data_ptr(), nb + 2, fmt,
                            torch.cuda.current_stream().cuda_stream)
    assert st == thl.THL_OK
    torch.cuda.synchronize()
    want, want_sf = torch.full_like(y, 0xEE).cpu(), torch.full_like(sfy, 0xEE).cpu()
    for j, places in enumerate(rows.cpu().tolist()):
        for p in places:
            if p >= 0:
                want[p, :size(m)] = x[j, :size(m)].cpu()
                want_sf[p, :nb] = sfx[j, :nb].cpu()
    assert torch.equal(y.cpu(), want) and torch.equal(sfy.cpu(), want_sf)


def test_sort_of_the_most_choices():
    # 2^30: places and their inverse, the experts in order, and within one the choices in order
    n, topk, experts = 1 << 27, 8, 100
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.empty(n, topk, dtype=torch.int32, device="cuda")
    ids.random_(0, experts + 1, generator=g)  # `experts` itself is dropped
    rows, offsets = torch.empty_like(ids), torch.empty(experts + 1, dtype=torch.int32, device="cuda")
    order = torch.full((n * topk,), -7, dtype=torch.int32, device="cuda")
    thl.moe_sort(ids, experts, rows, offsets, order=order)
    torch.cuda.synchronize()
    ids, rows = ids.view(-1), rows.view(-1)
    counts = torch.zeros(experts, dtype=torch.int64, device="cuda")
    step, last = 1 << 26, -1
    for a in range(0, n * topk, step):
        counts += torch.stack([(ids[a:a + step] == e).sum() for e in range(experts)])
    assert offsets.tolist() == [0] + counts.cumsum(0).tolist()
    kept = int(offsets[-1])
    assert kept < n * topk and bool((order[kept:] == -7).all())
    for a in range(0, kept, step):
        at = order[a:min(kept, a + step)].long()
        assert bool((rows[at] == torch.arange(a, a + at.numel(), device="cuda")).all())
        key = (ids[at].long() << 32) | at
        assert int(key[0]) > last and bool((key[1:] > key[:-1]).all())
        last = int(key[-1])
    for a in range(0, n * topk, step):
        assert bool(((rows[a:a + step] == -1) == (ids[a:a + step] == experts)).all())


def test_combine_of_the_longest_tokens():
    m = 1 << 26
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-3, 4, (3, m), generator=g, device="cuda").bfloat16()
    rows = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    weights = torch.tensor([[2.0, -0.5]], device="cuda")
    y, dx, dw = torch.empty(1, m, device="cuda"), torch.full_like(x, 9.0), torch.empty_like(weights)
    thl.moe_combine(x, rows, y, weights=weights)
    torch.cuda.synchronize()
    assert torch.equal(y[0], 2 * x[2].float() - 0.5 * x[0].float())
    dy = torch.randint(0, 2, (1, m), generator=g, device="cuda").bfloat16()
    thl.moe_combine_backward(dy, x, rows, weights, dx, dw)
    torch.cuda.synchronize()
    assert torch.equal(dx[2], 2 * dy[0]) and torch.equal(dx[0], -0.5 * dy[0]) and bool((dx[1] == 9.0).all())
    # whole numbers, of which 256 lanes add 2^18 each: exact
    assert torch.equal(dw.double()[0], torch.stack([(dy.double()[0] * x[r].double()).sum() for r in (2, 0)]))
