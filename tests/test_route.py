"""thl.moe_route and its gradient against the plain fp64 forms, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import tile_hierarchy_linear_amd as thl
from oracle import operators as ref

pytestmark = pytest.mark.gpu
F = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# exponentials and quotients: an ulp or two each, the shift's rounding (2^-24 of a difference up to 30), sums of up to
# 16 + 6 terms
REL = (30 + 22 + 12) * ref.U


@pytest.fixture(scope="module", autouse=True)
def _give_back():
    """What lives on (a library's workspace, say) is not cut from these tests' large blocks."""
    yield
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _rand(seed, n, m, dtype="f32", scale=2.0):
    return (torch.randn(n, m, generator=torch.Generator().manual_seed(seed)) * scale).to(F[dtype]).cuda()


def _run(logits, topk, score="softmax", renorm=True, scale=1.0, bias=None):
    n = logits.shape[0]
    ids = torch.full((n, topk), -7, dtype=torch.int32, device="cuda")
    weights = torch.full((n, topk), float("nan"), device="cuda")
    thl.moe_route(logits, ids, weights, score=score, renormalize=renorm, scale=scale, bias=bias)
    torch.cuda.synchronize()
    want, w, p, by = ref.moe_route(logits, topk, score, renorm, scale, bias)
    if bias is None:
        assert torch.equal(ids.cpu(), want)
    else:  # compared in fp32: another order only where the values are that near
        i, at = ids.cpu().long(), want.long()
        assert bool(((i < 0) == (at < 0)).all())
        near = (by.gather(1, i.clamp(min=0)) - by.gather(1, at.clamp(min=0))).abs()
        assert bool(((i == at) | (near <= 2 * REL)).all())
        chosen = torch.where(i >= 0, p.gather(1, i.clamp(min=0)), 0.0)
        total = chosen.sum(dim=1, keepdim=True) if renorm else 1.0
        w = scale * chosen / total
    assert bool(((ref.f64(weights) - w).abs() <= REL * w.abs() + 1e-38).all())
    return ids, weights


@pytest.mark.parametrize("experts", [1, 2, 5, 63, 64, 65, 128, 130, 256, 300, 512, 513, 1000, 1024])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_experts(experts, score, renorm):
    for n, topk in ((1, 1), (7, min(8, experts)), (5, 3)):
        _run(_rand(experts, n, experts), topk, score, renorm, scale=2.5)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("topk", [1, 2, 8, 33, 64])
def test_types_and_choices(dtype, topk):
    _run(_rand(topk, 40, 192, dtype), topk)  # 16-bit logits: many ties


def test_ties_go_to_the_lowest_expert():
    l = torch.zeros(3, 300, device="cuda")
    l[1, 150:] = -0.0  # equal to 0
    l[2, 299], l[2, 64], l[2, 65] = 1.0, 1.0, 1.0
    ids, w = _run(l, 5)
    assert ids[0].tolist() == ids[1].tolist() == [0, 1, 2, 3, 4] and ids[2].tolist() == [64, 65, 299, 0, 1]


def test_masks():
    l = _rand(0, 8, 100)
    l[0] = -torch.inf  # nothing left
    l[1, 3:] = -torch.inf  # fewer than topk
    l[2, 50] = float("nan")
    l[3] = torch.finfo(torch.float32).min  # the type's lowest value masks nothing, all alike
    l[4, 10:] = torch.finfo(torch.float32).min
    l[5] = float("nan")
    l[6, ::2] = -torch.inf
    for score, renorm in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        ids, w = _run(l[[0, 1, 2, 4, 5, 6, 7]], 5, score, renorm)
        assert ids[0].tolist() == ids[4].tolist() == [-1] * 5 and bool((w[0] == 0).all()) and bool((w[4] == 0).all())
        assert ids[1].tolist()[3:] == [-1, -1]
    ids, w = _run(l[3:4], 4, "softmax", True)
    assert ids[0].tolist() == [0, 1, 2, 3] and bool((w == 0.25).all())
    # sigmoids that are all zero in fp32: nothing to divide by
    ids = torch.empty(1, 2, dtype=torch.int32, device="cuda")
    w = torch.empty(1, 2, device="cuda")
    thl.moe_route(l[3:4].contiguous(), ids, w, score="sigmoid", renormalize=True)
    torch.cuda.synchronize()
    assert ids[0].tolist() == [0, 1] and bool((w == 0).all())
    l = _rand(1, 1, 40)
    l[0, 7] = torch.inf
    thl.moe_route(l, ids, w, score="softmax", renormalize=True)
    torch.cuda.synchronize()
    assert int(ids[0, 0]) == 7 and bool(torch.isnan(w[0, 0]))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts", [20, 256, 700])
def test_bias_for_the_choice(score, experts):
    bias = _rand(9, 1, experts, scale=0.3)[0].contiguous()
    l = _rand(experts, 60, experts)
    l[3, :experts // 2] = -torch.inf
    for renorm in (True, False):
        ids, _ = _run(l, 6, score, renorm, bias=bias)
    plain = ref.moe_route(l, 6, score, True, 1.0)[0]
    assert not torch.equal(ids.cpu(), plain)  # the bias does choose


def test_bias_that_chooses_far_below_the_largest():
    # the chosen ones' softmax against the largest logit is nothing in fp32, their quotients are ordinary
    l = _rand(3, 6, 200)
    l[:, 7] = 300.0
    bias = torch.zeros(200, device="cuda")
    bias[[20, 90, 150]] = torch.tensor([6.0, 4.0, 2.0], device="cuda")
    bias[7] = -1.5
    ids, w = _run(l, 3, "softmax", True, bias=bias)
    assert ids.tolist() == [[20, 90, 150]] * 6 and bool((w > 0).all())


def test_bias_keeps_experts_from_being_chosen():
    l = _rand(4, 5, 70)
    bias = torch.zeros(70, device="cuda")
    bias[2:60], bias[60:] = -torch.inf, float("nan")
    for score in ("softmax", "sigmoid"):
        ids = torch.empty(5, 4, dtype=torch.int32, device="cuda")
        w = torch.empty(5, 4, device="cuda")
        thl.moe_route(l, ids, w, score=score, renormalize=True, bias=bias)
        torch.cuda.synchronize()
        assert sorted(ids[0].tolist()) == [-1, -1, 0, 1] and ids[:, 2:].eq(-1).all() and w[:, 2:].eq(0).all()
        assert bool((w.sum(dim=1) - 1).abs().max() <= 4 * ref.U)


def test_many_tokens_and_pitched_rows():
    _run(_rand(0, 5000, 64), 4)
    n = (1 << 18) + 5  # more tokens than wavefronts of the grid
    l = torch.randn(n, 8, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    ids, w = torch.empty(n, 2, dtype=torch.int32, device="cuda"), torch.empty(n, 2, device="cuda")
    dl = torch.full_like(l, float("nan"))
    thl.moe_route(l, ids, w)
    thl.moe_route_backward(l, ids, torch.ones_like(w), dl)
    torch.cuda.synchronize()
    assert torch.equal(ids.long(), torch.sort(l, dim=1, descending=True, stable=True).indices[:, :2])
    p = torch.softmax(l.double(), dim=1)
    assert bool(((w.double() - p.gather(1, ids.long())).abs() <= REL).all())
    some = p.gather(1, ids.long()).sum(dim=1, keepdim=True)
    want = p * (torch.zeros_like(p).scatter_(1, ids.long(), 1.0) - some)
    assert bool(((dl.double() - want).abs() <= 4 * REL).all())
    big = torch.zeros(1 + 50 * 103, device="cuda")
    v = big[1:].view(50, 103)[:, :100]
    v.copy_(_rand(3, 50, 100))
    _run(v, 7)
    big = torch.zeros(3000 * (1 << 20) + 64, dtype=torch.bfloat16, device="cuda")  # past 2^31 elements
    v = torch.as_strided(big, (3000, 64), (1 << 20, 1))
    v.copy_(_rand(4, 3000, 64))
    _run(v, 3)


# ------------------------------------------------------------------ gradient

def _grad(logits, topk, score, renorm, scale=1.0, ids=None):
    n, experts = logits.shape
    if ids is None:
        ids, _ = _run(logits, topk, score, renorm)
    dw = _rand(5, n, topk)
    dl = torch.full_like(logits, float("nan"))
    thl.moe_route_backward(logits, ids, dw, dl, score=score, renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    want = ref.moe_route_backward(logits, ids.cpu(), dw, score, renorm, scale)
    # each element is a sum over its choices of a weight (or a score) times a difference of two gradients, each of a few
    # roundings beyond the weight's
    p = ref.moe_route(logits, 1, score, renorm, 1.0)[2]
    ok = (ids.cpu() >= 0) & (ids.cpu() < experts)
    at = torch.where(ok, ids.cpu(), 0).long()
    share = torch.where(ok, p.gather(1, at), 0.0)
    if renorm:
        share = share / share.sum(dim=1, keepdim=True).clamp(min=1e-300)
    size = torch.zeros_like(p).scatter_add_(1, at, share)
    if score == "softmax" and not renorm:
        size = size + topk * p
    bound = 8 * REL * abs(scale) * size * ref.f64(dw).abs().amax(dim=1, keepdim=True) + 1e-15
    d = (ref.f64(dl) - want).abs()
    assert bool((d <= bound + ref.half_step(want.abs() + bound, dl.dtype)).all()), float((d - bound).max())
    return ids, dw, dl


@pytest.mark.parametrize("experts", [1, 5, 64, 65, 200, 256, 513, 1024])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient(experts, score, renorm):
    for n, topk in ((1, 1), (9, min(8, experts))):
        _grad(_rand(experts, n, experts), topk, score, renorm, scale=1.5)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_types_and_masks(dtype, score, renorm):
    l = _rand(2, 12, 100, dtype)
    l[0] = -torch.inf
    l[1, 2:] = -torch.inf
    l[2, ::2] = -torch.inf
    ids, _, dl = _grad(l, 4, score, renorm)
    assert bool((dl[0] == 0).all())


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_of_the_same_expert_twice_and_of_none(score, renorm):
    ids = torch.tensor([[3, 3, 1], [-1, 4, 99], [-1, -1, -1]], dtype=torch.int32, device="cuda")
    _grad(_rand(8, 3, 50), 3, score, renorm, ids=ids)
    l, dl = _rand(8, 3, 50), torch.full((3, 50), float("nan"), device="cuda")
    thl.moe_route_backward(l, ids[:, :0].contiguous(), l[:, :0].contiguous(), dl, score=score, renormalize=renorm)
    torch.cuda.synchronize()
    assert bool((dl == 0).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,experts,topk", [(4099, 60, 16), (4099, 64, 17), (8195, 100, 5), (16385, 200, 8)])
def test_gradient_of_many_tokens(score, n, experts, topk):
    # few experts, many tokens: several tokens a wavefront; some choices shared, some of no expert
    g = torch.Generator().manual_seed(n)
    l = _rand(n, n, experts)
    ids = torch.stack([torch.randperm(experts, generator=g)[:topk] for _ in range(n)]).int()
    ids[5::9, 1] = ids[5::9, 0]
    ids[2::7, -1] = -1
    ids[n - 1] = experts
    dw = torch.randn(n, topk, generator=g)
    dl = torch.full_like(l, float("nan"))
    thl.moe_route_backward(l, ids.cuda(), dw.cuda(), dl, score=score, renormalize=True, scale=1.5)
    torch.cuda.synchronize()
    want = ref.moe_route_backward(l, ids, dw, score, True, 1.5)
    # each choice's w (g - along), with |along| <= max|g| and w <= 1: REL of w, of along and (sigmoid) of the slope, of
    # magnitudes up to 2 max|g|; two choices at most in one place
    near = 10 * REL * 1.5 * dw.abs().amax(dim=1, keepdim=True).double()
    assert bool(((ref.f64(dl) - want).abs() <= near).all())
    thl.moe_route_backward(l, ids.cuda(), dw.cuda(), l, score=score, renormalize=True, scale=1.5)  # in place
    torch.cuda.synchronize()
    assert torch.equal(l, dl)


def test_gradient_against_differences():
    """Central differences of the fp64 weights in a random direction: off by h^2 / 6 of a third derivative of order one."""
    l = _rand(3, 6, 40)
    h, dirs = 1e-4, torch.randn(6, 40, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, dw, dl = _grad(l, 4, score, renorm)
            at = ids.cpu().long()

            def loss(v):
                p = torch.softmax(v, dim=1) if score == "softmax" else torch.sigmoid(v)
                p = p.gather(1, at)
                return float(((p / p.sum(dim=1, keepdim=True) if renorm else p) * ref.f64(dw)).sum())

            num = (loss(ref.f64(l) + h * dirs) - loss(ref.f64(l) - h * dirs)) / (2 * h)
            got = ref.f64(dl) * dirs
            assert abs(num - float(got.sum())) <= 1e-5 * float(got.abs().sum())


def test_gradient_over_the_logits():
    for score, renorm in (("softmax", True), ("softmax", False), ("sigmoid", True)):
        l = _rand(3, 60, 300)
        ids, dw, dl = _grad(l, 4, score, renorm)
        thl.moe_route_backward(l, ids, dw, l, score=score, renormalize=renorm)
        torch.cuda.synchronize()
        assert torch.equal(l, dl)


@pytest.mark.parametrize("bad", ["ids", "weights", "score", "bias", "dlogits", "device"])
def test_torch_form_refusals(bad):
    l, ids, w = _rand(0, 4, 16), torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    with pytest.raises((ValueError, thl.ThlError)):
        if bad == "ids":
            thl.moe_route(l, ids.long(), w)
        elif bad == "weights":
            thl.moe_route(l, ids, w.half())
        elif bad == "score":
            thl.moe_route(l, ids, w, score="tanh")
        elif bad == "bias":
            thl.moe_route(l, ids, w, bias=torch.zeros(16, device="cuda").half())
        elif bad == "dlogits":
            thl.moe_route_backward(l, ids, w, l.half())
        else:
            thl.moe_route(l, ids.cpu(), w)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("experts", [40, 256, 700])
def test_infinite_logits_and_a_bias(renorm, experts):
    """Softmax scores of a token with a logit of +infinity are NaN: its weights say so, and the logits alone are compared
    (a bias still keeps its expert out).  Other tokens and sigmoid scores go on as they are."""
    l = _rand(experts, 7, experts)
    plain = l.clone()
    l[1, 7] = torch.inf
    l[2, [30, 9]] = torch.inf
    l[4, 5], l[4, 8:] = torch.inf, -torch.inf
    bias = _rand(1, 1, experts, scale=0.3)[0].contiguous()
    bias[9], bias[11] = -torch.inf, float("nan")
    out = []
    for v in (plain, l):
        ids, w = torch.empty(7, 6, dtype=torch.int32, device="cuda"), torch.empty(7, 6, device="cuda")
        thl.moe_route(v, ids, w, score="softmax", renormalize=renorm, bias=bias)
        out += [ids.cpu(), w.cpu()]
    torch.cuda.synchronize()
    same = [0, 3, 5, 6]
    assert torch.equal(out[2][same], out[0][same]) and torch.equal(out[3][same], out[1][same])
    may = torch.isfinite(bias).cpu()
    for j in (1, 2, 4):
        by = torch.where(may, l[j].cpu(), -torch.inf)
        want = [e for e in torch.sort(by, descending=True, stable=True).indices.tolist() if by[e] > -torch.inf][:6]
        assert out[2][j].tolist() == want + [-1] * (6 - len(want))
        assert bool(torch.isnan(out[3][j, :len(want)]).all()) and bool((out[3][j, len(want):] == 0).all())
    ids, w = _run(l, 6, "sigmoid", renorm, bias=torch.where(torch.isfinite(bias), bias, 0.0))
    assert bool(torch.isfinite(w).all())
