"""Layer norm, MX quantization, the router and the layer of experts as a model's layer runs them, captured, on several
streams and inside autograd functions, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import tile_hierarchy_linear_amd as thl
from oracle import operators as ref

pytestmark = pytest.mark.gpu
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


def _up(v, q):
    return -(-v // q) * q


def _mx(x, kind="e2m1"):
    """(elements, scales) of a (rows, k) array, laid out as the products want them."""
    n, m = x.shape
    sf = torch.zeros(n, _up(-(-m // 32), 16), dtype=torch.uint8, device="cuda")
    if kind == "e2m1":
        y = torch.zeros(n, _up((m + 1) // 2, 16), dtype=torch.uint8, device="cuda")[:, :(m + 1) // 2]
    else:
        y = torch.zeros(n, _up(m, 16), dtype=torch.uint8, device="cuda")[:, :m].view(torch.float8_e4m3fn)
    thl.mx_quantize(x, y, sf)
    return y, sf


def _values(x, kind):
    q, codes = ref.mx_quantize(x, kind)
    return q * torch.pow(2.0, codes.double() - 127).repeat_interleave(32, dim=1)[:, :x.shape[1]]


@pytest.mark.parametrize("kind", ["e2m1", "e4m3"])
def test_quantized_operands_multiply(kind):
    """norm -> blocks -> product, and the weight's gradient from the blocks along the tokens (K = tokens).  Products of
    these elements are exact in fp32 and their sums rounded: K + 8 whole steps of the sum of magnitudes."""
    g = torch.Generator().manual_seed(0)
    n, m, out = 160, 256, 192
    x = (torch.randn(n, m, generator=g) + 0.5).bfloat16().cuda()
    w = (torch.randn(out, m, generator=g) / 16).bfloat16().cuda()
    dy = torch.randn(n, out, generator=g).bfloat16().cuda()
    h = torch.empty_like(x)
    thl.layernorm(x, None, None, h, eps=EPS)
    code = 2 if kind == "e2m1" else 1

    def product(a, sa, b, sb, rows, cols, k):  # (cols, rows): column-major rows x cols
        d = torch.empty(cols, rows, device="cuda")
        thl.gemm(a, b, d, m=rows, n=cols, k=k, lda=code * a.stride(0), ldb=code * b.stride(0), ldd=rows, op_a="T",
                 op_b="N", type_ab=kind, sfa=sa, ld_sfa=sa.stride(0), sfb=sb, ld_sfb=sb.stride(0))
        torch.cuda.synchronize()
        return d

    def check(d, a, b, k):
        want, size = b @ a.t(), b.abs() @ a.abs().t()
        assert bool(((ref.f64(d) - want).abs() <= (k + 8) * 2 * ref.U * size).all())

    qw, sw = _mx(w, kind)
    qh, sh = _mx(h, kind)
    check(product(qw, sw, qh, sh, out, n, m), _values(w, kind), _values(h, kind), m)
    # dW (out, m) = dy^T h: both operands' blocks along the tokens
    def turned(v):
        c = v.shape[1]
        if kind == "e2m1":
            y = torch.zeros(c, _up(n // 2, 16), dtype=torch.uint8, device="cuda")[:, :n // 2]
        else:
            y = torch.zeros(c, _up(n, 16), dtype=torch.uint8, device="cuda")[:, :n].view(torch.float8_e4m3fn)
        sf = torch.zeros(c, _up(n // 32, 16), dtype=torch.uint8, device="cuda")
        thl.mx_quantize(v, y_t=y, sf_t=sf)
        return y, sf

    qt, st = turned(h)
    gt, sg = turned(dy)
    check(product(qt, st, gt, sg, m, out, n), _values(h.t(), kind), _values(dy.t(), kind), n)


class _Layer:
    """norm -> router's product -> router -> experts on MX weights, for a few tokens, and the training side's gradients."""

    def __init__(self, seed, n=5, m=256, hidden=96, experts=12, topk=3, w="e2m1"):
        g = torch.Generator().manual_seed(seed)
        self.n, self.m, self.hidden, self.experts, self.topk = n, m, hidden, experts, topk
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.x, self.res, self.dy = (torch.empty(n, m, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        self.w, self.b = (1 + 0.2 * r(m)).bfloat16().cuda(), (0.1 * r(m)).bfloat16().cuda()
        self.wr = (r(experts, m) / m ** 0.5).bfloat16().cuda()
        self.w1 = (r(experts, 2 * hidden, m) / m ** 0.5).bfloat16().cuda()
        self.w2 = (r(experts, m, hidden) / hidden ** 0.5).bfloat16().cuda()
        e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.h, self.s = torch.empty_like(self.x), torch.empty_like(self.x)
        self.logits, self.dlogits = e(n, experts), e(n, experts)
        self.ids, self.weights, self.dweights = e(n, topk, dtype=torch.int32), e(n, topk), r(n, topk).cuda()
        self.y, self.dx = e(n, m, dtype=torch.bfloat16), torch.empty_like(self.x)
        self.dw, self.db = e(m), e(m)
        if w == "bf16":
            self.q1, self.q2, self.s1, self.s2 = self.w1, self.w2, None, None
        else:
            q1, s1 = _mx(self.w1.reshape(-1, m), w)
            q2, s2 = _mx(self.w2.reshape(-1, hidden), w)
            self.q1, self.s1 = q1.unflatten(0, (experts, -1)), s1.unflatten(0, (experts, -1))
            self.q2, self.s2 = q2.unflatten(0, (experts, -1)), s2.unflatten(0, (experts, -1))
        self.blocks, self.sf = _mx(self.x)
        self.fill(seed)

    def fill(self, seed):
        g = torch.Generator().manual_seed(1000 + seed)
        for t in (self.x, self.res, self.dy):
            t.copy_(torch.randn(self.n, self.m, generator=g))
        torch.cuda.synchronize()

    def run(self):
        thl.layernorm(self.x, self.w, self.b, self.h, eps=EPS, residual=self.res, residual_out=self.s)
        thl.gemm(self.wr, self.h, self.logits, m=self.experts, n=self.n, k=self.m, lda=self.m, ldb=self.m,
                 ldd=self.experts, op_a="T", op_b="N", type_ab="bf16")
        thl.moe_route(self.logits, self.ids, self.weights, renormalize=True)
        thl.moe_layer(self.h, self.ids, self.weights, self.q1, self.q2, self.y, sf1=self.s1, sf2=self.s2)
        thl.mx_quantize(self.h, self.blocks, self.sf)
        thl.moe_route_backward(self.logits, self.ids, self.dweights, self.dlogits, renormalize=True)
        thl.layernorm_backward(self.s, self.dy, self.w, self.dx, self.dw, self.db, eps=EPS)

    def outputs(self):
        return [t.clone() for t in (self.s, self.h, self.logits, self.ids, self.weights, self.y, self.blocks, self.sf,
                                    self.dlogits, self.dx, self.dw, self.db)]

    def expected(self, seed):
        self.fill(seed)
        self.run()
        torch.cuda.synchronize()
        return self.outputs()


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("w", ["bf16", "e2m1", "e4m3"])
def test_a_layer_against_the_formulas(w):
    l = _Layer(0, w=w)
    l.run()
    torch.cuda.synchronize()
    # each operator on what the one before it gave, in fp64
    s, h, err = ref.layernorm(l.x, l.res, l.w, l.b, EPS)
    assert bool(((ref.f64(l.h) - h).abs() <= err + ref.half_step(h.abs() + err, torch.bfloat16)).all())
    logits = ref.f64(l.h) @ ref.f64(l.wr).t()
    size = ref.f64(l.h).abs() @ ref.f64(l.wr).abs().t()
    assert bool(((ref.f64(l.logits) - logits).abs() <= (l.m + 8) * 2 * ref.U * size).all())
    ids, weights, _, _ = ref.moe_route(l.logits, l.topk, "softmax", True, 1.0)
    assert torch.equal(l.ids.cpu(), ids) and bool(((ref.f64(l.weights) - weights).abs() <= 64 * ref.U).all())
    v1, v2 = l.w1, l.w2
    if w != "bf16":
        v1 = _values(l.w1.reshape(-1, l.m), w).reshape(l.w1.shape)
        v2 = _values(l.w2.reshape(-1, l.hidden), w).reshape(l.w2.shape)
    y, bound = ref.moe_layer(l.h, l.ids.cpu(), l.weights, v1.double().cpu(), v2.double().cpu(), True, "silu")
    assert bool(((ref.f64(l.y) - y).abs() <= bound + ref.half_step(y.abs() + bound, torch.bfloat16)).all())


def test_the_few_token_layer_is_the_sorted_one():
    """moe_layer beside sort -> gather -> products by expert -> combine on the same inputs; between the two products the
    latter rounds u to bf16, half a step of 2^-8 each, and both round y once."""
    l = _Layer(3, n=40, w="bf16")
    l.run()
    rows = torch.empty(l.n, l.topk, dtype=torch.int32, device="cuda")
    offsets = torch.empty(l.experts + 1, dtype=torch.int32, device="cuda")
    thl.moe_sort(l.ids, l.experts, rows, offsets)
    xs, out = (torch.zeros(l.n * l.topk, l.m, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    thl.moe_gather(l.h, rows, xs)
    off = offsets.tolist()
    size = torch.zeros(l.n * l.topk, l.m, dtype=torch.float64)
    for e in range(l.experts):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        u = xs[a:b].float() @ l.w1[e].float().t()
        u = (torch.nn.functional.silu(u[:, :l.hidden]) * u[:, l.hidden:]).bfloat16()
        thl.gemm(l.w2[e], u, out[a:b], m=l.m, n=b - a, k=l.hidden, lda=l.hidden, ldb=l.hidden, ldd=l.m, op_a="T",
                 op_b="N", type_ab="bf16", type_d="bf16")
        torch.cuda.synchronize()
        size[a:b] = u.double().abs().cpu() @ l.w2[e].double().abs().t().cpu()
    y = torch.empty(l.n, l.m, device="cuda")
    thl.moe_combine(out, rows, y, weights=l.weights)
    torch.cuda.synchronize()
    most = torch.stack([size[rows.cpu()[:, t].long()] * ref.f64(l.weights)[:, t:t + 1] for t in range(l.topk)]).sum(dim=0)
    d = (ref.f64(l.y) - ref.f64(y)).abs()
    # u off by 2^-9 of each, fp32 products by far less; out rounded to bf16, y once more
    assert bool((d <= most * 2.0 ** -8 + 2 * ref.half_step(ref.f64(y), torch.bfloat16) + most * 2.0 ** -9).all())


def test_captured_and_replayed():
    for w in ("bf16", "e2m1"):
        s = _Layer(1, n=24, w=w)
        want = [s.expected(i) for i in range(4)]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            s.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.run()
        for i in (0, 1, 2, 3, 1):  # with eager work and other allocations between the replays
            s.fill(i)
            junk = torch.randn(1 << 20, device="cuda").sum()
            graph.replay()
            torch.cuda.synchronize()
            assert _same(s.outputs(), want[i]), i
            assert bool(torch.isfinite(junk))


def test_two_graphs_and_two_streams_at_once():
    a, b = _Layer(1, n=3), _Layer(2, n=33, w="bf16")
    want_a, want_b = a.expected(5), b.expected(6)
    graphs = []
    for s in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.run()
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for how in ("graphs", "calls"):
        for _ in range(6):
            for s, graph, stream in zip((a, b), graphs, streams):
                with torch.cuda.stream(stream):
                    s.y.zero_()
                    if how == "graphs":
                        graph.replay()
                    else:
                        s.run()
                        s.run()
            torch.cuda.synchronize()
            assert _same(a.outputs(), want_a) and _same(b.outputs(), want_b), how


def test_inputs_made_on_the_calling_stream():
    s = _Layer(5, n=17)
    want = s.expected(3)
    s.fill(4)
    g = torch.Generator().manual_seed(1003)
    new = [torch.randn(s.n, s.m, generator=g).cuda() for _ in range(3)]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            big = big @ big * 1e-3
        for t, v in zip((s.x, s.res, s.dy), new):
            t.copy_(v)
        s.run()
    torch.cuda.synchronize()
    assert _same(s.outputs(), want)


# ------------------------------------------------------------------ training

class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b):
        y = torch.empty_like(x)
        thl.layernorm(x, w, b, y, eps=EPS)
        ctx.save_for_backward(x, w)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
        thl.layernorm_backward(x, dy.contiguous(), w, dx, dw, db, eps=EPS)
        return dx, dw, db


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk):
        ids = torch.empty(logits.shape[0], topk, dtype=torch.int32, device="cuda")
        weights = torch.empty(logits.shape[0], topk, device="cuda")
        thl.moe_route(logits, ids, weights, renormalize=True)
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    def backward(ctx, dweights, _):
        logits, ids = ctx.saved_tensors
        dlogits = torch.empty_like(logits)
        thl.moe_route_backward(logits, ids, dweights.contiguous(), dlogits, renormalize=True)
        return dlogits, None


def test_gradients_through_norm_and_router():
    # fp32 throughout, sums of up to 200 terms: each side within 2e-5 of the gradient's norm
    g = torch.Generator().manual_seed(2)
    x, w, b = torch.randn(30, 200, generator=g) + 1, 1 + 0.2 * torch.randn(200, generator=g), torch.randn(200, generator=g)
    wr, up = torch.randn(200, 24, generator=g) / 14, torch.randn(30, 4, generator=g)
    leaves = [t.double().requires_grad_() for t in (x, w, b)]
    logits = torch.nn.functional.layer_norm(leaves[0], (200,), leaves[1], leaves[2], EPS) @ wr.double()
    mine = [t.cuda().requires_grad_() for t in (x, w, b)]
    weights, ids = _Route.apply(_Norm.apply(*mine) @ wr.cuda(), 4)
    (weights * up.cuda()).sum().backward()
    p = torch.softmax(logits, dim=1).gather(1, ids.cpu().long())
    (p / p.sum(dim=1, keepdim=True) * up.double()).sum().backward()
    for got, want in zip(mine, leaves):
        assert float((got.grad.cpu().double() - want.grad).norm()) <= 2e-5 * float(want.grad.norm())


# ------------------------------------------------------------------ the torch forms

def _calls(device):
    """One call of every form: its function, its tensors by name, its other arguments, and the names it writes."""
    f, i, u = torch.float32, torch.int32, torch.uint8

    def t(*shape, dtype=f):
        return torch.zeros(*shape, dtype=dtype, device=device)

    return {
        "layernorm": (thl.layernorm, dict(x=t(4, 64), w=t(64), b=t(64), y=t(4, 64), residual=t(4, 64),
                                          residual_out=t(4, 64)), {}, ("y", "residual_out")),
        "layernorm_mx": (thl.layernorm, dict(x=t(4, 64), w=t(64), b=t(64), y=t(4, 64, dtype=torch.float8_e4m3fn),
                                             sf=t(4, 16, dtype=u)), {}, ("y", "sf")),
        "layernorm_backward": (thl.layernorm_backward, dict(s=t(4, 64), dy=t(4, 64), w=t(64), dx=t(4, 64), dw=t(64),
                                                            db=t(64), dres=t(4, 64)), {}, ("dx", "dw", "db")),
        "mx_quantize": (thl.mx_quantize, dict(x=t(4, 64), y=t(4, 32, dtype=u), sf=t(4, 2, dtype=u),
                                              y_t=t(64, 2, dtype=u), sf_t=t(64, 1, dtype=u)), {},
                        ("y", "sf", "y_t", "sf_t")),
        "moe_route": (thl.moe_route, dict(logits=t(4, 16), ids=t(4, 2, dtype=i), weights=t(4, 2), bias=t(16)), {},
                      ("ids", "weights")),
        "moe_route_backward": (thl.moe_route_backward, dict(logits=t(4, 16), ids=t(4, 2, dtype=i), dweights=t(4, 2),
                                                            dlogits=t(4, 16)), {}, ("dlogits",)),
        "moe_layer": (thl.moe_layer, dict(x=t(4, 64, dtype=torch.bfloat16), ids=t(4, 2, dtype=i), weights=t(4, 2),
                                          w1=t(3, 32, 64, dtype=u).view(torch.float8_e4m3fn),
                                          w2=t(3, 64, 16, dtype=u).view(torch.float8_e4m3fn), y=t(4, 64),
                                          sf1=t(3, 32, 2, dtype=u), sf2=t(3, 64, 1, dtype=u), b1=t(3, 32), b2=t(3, 64)),
                      {}, ("y",)),
    }


FORMS = list(_calls("cpu"))


@pytest.mark.parametrize("form", FORMS)
def test_tensors_that_require_a_gradient(form):
    floats = [k for k, v in _calls("cuda")[form][1].items() if v.dtype in (torch.float32, torch.bfloat16)]
    for name in floats:
        call, tensors, rest, _ = _calls("cuda")[form]
        tensors[name].requires_grad_()
        with pytest.raises(ValueError, match=f"{name}: requires a gradient"):
            call(**tensors, **rest)
        with torch.no_grad():
            call(**tensors, **rest)
    torch.cuda.synchronize()


@pytest.mark.parametrize("form", FORMS)
def test_outputs_count_as_written(form):
    call, tensors, rest, written = _calls("cuda")[form]
    before = {k: v._version for k, v in tensors.items()}
    call(**tensors, **rest)
    torch.cuda.synchronize()
    for k, v in tensors.items():
        assert (v._version > before[k]) == (k in written), k


def test_one_token_of_strided_rows():
    # a tensor of one row may carry any stride there
    x = torch.randn(3, 64, device="cuda")
    one, same = x[:1].expand(1, 64), torch.as_strided(x, (1, 64), (7, 1))
    y, z = torch.empty(1, 64, device="cuda"), torch.empty(1, 64, device="cuda")
    thl.layernorm(one, None, None, y)
    thl.layernorm(same, None, None, z)
    torch.cuda.synchronize()
    assert torch.equal(y, z)
