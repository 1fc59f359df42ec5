"""The operators as they are used: an expert layer around grouped products,
its gradients, and captured, concurrent and side-stream calls, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import tile_hierarchy_linear_amd as thl
from oracle import operators as ref

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _grouped(problems, dts, act):
    arr = (thl.thl_group_problem * len(problems))(*problems)
    dev = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8).cuda()
    flags = {"none": 0, "relu": thl.THL_EPI_RELU, "gelu": thl.THL_EPI_GELU}[act]
    st = thl.thl_gemm_grouped(len(problems), arr, dev.data_ptr(), "T", "N", 1.0, 0.0, dts, thl.thl_epilogue(flags),
                              thl.thl_scales(1.0, 1.0, None, 0, None, 0), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    return dev  # kept until the launch completes


def _bar(k, a, b, want, dtype, g=1.0):
    """The grouped product's bar: 2^-20 K max|a| max|b|, and one step of the output."""
    return 2.0 ** -20 * k * float(a.abs().max()) * float(b.abs().max()) * g + 2 * ref.half_step(want, dtype)


def test_expert_layer():
    """Residual and norm into MX rows, tokens to experts, an MX grouped product with GELU, a bf16 grouped product, and
    back: each stage against fp64 on what the stage before it stored."""
    n, h, ffn, experts, topk = 150, 256, 320, 6, 2
    g = torch.Generator().manual_seed(0)
    x = torch.randn(n, h, generator=g).bfloat16().cuda()
    res = torch.randn(n, h, generator=g).cuda()
    w = (1 + 0.2 * torch.randn(h, generator=g)).bfloat16().cuda()
    w1 = torch.randint(0, 256, (experts, ffn, h), generator=g).to(torch.uint8)
    w1[(w1 & 127) > 120] = 17  # no NaN, no largest values
    w1 = w1.cuda()
    s1 = torch.randint(112, 122, (experts, ffn, 16), generator=g).to(torch.uint8).cuda()
    w2 = (0.05 * torch.randn(experts, h, ffn, generator=g)).bfloat16().cuda()
    logits = torch.randn(n, experts, generator=g).cuda()
    logits[:, 3] = -50.0  # an expert without tokens
    top = torch.topk(logits, topk, dim=1)
    weights = torch.softmax(top.values, dim=1).contiguous()

    y = torch.empty(n, h, dtype=torch.float8_e4m3fn, device="cuda")
    sf = torch.zeros(n, 16, dtype=torch.uint8, device="cuda")
    thl.rmsnorm(x, w, y, eps=EPS, residual=res, residual_out=res, sf=sf)
    rows = torch.empty(n, topk, dtype=torch.int32, device="cuda")
    offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
    thl.moe_sort(top.indices, experts, rows, offsets)
    xs = torch.zeros(n * topk, h, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sfs = torch.zeros(n * topk, 16, dtype=torch.uint8, device="cuda")
    thl.moe_gather(y, rows, xs, sf=sf, sf_y=sfs)
    off = offsets.tolist()
    assert off[-1] == n * topk and off[3] == off[4]
    d1 = torch.full((n * topk, ffn), float("nan"), dtype=torch.bfloat16, device="cuda")
    d2 = torch.full((n * topk, h), float("nan"), dtype=torch.bfloat16, device="cuda")

    def row(t, r):
        return t.data_ptr() + r * t.stride(0) * t.element_size()

    keep = [_grouped([thl.thl_group_problem(ffn, off[e + 1] - off[e], h, w1[e].data_ptr(), h, row(xs, off[e]), h, None,
                                            ffn, row(d1, off[e]), ffn, None, s1[e].data_ptr(), 16, row(sfs, off[e]), 16)
                      for e in range(experts)], thl.make_dtypes("e4m3", "e4m3", "f32", "bf16"), "gelu")]
    keep.append(_grouped([thl.thl_group_problem(h, off[e + 1] - off[e], ffn, w2[e].data_ptr(), ffn, row(d1, off[e]), ffn,
                                                None, h, row(d2, off[e]), h, None, None, 0, None, 0)
                          for e in range(experts)], thl.make_dtypes("bf16", "bf16", "f32", "bf16"), "none"))
    out = torch.empty(n, h, device="cuda")
    thl.moe_combine(d2, rows, out, weights=weights)
    torch.cuda.synchronize()

    def mx(codes, scales):
        v = codes.view(torch.float8_e4m3fn).cpu().double()
        return v * torch.pow(2.0, scales[:, :v.shape[1] // 32].cpu().double() - 127).repeat_interleave(32, dim=1)

    for e in range(experts):
        if off[e] == off[e + 1]:
            continue
        r = slice(off[e], off[e + 1])
        a, b = mx(w1[e], s1[e]), mx(xs[r], sfs[r])
        v = b @ a.t()
        want = 0.5 * v * (1 + torch.erf(v / 2 ** 0.5))
        assert bool(((ref.f64(d1[r]) - want).abs() <= _bar(h, a, b, want, torch.bfloat16, 1.13)).all())
        a, b = ref.f64(w2[e]), ref.f64(d1[r])
        want = b @ a.t()
        assert bool(((ref.f64(d2[r]) - want).abs() <= _bar(ffn, a, b, want, torch.bfloat16)).all())
    want, bound = ref.moe_combine(d2, rows, weights.cpu(), n, h)
    assert bool(((ref.f64(out) - want).abs() <= bound + ref.half_step(want, torch.float32) * 1.001).all())
    # every token's MX row reached its places
    for j in (0, 77, n - 1):
        for p in rows[j].tolist():
            assert torch.equal(xs[p].view(torch.uint8), y[j].view(torch.uint8)) and torch.equal(sfs[p, :8], sf[j, :8])
    del keep


def test_gradients_through_the_chain():
    """norm, gather, a factor per expert, combine; its gradients against fp64 autograd of the same chain.  All fp32:
    each stage's relative error is below 2e-6 of its sums' magnitudes, the chain's below 1e-5."""
    n, m, experts, topk = 60, 130, 5, 3
    g = torch.Generator().manual_seed(1)
    x = torch.randn(n, m, generator=g)
    w = 1 + 0.2 * torch.randn(m, generator=g)
    c = 0.5 + torch.rand(experts, m, generator=g)
    up = torch.randn(n, m, generator=g)
    wt = torch.rand(n, topk, generator=g)
    ids = torch.randint(-1, experts, (n, topk), generator=g)  # some dropped

    X, W, T = (t.double().requires_grad_() for t in (x, w, wt))
    y = X * torch.rsqrt(X.square().mean(dim=1, keepdim=True) + EPS) * W
    per = torch.where((ids >= 0)[:, :, None], y[:, None, :] * c.double()[ids.clamp(min=0)], 0.0)
    (((per * T[:, :, None]).sum(dim=1)) * up.double()).sum().backward()

    xd, wd, cd, td = x.cuda(), w.cuda(), c.cuda(), wt.cuda()
    yd = torch.empty_like(xd)
    thl.rmsnorm(xd, wd, yd, eps=EPS)
    rows = torch.empty(n, topk, dtype=torch.int32, device="cuda")
    offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
    order = torch.empty(n * topk, dtype=torch.int32, device="cuda")
    thl.moe_sort(ids.cuda(), experts, rows, offsets, order=order)
    total = int(offsets[-1])
    e_of = torch.zeros(n * topk, dtype=torch.long, device="cuda")
    e_of[:total] = ids.cuda().reshape(-1)[order[:total].long()]
    xs = torch.zeros(n * topk, m, device="cuda")
    thl.moe_gather(yd, rows, xs)
    scaled = xs * cd[e_of]
    out = torch.empty(n, m, device="cuda")
    thl.moe_combine(scaled, rows, out, weights=td)
    d_scaled, d_t = torch.zeros_like(xs), torch.empty_like(td)
    thl.moe_combine_backward(up.cuda(), scaled, rows, td, d_scaled, d_t)
    d_y = torch.empty_like(yd)
    thl.moe_combine(d_scaled * cd[e_of], rows, d_y)  # gather's gradient
    d_x, d_w = torch.empty_like(xd), torch.empty_like(wd)
    thl.rmsnorm_backward(xd, d_y, wd, d_x, d_w, eps=EPS)
    torch.cuda.synchronize()
    for got, want in ((d_x, X.grad), (d_w, W.grad), (d_t, T.grad)):
        assert float((ref.f64(got) - want).norm()) <= 1e-5 * float(want.norm())


class _Step:
    """One call of every operator, on buffers of its own."""

    def __init__(self, seed, n=700, m=512, experts=9, topk=8, features=260):
        g = torch.Generator().manual_seed(seed)
        self.g, self.n, self.m, self.experts, self.topk = g, n, m, experts, topk
        self.x = torch.empty(n, m, dtype=torch.bfloat16, device="cuda")
        self.dy = torch.empty_like(self.x)
        self.ids = torch.empty(n, topk, dtype=torch.int64, device="cuda")
        self.w = torch.ones(m, device="cuda")
        self.weights = torch.rand(n, topk, generator=g).cuda()
        self.w4 = torch.randint(0, 256, (features, m // 2), generator=g).to(torch.uint8).cuda()
        self.scales = torch.rand(features, m // 64, generator=g).half().cuda()
        self.y = torch.empty_like(self.x)
        self.rows = torch.empty(n, topk, dtype=torch.int32, device="cuda")
        self.offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
        self.xs = torch.zeros(n * topk, m, dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty(n, m, dtype=torch.bfloat16, device="cuda")
        self.dxs, self.dwt = torch.zeros_like(self.xs), torch.empty_like(self.weights)
        self.dx, self.dw = torch.empty_like(self.x), torch.empty_like(self.w)
        self.d = torch.empty(40, features, dtype=torch.bfloat16, device="cuda")
        self.d1 = torch.empty(1, features, dtype=torch.bfloat16, device="cuda")
        self.fill(seed)

    def fill(self, seed):
        g = torch.Generator().manual_seed(1000 + seed)
        self.x.copy_(torch.randn(self.n, self.m, generator=g))
        self.dy.copy_(torch.randn(self.n, self.m, generator=g))
        self.ids.copy_(torch.randint(0, self.experts, (self.n, self.topk), generator=g))

    def run(self):
        thl.rmsnorm(self.x, self.w, self.y, eps=EPS)
        thl.moe_sort(self.ids, self.experts, self.rows, self.offsets)  # takes a workspace
        thl.moe_gather(self.y, self.rows, self.xs)
        thl.moe_combine(self.xs, self.rows, self.out, weights=self.weights)
        thl.moe_combine_backward(self.dy, self.xs, self.rows, self.weights, self.dxs, self.dwt)
        thl.rmsnorm_backward(self.x, self.dy, self.w, self.dx, self.dw, eps=EPS)  # takes a workspace
        thl.gemm_w4(self.w4, self.y[:40], self.d, scales=self.scales, group=64, type_w="i4")  # takes a workspace
        thl.gemm_w4(self.w4, self.y[:1], self.d1, scales=self.scales, group=64, type_w="i4")

    def outputs(self):
        return [t.clone() for t in (self.y, self.rows, self.offsets, self.xs, self.out, self.dxs, self.dwt, self.dx,
                                    self.dw, self.d, self.d1)]

    def expected(self, seed):
        self.fill(seed)
        self.run()
        torch.cuda.synchronize()
        return self.outputs()


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_workspaces_are_taken():
    s = _Step(0)
    assert thl.thl_moe_sort_workspace(s.n, s.topk, s.experts) > 0
    assert thl.thl_rmsnorm_backward_workspace(s.m, s.n) > 0
    assert thl.thl_gemm_w4_workspace(260, 40, s.m) == 0 and thl.thl_gemm_w4_workspace(260, 40, 1024) > 0


def test_captured_and_replayed():
    s = _Step(0)
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


def test_two_graphs_at_once():
    a, b = _Step(1), _Step(2)
    want_a, want_b = a.expected(5), b.expected(6)
    graphs = []
    for s in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.run()
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(6):
        for s, graph, stream in zip((a, b), graphs, streams):
            with torch.cuda.stream(stream):
                s.out.zero_()
                graph.replay()
        torch.cuda.synchronize()
        assert _same(a.outputs(), want_a) and _same(b.outputs(), want_b)


def test_two_streams_at_once():
    a, b = _Step(3), _Step(4)
    want_a, want_b = a.expected(7), b.expected(8)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(6):
        for s, stream in zip((a, b), streams):
            with torch.cuda.stream(stream):
                for _ in range(2):
                    s.run()
        torch.cuda.synchronize()
        assert _same(a.outputs(), want_a) and _same(b.outputs(), want_b)


def test_long_codes_split_over_workgroups_captured():
    # K long enough for the 4-bit product to split: the splits' sums live in a workspace of the graph's
    g = torch.Generator().manual_seed(9)
    w = torch.randint(0, 256, (300, 4096), generator=g).to(torch.uint8).cuda()
    scales = torch.rand(300, 64, generator=g).bfloat16().cuda()
    x, d = torch.empty(33, 8192, dtype=torch.bfloat16, device="cuda"), torch.empty(33, 300, device="cuda")
    assert thl.thl_gemm_w4_workspace(300, 33, 8192) > 0

    def call():
        thl.gemm_w4(w, x, d, scales=scales, group=128, type_w="i4")

    want = []
    for i in range(3):
        x.copy_(torch.randn(33, 8192, generator=torch.Generator().manual_seed(i)))
        call()
        torch.cuda.synchronize()
        want.append(d.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in (2, 0, 1, 1):
        x.copy_(torch.randn(33, 8192, generator=torch.Generator().manual_seed(i)))
        d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want[i])


def test_inputs_made_on_the_calling_stream():
    # a side stream makes the inputs late; the call is ordered behind them
    s = _Step(5)
    want = s.expected(3)
    s.fill(4)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    h = torch.Generator().manual_seed(1003)
    x, dy = torch.randn(s.n, s.m, generator=h), torch.randn(s.n, s.m, generator=h)
    ids = torch.randint(0, s.experts, (s.n, s.topk), generator=h)
    xd, dyd, idd = x.cuda(), dy.cuda(), ids.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            big = big @ big * 1e-3
        s.x.copy_(xd)
        s.dy.copy_(dyd)
        s.ids.copy_(idd)
        s.run()
    torch.cuda.synchronize()
    assert _same(s.outputs(), want)

