"""Layer norm, MX quantization, the router and a layer of experts for a few tokens, as timed cases.

Five operators: the layer norm (centred, with weight and bias, the residual's
addition before it) and its gradient with the sums of dw and db; arrays
quantized to MX blocks along the features, along the tokens, or both in one
read, also with the product that reads them; the router's choice of experts
from its logits, with its gradient; and a whole mixture-of-experts layer for
a few tokens.

A token's features are contiguous: a (tokens, features) tensor here is the
library's column-major features x tokens matrix.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0, "e2m1": 6.0}  # largest finite values
EMAX = {"e4m3": 8, "e5m2": 15, "e2m1": 2}  # their exponents
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # by magnitude code
STEPS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # between them; ties go to the even code


def listed():
    return [
        # a decode batch of eight tokens, the residual stream's norm
        {"name": "norm_decode", "op": "norm", "n": 8, "m": 8192, "x": "bf16", "res": "bf16", "y": "bf16"},
        # a long prompt's
        {"name": "norm_prompt", "op": "norm", "n": 16384, "m": 4096, "x": "bf16", "res": "bf16", "y": "bf16"},
        # a training step's gradient, the residual branch's own gradient added
        {"name": "norm_grad", "op": "norm_grad", "n": 8192, "m": 4096, "x": "bf16", "g": "bf16", "dres": True},
        # a ragged batch of an odd width in fp32
        {"name": "norm_grad_ragged", "op": "norm_grad", "n": 777, "m": 1001, "x": "f32", "g": "f32", "dres": False},
        # a training step's activations as the fp4 operands of the forward product and of the weights' gradient
        {"name": "mx_both_ways", "op": "mx", "n": 8192, "m": 8192, "x": "bf16", "y": "e2m1", "rows": True,
         "cols": True, "out": 0},
        # a ragged batch of fp32 values to 8 bits
        {"name": "mx_ragged", "op": "mx", "n": 1531, "m": 5003, "x": "f32", "y": "e4m3", "rows": True, "cols": False,
         "out": 0},
        # a prompt through an fp4 projection: its activations quantized, then the product
        {"name": "mx_projection", "op": "mx", "n": 2048, "m": 8192, "x": "bf16", "y": "e2m1", "rows": True,
         "cols": False, "out": 8192},
        # a decode batch's choice of 8 of 128 experts
        {"name": "route_decode", "op": "route", "n": 16, "experts": 128, "topk": 8, "x": "bf16", "score": "softmax",
         "renorm": True, "grad": False},
        # a training step's, with the gradient
        {"name": "route_train", "op": "route", "n": 16384, "experts": 256, "topk": 8, "x": "f32", "score": "sigmoid",
         "renorm": True, "grad": True},
        # one token of a decode step: 8 of 128 experts on MX fp4 weights
        {"name": "experts_one_token", "op": "experts", "n": 1, "m": 4096, "h": 1024, "experts": 128, "topk": 8,
         "x": "bf16", "w": "e2m1", "gated": True, "act": "silu", "bias": False, "drop": 0.0},
        # a decode batch that reaches nearly all of the experts, 16 bits: the largest
        {"name": "experts_batch", "op": "experts", "n": 48, "m": 4096, "h": 1024, "experts": 64, "topk": 8,
         "x": "bf16", "w": "bf16", "gated": True, "act": "silu", "bias": False, "drop": 0.0},
        # fp16, odd sizes, biases, no gate; a tenth of the choices on experts held elsewhere
        {"name": "experts_ragged", "op": "experts", "n": 17, "m": 1001, "h": 333, "experts": 20, "topk": 3,
         "x": "f16", "w": "f16", "gated": False, "act": "gelu", "bias": True, "drop": 0.1},
    ]


def _size(rng, lo, hi, step=1):
    """A whole number of [lo, hi], even over its logarithm, a multiple of step half the time."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if step > 1 and rng.random() < 0.5:
        v = max(step, v // step * step)
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "mx", "route", "experts"])
    if op == "norm":
        m = _size(rng, 64, 16384, 64)
        x = rng.choice(["bf16", "bf16", "f16", "f32"])
        return {"op": op, "n": _size(rng, 1, max(1, min(16384, 16384 * 4096 // m))), "m": m, "x": x,
                "res": rng.choice(["none", x, "f32"]), "y": rng.choice(["bf16", "f16", "f32"])}
    if op == "norm_grad":
        m = _size(rng, 64, 16384, 64)
        return {"op": op, "n": _size(rng, 1, max(1, min(16384, 8192 * 4096 // m))), "m": m,
                "x": rng.choice(["bf16", "f16", "f32"]), "g": rng.choice(["bf16", "f32"]), "dres": rng.random() < 0.5}
    if op == "mx":
        ways = rng.choice([(True, False), (False, True), (True, True)])
        if rng.random() < 0.3:  # with the product, whose K is whole blocks
            return {"op": op, "n": _size(rng, 1, 2048), "m": 32 * _size(rng, 4, 256, 4), "x": rng.choice(["bf16", "f32"]),
                    "y": rng.choice(["e2m1", "e4m3"]), "rows": True, "cols": False, "out": _size(rng, 128, 8192, 128)}
        m = _size(rng, 32, 16384, 32)
        return {"op": op, "n": _size(rng, 1, max(1, min(16384, 8192 * 8192 // m)), 32), "m": m,
                "x": rng.choice(["bf16", "f16", "f32"]), "y": rng.choice(["e2m1", "e2m1", "e4m3", "e5m2"]),
                "rows": ways[0], "cols": ways[1], "out": 0}
    if op == "route":
        experts = _size(rng, 4, 512, 8)
        return {"op": op, "n": _size(rng, 1, 16384), "experts": experts, "topk": rng.choice([1, 2, 3, 4]),
                "x": rng.choice(["bf16", "f16", "f32"]), "score": rng.choice(["softmax", "sigmoid"]),
                "renorm": rng.random() < 0.6, "grad": rng.random() < 0.5}
    experts, topk = _size(rng, 4, 128, 4), rng.choice([1, 2, 3, 4])
    m = _size(rng, 64, 4096, 32)
    x = rng.choice(["bf16", "bf16", "f16"])
    return {"op": op, "n": rng.choice([1, 2, _size(rng, 3, 64)]), "m": m,
            "h": _size(rng, 48, max(48, min(4096, 64 * 1024 * 4096 // (experts * m))), 32), "experts": experts,
            "topk": topk, "x": x, "w": rng.choice([x, "e2m1", "e4m3"]), "gated": rng.random() < 0.7,
            "act": rng.choice(["silu", "gelu", "relu"]), "bias": rng.random() < 0.3, "drop": rng.choice([0.0, 0.0, 0.1])}


# ------------------------------------------------------------------ inputs

def _up(v, q):
    return -(-v // q) * q


def _randn(g, *shape, dtype="f32", scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(TORCH[dtype])


def _narrow(n, m, kind):
    """An empty array of n rows of m narrow values, rows of whole 16 bytes, as the matrix products like them."""
    if kind == "e2m1":
        return torch.zeros(n, _up(-(-m // 2), 16), dtype=torch.uint8, device=DEV)[:, :-(-m // 2)]
    return torch.zeros(n, _up(m, 16), dtype=torch.uint8, device=DEV)[:, :m].view(TORCH[kind])


def _scales(n, m):
    return torch.zeros(n, _up(-(-m // 32), 16), dtype=torch.uint8, device=DEV)


def _weights(g, kind, experts, rows, k):
    """The experts' matrices (rows of k), of about unit gain, with their block scales."""
    if kind in ("bf16", "f16"):
        w = torch.empty(experts, rows, k, dtype=TORCH[kind], device=DEV)
        for e in range(experts):
            w[e] = torch.randn(rows, k, generator=g, device=DEV) / math.sqrt(k)
        return w, None
    rms = 2.95 if kind == "e2m1" else 1.0  # of the elements
    mid = 127 - round(math.log2(rms * math.sqrt(k)))
    sf = torch.randint(mid - 1, mid + 2, (experts, rows, _up(-(-k // 32), 16)), generator=g, device=DEV).to(torch.uint8)
    if kind == "e2m1":
        return torch.randint(0, 256, (experts, rows, -(-k // 2)), generator=g, device=DEV).to(torch.uint8), sf
    w = torch.empty(experts, rows, k, dtype=TORCH[kind], device=DEV)
    for e in range(experts):
        w[e] = torch.randn(rows, k, generator=g, device=DEV).to(TORCH[kind])
    return w, sf


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s, op, n = {"case": c}, c["op"], c["n"]
    if op in ("norm", "norm_grad"):
        m = c["m"]
        vec = "f32" if c["x"] == "f32" else c["x"]
        s["w"] = (1.0 + 0.2 * _randn(g, m)).to(TORCH[vec])
        if op == "norm":
            # a residual stream: an offset, and a few features far larger than the rest
            s["x"] = (0.5 + _randn(g, n, m)).to(TORCH[c["x"]])
            big = 1.0 + 30.0 * (torch.rand(m, generator=g, device=DEV) < 0.005)
            s["res"] = None if c["res"] == "none" else (_randn(g, n, m, scale=2.0) * big).to(TORCH[c["res"]])
            s["sum"] = None if c["res"] == "none" else torch.empty_like(s["res"])
            s["b"] = _randn(g, m, dtype=vec, scale=0.1)
            s["y"] = torch.empty(n, m, dtype=TORCH[c["y"]], device=DEV)
        else:
            s["x"] = (0.5 + _randn(g, n, m, scale=2.0)).to(TORCH[c["x"]])
            s["dy"] = _randn(g, n, m, dtype=c["g"])
            s["dres"] = _randn(g, n, m, dtype=c["g"]) if c["dres"] else None
            s["dx"] = torch.empty(n, m, dtype=TORCH[c["g"]], device=DEV)
            s["dw"] = torch.empty(m, dtype=torch.float32, device=DEV)
            s["db"] = torch.empty(m, dtype=torch.float32, device=DEV)
    elif op == "mx":
        m = c["m"]
        # values of uneven size, as activations and gradients have
        s["x"] = (_randn(g, n, m) * torch.exp(_randn(g, n, 1)) * torch.exp(_randn(g, 1, m))).to(TORCH[c["x"]])
        s["y"] = _narrow(n, m, c["y"]) if c["rows"] else None
        s["sf"] = _scales(n, m) if c["rows"] else None
        s["y_t"] = _narrow(m, n, c["y"]) if c["cols"] else None
        s["sf_t"] = _scales(m, n) if c["cols"] else None
        if c["out"]:
            w, sf = _weights(g, c["y"], 1, c["out"], m)
            s["w"], s["sf_w"] = _narrow(c["out"], m, c["y"]), sf[0]
            s["w"].view(torch.uint8).copy_(w[0].view(torch.uint8))
            s["d"] = torch.empty(n, c["out"], dtype=torch.bfloat16, device=DEV)
    elif op == "route":
        experts, topk = c["experts"], c["topk"]
        # some experts more popular than others
        logits = 1.5 * _randn(g, n, experts) + 0.7 * _randn(g, experts)
        s["logits"] = logits.to(TORCH[c["x"]])
        s["ids"] = torch.empty(n, topk, dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(n, topk, dtype=torch.float32, device=DEV)
        s["dweights"] = _randn(g, n, topk)
        s["dlogits"] = torch.empty_like(s["logits"]) if c["grad"] else None
    else:
        m, h, experts, topk = c["m"], c["h"], c["experts"], c["topk"]
        up = 2 * h if c["gated"] else h
        s["x"] = _randn(g, n, m, dtype=c["x"])
        s["w1"], s["sf1"] = _weights(g, c["w"], experts, up, m)
        s["w2"], s["sf2"] = _weights(g, c["w"], experts, m, h)
        s["b1"] = _randn(g, experts, up, dtype=c["x"], scale=0.1) if c["bias"] else None
        s["b2"] = _randn(g, experts, m, dtype=c["x"], scale=0.1) if c["bias"] else None
        logits = _randn(g, n, experts) + 0.7 * _randn(g, experts)
        best = torch.topk(logits, topk, dim=1)
        gone = torch.rand(n, topk, generator=g, device=DEV) < c["drop"]
        s["ids"] = torch.where(gone, -1, best.indices).to(torch.int32)
        s["weights"] = torch.softmax(best.values, dim=1)
        s["y"] = torch.empty(n, m, dtype=TORCH[c["x"]], device=DEV)
    return s


# ------------------------------------------------------------------ plain forms

def _norm(s, f):
    v = s["x"].to(f) if s["res"] is None else s["x"].to(f) + s["res"].to(f)
    d = v - v.mean(dim=1, keepdim=True)
    return v, d * torch.rsqrt(d.square().mean(dim=1, keepdim=True) + EPS) * s["w"].to(f) + s["b"].to(f)


def _norm_grad(s, f):
    x, dy = s["x"].to(f), s["dy"].to(f)
    d = x - x.mean(dim=1, keepdim=True)
    r = torch.rsqrt(d.square().mean(dim=1, keepdim=True) + EPS)
    h = d * r
    t = dy * s["w"].to(f)
    dx = r * (t - t.mean(dim=1, keepdim=True) - h * (t * h).mean(dim=1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].to(f)
    return dx, (dy * h).sum(dim=0), dy.sum(dim=0)


def _mx(v, kind, y, sf):
    """v (n, m) in fp32 as MX blocks of 32 along m, laid out as y and sf, and the values that they stand for."""
    n, m = v.shape
    nb = -(-m // 32)
    b = torch.nn.functional.pad(v, (0, 32 * nb - m)).reshape(n, nb, 32)
    amax = b.abs().amax(dim=2)
    x = torch.clamp(torch.frexp(amax).exponent - 1 - EMAX[kind], -127, 127)
    code = torch.where(amax > 0, x + 127, 0)
    e = torch.ldexp(b, (127 - code)[:, :, None].to(b.dtype)).reshape(n, 32 * nb)[:, :m]
    scales = torch.zeros_like(sf)
    scales[:, :nb] = code.to(torch.uint8)
    if kind == "e2m1":
        a = torch.clamp(e.abs(), max=6.0)
        low = (a > STEPS[0]).int() + (a > STEPS[2]) + (a > STEPS[4]) + (a > STEPS[6])
        codes = low + (a >= STEPS[1]) + (a >= STEPS[3]) + (a >= STEPS[5])
        codes = torch.nn.functional.pad(codes + 8 * torch.signbit(e), (0, m % 2)).to(torch.uint8)
        q = codes[:, 0::2] | (codes[:, 1::2] << 4)
        values = torch.tensor(E2M1, device=DEV)[(codes & 7).int()][:, :m] * torch.where(torch.signbit(e), -1.0, 1.0)
    else:
        q = torch.clamp(e, -TOP[kind], TOP[kind]).to(TORCH[kind])
        values = q.float()
    out = torch.zeros_like(y.view(torch.uint8)).view(y.dtype)
    out.view(torch.uint8).copy_(q.view(torch.uint8))
    scale = torch.ldexp(torch.ones((), device=DEV), code.float() - 127).repeat_interleave(32, dim=1)[:, :m]
    return out, scales, values * scale


def _values(w, sf, kind, k, f):
    """The values of weights (..., k) as stored, in f."""
    if sf is None:
        return w.to(f)
    if kind == "e2m1":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=f, device=DEV)
        codes = torch.stack([w & 15, w >> 4], dim=-1).reshape(*w.shape[:-1], 2 * w.shape[-1])[..., :k]
        v = table[codes.int()]
    else:
        v = w.to(f)
    scale = torch.ldexp(torch.ones((), dtype=f, device=DEV), sf.to(f) - 127)[..., :-(-k // 32)]
    return v * scale.repeat_interleave(32, dim=-1)[..., :k]


def _act(v, act):
    if act == "relu":
        return torch.clamp(v, min=0.0)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return 0.5 * v * (1.0 + torch.erf(v / math.sqrt(2.0)))


def _score(logits, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _route(s, f):
    c, logits = s["case"], s["logits"].to(f)
    # the largest first, the lowest index first among equals
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :c["topk"]]
    score = _score(logits, c["score"])
    chosen = torch.gather(score, 1, ids)
    total = chosen.sum(dim=1, keepdim=True)
    weights = chosen / total if c["renorm"] else chosen
    if not c["grad"]:
        return ids, weights, None
    dw = s["dweights"].to(f)
    if c["renorm"]:
        dw = (dw - (dw * weights).sum(dim=1, keepdim=True)) / total
    dscore = torch.zeros_like(score).scatter(1, ids, dw)
    if c["score"] == "sigmoid":
        return ids, weights, dscore * score * (1.0 - score)
    return ids, weights, score * (dscore - (dscore * score).sum(dim=1, keepdim=True))


def _experts(s, f):
    c, x, ids = s["case"], s["x"].to(f), s["ids"].long()
    n, m, h, topk = c["n"], c["m"], c["h"], c["topk"]
    live = ids >= 0
    wt = torch.where(live, s["weights"].to(f), 0.0)
    few = n * topk < c["experts"]  # each choice's own matrices, or every expert on every token
    pick = (lambda a: None if a is None else a[ids.clamp(min=0).reshape(-1)]) if few else (lambda a: a)
    w1 = _values(pick(s["w1"]), pick(s["sf1"]), c["w"], m, f)
    b1, b2 = pick(s["b1"]), pick(s["b2"])
    if few:
        at = x.repeat_interleave(topk, dim=0)[:, :, None].contiguous()  # (choices, m, 1)
    else:
        at = x.t().contiguous()[None].expand(c["experts"], m, n).contiguous()  # (experts, m, n)
    u = torch.bmm(w1, at)
    del w1
    if b1 is not None:
        u = u + b1.to(f)[:, :, None]
    u = _act(u[:, :h], c["act"]) * u[:, h:] if c["gated"] else _act(u, c["act"])
    z = torch.bmm(_values(pick(s["w2"]), pick(s["sf2"]), c["w"], h, f), u.contiguous())
    if b2 is not None:
        z = z + b2.to(f)[:, :, None]
    if few:
        return (z.reshape(n, topk, m) * wt[:, :, None]).sum(dim=1)
    share = (wt[:, :, None] * (ids[:, :, None] == torch.arange(c["experts"], device=DEV))).sum(dim=1)  # (n, experts)
    return (z * share.t()[:, None, :]).sum(dim=0).t()


def _plain(s):
    c, f = s["case"], torch.float32
    op = c["op"]
    if op == "norm":
        v, y = _norm(s, f)
        return None if s["res"] is None else v.to(s["res"].dtype), y.to(TORCH[c["y"]])
    if op == "norm_grad":
        dx, dw, db = _norm_grad(s, f)
        return dx.to(s["dx"].dtype), dw, db
    if op == "mx":
        x, y, sf, y_t, sf_t, d = s["x"].to(f), None, None, None, None, None
        if c["rows"]:
            y, sf, values = _mx(x, c["y"], s["y"], s["sf"])
        if c["cols"]:
            y_t, sf_t, _ = _mx(x.t().contiguous(), c["y"], s["y_t"], s["sf_t"])
        if c["out"]:
            d = (values @ _values(s["w"], s["sf_w"], c["y"], c["m"], f).t()).to(torch.bfloat16)
        return y, sf, y_t, sf_t, d
    if op == "route":
        ids, weights, dlogits = _route(s, f)
        return ids.to(torch.int32), weights, None if dlogits is None else dlogits.to(s["logits"].dtype)
    return _experts(s, f).to(s["y"].dtype).contiguous()


# ------------------------------------------------------------------ the framework's kernels

def _kernels(s):
    import tile_hierarchy_linear_amd as thl

    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        thl.layernorm(s["x"], s["w"], s["b"], s["y"], eps=EPS, residual=s["res"], residual_out=s["sum"])
        return s["sum"], s["y"]
    if op == "norm_grad":
        thl.layernorm_backward(s["x"], s["dy"], s["w"], s["dx"], s["dw"], s["db"], eps=EPS, dres=s["dres"])
        return s["dx"], s["dw"], s["db"]
    if op == "mx":
        thl.mx_quantize(s["x"], s["y"], s["sf"], y_t=s["y_t"], sf_t=s["sf_t"])
        if c["out"]:
            codes = 2 if c["y"] == "e2m1" else 1  # a byte
            thl.gemm(s["w"], s["y"], s["d"], m=c["out"], n=c["n"], k=c["m"], lda=codes * s["w"].stride(0),
                     ldb=codes * s["y"].stride(0), ldd=c["out"], op_a="T", op_b="N", type_ab=c["y"], type_d="bf16",
                     sfa=s["sf_w"], ld_sfa=s["sf_w"].stride(0), sfb=s["sf"], ld_sfb=s["sf"].stride(0))
            return s["y"], s["sf"], s["y_t"], s["sf_t"], s["d"]
        return s["y"], s["sf"], s["y_t"], s["sf_t"], None
    if op == "route":
        thl.moe_route(s["logits"], s["ids"], s["weights"], score=c["score"], renormalize=c["renorm"])
        if c["grad"]:
            thl.moe_route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"], score=c["score"],
                                   renormalize=c["renorm"])
        return s["ids"], s["weights"], s["dlogits"]
    thl.moe_layer(s["x"], s["ids"], s["weights"], s["w1"], s["w2"], s["y"], gated=c["gated"], act=c["act"],
                  sf1=s["sf1"], sf2=s["sf2"], b1=s["b1"], b2=s["b2"])
    return s["y"]


def run(state):
    """One pass.  MX codes and block scales come as stored: two 4-bit codes a byte are whole numbers, to be equal."""
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits, and the work

def exact(case, seed):
    """From the definitions, in fp64.  None for what has no value but itself (sums of bits, codes, choices)."""
    s, d = prepare(case, seed), torch.float64
    c, op, n = s["case"], s["case"]["op"], case["n"]
    if op == "norm":
        x = s["x"].to(d)
        if s["res"] is not None:
            x += s["res"].to(d)
        mu = x.sum(dim=1, keepdim=True) / c["m"]
        var = (x * x).sum(dim=1, keepdim=True) / c["m"] - mu * mu
        y = (x - mu) / torch.sqrt(var + EPS) * s["w"].to(d) + s["b"].to(d)
        return None if s["res"] is None else x, y
    if op == "norm_grad":
        x, dy, w, m = s["x"].to(d), s["dy"].to(d), s["w"].to(d), c["m"]
        mu = x.sum(dim=1, keepdim=True) / m
        sigma = torch.sqrt((x * x).sum(dim=1, keepdim=True) / m - mu * mu + EPS)
        h = (x - mu) / sigma
        # dx_i = sum_k w_k dy_k dh_k/dx_i, with dh_k/dx_i = ([i = k] - 1/m - h_i h_k / m) / sigma
        along, level = ((dy * w) * h).sum(dim=1, keepdim=True), (dy * w).sum(dim=1, keepdim=True)
        dx = (dy * w - level / m - h * along / m) / sigma
        if s["dres"] is not None:
            dx += s["dres"].to(d)
        return dx, (dy * h).sum(dim=0), dy.sum(dim=0)
    if op == "mx":
        kind, m = c["y"], c["m"]

        def blocks(v):  # the elements in 8 bits (division by a power of two is exact), and what the blocks stand for
            block = torch.arange(v.shape[1], device=DEV) // 32
            amax = torch.zeros(v.shape[0], -(-v.shape[1] // 32), dtype=d, device=DEV)
            amax.scatter_reduce_(1, block.expand(v.shape), v.abs(), "amax")
            e = torch.clamp(torch.floor(torch.log2(amax)) - EMAX[kind], -127, 127)
            scale = torch.pow(2.0, torch.where(amax > 0, e, -127))[:, block]
            q = torch.clamp(v / scale, -TOP[kind], TOP[kind])
            if kind == "e2m1":
                grid = torch.tensor([-v for v in E2M1[:0:-1]] + list(E2M1), dtype=d, device=DEV)
                hi = torch.searchsorted(grid, q.contiguous()).clamp(1, 14)
                below, above = q - grid[hi - 1], grid[hi] - q
                # the even code of two as near: every second of the grid, zero among them
                up = (above < below) | ((above == below) & ((hi - 7) % 2 == 0))
                return None, torch.where(up, grid[hi], grid[hi - 1]) * scale
            q = q.to(TORCH[kind]).to(d)
            return q, q * scale

        x = s["x"].to(d)
        y, values = blocks(x) if c["rows"] else (None, None)
        y_t = blocks(x.t().contiguous())[0] if c["cols"] else None
        if not c["out"]:
            return None if kind == "e2m1" else (y, None, y_t, None, None)
        w = s["w"]
        if kind == "e2m1":
            table = torch.tensor(list(E2M1) + [-v for v in E2M1], dtype=d, device=DEV)
            w = torch.stack([table[(w & 15).long()], table[(w >> 4).long()]], dim=2).reshape(c["out"], -1)[:, :m]
        w = w.to(d) * torch.pow(2.0, s["sf_w"].to(d) - 127)[:, torch.arange(m, device=DEV) // 32]
        return y, None, y_t, None, values @ w.t()
    if op == "route":
        logits, topk = s["logits"].to(d), c["topk"]
        rest, ids = logits.clone(), []
        for _ in range(topk):
            best = rest.max(dim=1, keepdim=True).values
            at = (rest == best).to(torch.int8).argmax(dim=1, keepdim=True)
            ids.append(at)
            rest.scatter_(1, at, -math.inf)
        ids = torch.cat(ids, dim=1)
        p = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.softmax(logits, dim=1)
        chosen = p.gather(1, ids)
        total = chosen.sum(dim=1, keepdim=True) if c["renorm"] else torch.ones(n, 1, dtype=d, device=DEV)
        weights = chosen / total
        if not c["grad"]:
            return None, weights, None
        leaf = logits.clone().requires_grad_()
        with torch.enable_grad():
            q = torch.sigmoid(leaf) if c["score"] == "sigmoid" else torch.softmax(leaf, dim=1)
            q = q.gather(1, ids)
            q = q / q.sum(dim=1, keepdim=True) if c["renorm"] else q
            (q * s["dweights"].to(d)).sum().backward()
        return None, weights, leaf.grad
    m, h = c["m"], c["h"]
    y = torch.zeros(n, m, dtype=d, device=DEV)
    ids, wt, x = s["ids"].tolist(), s["weights"].to(d), s["x"].to(d)

    def matrix(w, sf, k):
        if sf is None:
            return w.to(d)
        if c["w"] == "e2m1":
            table = torch.tensor(list(E2M1) + [-v for v in E2M1], dtype=d, device=DEV)
            w = torch.stack([table[(w & 15).long()], table[(w >> 4).long()]], dim=2).reshape(w.shape[0], -1)[:, :k]
        return w.to(d) * torch.pow(2.0, sf.to(d) - 127)[:, torch.arange(k, device=DEV) // 32]

    for e in range(c["experts"]):
        mine = [(j, t) for j in range(n) for t in range(c["topk"]) if ids[j][t] == e]
        if not mine:
            continue
        j, t = (torch.tensor(v, device=DEV) for v in zip(*mine))
        u = x[j] @ matrix(s["w1"][e], None if s["sf1"] is None else s["sf1"][e], m).t()
        if s["b1"] is not None:
            u = u + s["b1"][e].to(d)
        gate = u[:, :h]
        gate = {"relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[c["act"]](gate)
        u = gate * u[:, h:] if c["gated"] else gate
        z = u @ matrix(s["w2"][e], None if s["sf2"] is None else s["sf2"][e], h).t()
        if s["b2"] is not None:
            z = z + s["b2"][e].to(d)
        y.index_add_(0, j, z * wt[j, t][:, None])
    return y


def work(case):
    c, op, n = case, case["op"], case["n"]
    size = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "e5m2": 1, "e2m1": 0.5}
    if op == "norm":
        m = c["m"]
        b = n * m * (size[c["x"]] + size[c["y"]]) + 2 * m * size[c["x"]]
        if c["res"] != "none":
            b += 2 * n * m * size[c["res"]]
        return {"bytes": b, "flops": 8 * n * m}
    if op == "norm_grad":
        m = c["m"]
        return {"bytes": n * m * (size[c["x"]] + size[c["g"]] * (3 if c["dres"] else 2)) + m * (size[c["x"]] + 8),
                "flops": 14 * n * m}
    if op == "mx":
        m, q = c["m"], size[c["y"]] + 1 / 32
        b, out = n * m * size[c["x"]] + n * m * q * (c["rows"] + c["cols"]), c["out"]
        return {"bytes": b + out * m * q + 2 * n * out, "flops": 3 * n * m + 2 * n * m * out}
    if op == "route":
        b = n * c["experts"] * size[c["x"]] + 8 * n * c["topk"]
        if c["grad"]:
            b += 2 * n * c["experts"] * size[c["x"]] + 8 * n * c["topk"]
        return {"bytes": b, "flops": 10 * n * c["experts"]}
    m, h, experts, choices = c["m"], c["h"], c["experts"], n * c["topk"] * (1.0 - c["drop"])
    # experts that any token reaches, were they chosen evenly
    reached = experts * (1.0 - (1.0 - c["topk"] * (1.0 - c["drop"]) / experts) ** n)
    each = (3 if c["gated"] else 2) * m * h
    q = size[c["w"]] + (1 / 32 if c["w"] in EMAX else 0)
    return {"bytes": reached * each * q + 2 * n * m * size[c["x"]] + 8 * n * c["topk"], "flops": 2 * choices * each}
