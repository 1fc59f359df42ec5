"""The operators around a transformer layer's matrix products, as timed cases.

Four operators: the root-mean-square norm with the residual's addition and
an output in 16 or 8 bits (the operand of the next product), and its
gradient; tokens sorted by expert with their rows copied into expert order
(the operands of a grouped product); the experts' rows weighted and added
back per token, and its gradient; and the product of a few tokens with a
matrix of 4-bit weights under group scales.

A token's features are contiguous: a (tokens, features) tensor here is the
library's column-major features x tokens matrix.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}  # largest finite values
EMAX = {"e4m3": 8, "e5m2": 15}  # their exponents
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # by magnitude code


def listed():
    return [
        # one token of a decode step: the residual stream's norm before an MX product
        {"name": "norm_one_token", "op": "norm", "n": 1, "m": 8192, "x": "bf16", "res": "bf16", "y": "mx_e4m3"},
        # a long prompt's norm, 16 bits throughout: the largest
        {"name": "norm_prompt", "op": "norm", "n": 16384, "m": 8192, "x": "bf16", "res": "bf16", "y": "bf16"},
        # a ragged batch and an odd width, an fp32 residual stream, one scale for the whole tensor
        {"name": "norm_ragged", "op": "norm", "n": 1531, "m": 5003, "x": "f16", "res": "f32", "y": "e4m3"},
        # a training step's gradient, the residual branch's own gradient added
        {"name": "norm_grad", "op": "norm_grad", "n": 8192, "m": 4096, "x": "bf16", "g": "bf16", "dres": True},
        # a ragged batch in fp32
        {"name": "norm_grad_ragged", "op": "norm_grad", "n": 777, "m": 1001, "x": "f32", "g": "f32", "dres": False},
        # a decode batch: 24 tokens to 8 of 128 experts, MX rows with their block scales
        {"name": "dispatch_decode", "op": "dispatch", "n": 24, "topk": 8, "experts": 128, "m": 4096, "x": "mx_e4m3",
         "drop": 0.0},
        # a prompt: 16-bit rows, a few choices dropped for capacity
        {"name": "dispatch_prompt", "op": "dispatch", "n": 8192, "topk": 8, "experts": 64, "m": 4096, "x": "bf16",
         "drop": 0.02},
        # the same prompt's way back
        {"name": "combine_prompt", "op": "combine", "n": 8192, "topk": 8, "m": 4096, "x": "bf16", "y": "bf16",
         "drop": 0.02},
        # its gradient in a training step with two experts a token, a width off 8
        {"name": "combine_grad", "op": "combine_grad", "n": 4096, "topk": 2, "m": 5126, "x": "bf16", "drop": 0.0},
        # one token, a square projection: codes with zero points, fp16
        {"name": "w4_one_token", "op": "w4", "n": 1, "m": 4096, "k": 4096, "w": "u4", "group": 128, "x": "f16",
         "bias": False},
        # one token, a wide projection: signed codes, bf16
        {"name": "w4_wide", "op": "w4", "n": 1, "m": 28672, "k": 8192, "w": "i4", "group": 128, "x": "bf16",
         "bias": False},
        # a decode batch on MX fp4 weights
        {"name": "w4_batch", "op": "w4", "n": 48, "m": 8192, "k": 8192, "w": "e2m1", "group": 32, "x": "bf16",
         "bias": True},
    ]


def _size(rng, lo, hi, step=1):
    """A whole number of [lo, hi], even over its logarithm, a multiple of step half the time."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if step > 1 and rng.random() < 0.5:
        v = max(step, v // step * step)
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "dispatch", "combine", "combine_grad", "w4"])
    if op == "norm":
        m = _size(rng, 64, 16384, 64)
        n = _size(rng, 1, max(1, min(16384, 16384 * 8192 // m)))
        x = rng.choice(["bf16", "bf16", "f16", "f32"])
        return {"op": op, "n": n, "m": m, "x": x, "res": rng.choice(["none", x, "f32"]),
                "y": rng.choice(["bf16", "f16", "f32", "e4m3", "e5m2", "mx_e4m3", "mx_e5m2"])}
    if op == "norm_grad":
        m = _size(rng, 64, 16384, 64)
        return {"op": op, "n": _size(rng, 1, max(1, min(16384, 8192 * 4096 // m))), "m": m,
                "x": rng.choice(["bf16", "f16", "f32"]), "g": rng.choice(["bf16", "f32"]), "dres": rng.random() < 0.5}
    if op == "w4":
        k = 32 * _size(rng, 4, 512, 4)
        n = rng.choice([1, 1, 2, _size(rng, 3, 64)])
        m = _size(rng, 256, min(28672, 28672 * 8192 // (k * (2 if n > 16 else 1))), 16)
        w = rng.choice(["u4", "i4", "e2m1"])
        return {"op": op, "n": n, "m": m, "k": k, "w": w, "group": 32 if w == "e2m1" else rng.choice([32, 64, 128]),
                "x": rng.choice(["bf16", "f16"]), "bias": rng.random() < 0.5}
    topk = rng.choice([1, 2, 3, 4, 6, 8])
    m = _size(rng, 128, 8192, 128)
    n = _size(rng, 1, max(1, min(16384, 8192 * 8 * 4096 // (topk * m))))
    drop = rng.choice([0.0, 0.0, 0.05])
    if op == "dispatch":
        return {"op": op, "n": n, "topk": topk, "experts": _size(rng, max(8, topk), 256), "m": m,
                "x": rng.choice(["bf16", "f32", "mx_e4m3", "mx_e5m2"]), "drop": drop}
    x = rng.choice(["bf16", "f16", "f32"])
    if op == "combine":
        return {"op": op, "n": n, "topk": topk, "m": m, "x": x, "y": rng.choice([x, "f32"]), "drop": drop}
    return {"op": op, "n": n, "topk": topk, "m": m, "x": x, "drop": drop}


# ------------------------------------------------------------------ inputs

def _up(v, q):
    return -(-v // q) * q


def _randn(g, *shape, dtype="f32", scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(TORCH[dtype])


def _ids(g, n, topk, experts, drop):
    """Each token's topk experts, the strongest first, some experts more popular than others; -1: dropped."""
    logits = torch.randn(n, experts, generator=g, device=DEV)
    logits += 0.7 * torch.randn(experts, generator=g, device=DEV)
    ids = torch.topk(logits, topk, dim=1).indices
    if drop:
        ids = torch.where(torch.rand(n, topk, generator=g, device=DEV) < drop, -1, ids)
    return ids


def _mx(fmt):
    return fmt[3:] if fmt.startswith("mx_") else None


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s, op, n, m = {"case": c}, c["op"], c["n"], c["m"]
    if op == "norm":
        s["x"] = _randn(g, n, m, dtype=c["x"])
        # a residual stream has a few features far larger than the rest
        big = 1.0 + 30.0 * (torch.rand(m, generator=g, device=DEV) < 0.005)
        s["res"] = None if c["res"] == "none" else (_randn(g, n, m, scale=2.0) * big).to(TORCH[c["res"]])
        s["sum"] = None if c["res"] == "none" else torch.empty_like(s["res"])
        s["w"] = (1.0 + 0.2 * _randn(g, m)).to(TORCH["f32" if c["x"] == "f32" else c["x"]])
        kind = _mx(c["y"]) or c["y"]
        # 8-bit rows are pitched in whole 16-byte units, as the matrix products like them
        pitch = _up(m, 16) if kind in TOP else m
        s["y"] = torch.zeros(n, pitch, dtype=torch.uint8 if kind in TOP else TORCH[kind], device=DEV)[:, :m]
        if kind in TOP:
            s["y"] = s["y"].view(TORCH[kind])
        s["sf"] = torch.zeros(n, _up(-(-m // 32), 16), dtype=torch.uint8, device=DEV) if _mx(c["y"]) else None
        s["scale"] = 0.02 if kind == "e4m3" else 0.001  # one scale for the whole tensor, found beforehand
    elif op == "norm_grad":
        s["x"] = _randn(g, n, m, dtype=c["x"], scale=2.0)
        s["dy"] = _randn(g, n, m, dtype=c["g"])
        s["dres"] = _randn(g, n, m, dtype=c["g"]) if c["dres"] else None
        s["w"] = (1.0 + 0.2 * _randn(g, m)).to(TORCH["f32" if c["x"] == "f32" else c["x"]])
        s["dx"] = torch.empty(n, m, dtype=TORCH[c["g"]], device=DEV)
        s["dw"] = torch.empty(m, dtype=torch.float32, device=DEV)
    elif op == "dispatch":
        topk = c["topk"]
        s["ids"] = _ids(g, n, topk, c["experts"], c["drop"])
        kind = _mx(c["x"])
        if kind:
            s["x"] = torch.randn(n, _up(m, 16), generator=g, device=DEV).mul_(100.0).to(TORCH[kind])[:, :m]
            s["sf"] = torch.randint(100, 130, (n, _up(-(-m // 32), 16)), generator=g, device=DEV).to(torch.uint8)
            s["y"] = torch.zeros(n * topk, _up(m, 16), dtype=torch.uint8, device=DEV)[:, :m].view(TORCH[kind])
            s["sf_y"] = torch.zeros(n * topk, s["sf"].shape[1], dtype=torch.uint8, device=DEV)
        else:
            s["x"] = _randn(g, n, m, dtype=c["x"])
            s["y"] = torch.zeros(n * topk, m, dtype=TORCH[c["x"]], device=DEV)
            s["sf"] = s["sf_y"] = None
        s["rows"] = torch.empty(n, topk, dtype=torch.int32, device=DEV)
        s["offsets"] = torch.empty(c["experts"] + 1, dtype=torch.int32, device=DEV)
        s["order"] = torch.full((n * topk,), -1, dtype=torch.int32, device=DEV)
    elif op in ("combine", "combine_grad"):
        topk = c["topk"]
        ids = _ids(g, n, topk, 64 if topk > 2 else 8, c["drop"])
        # where each choice's row lies after a stable sort by expert, the dropped ones (-1) left out
        flat = ids.reshape(-1)
        place = torch.argsort(torch.where(flat < 0, 1 << 30, flat), stable=True)
        rows = torch.empty_like(place)
        rows[place] = torch.arange(n * topk, device=DEV)
        s["rows"] = torch.where(flat < 0, -1, rows).to(torch.int32).reshape(n, topk)
        s["x"] = _randn(g, n * topk, m, dtype=c["x"])
        s["weights"] = torch.softmax(torch.randn(n, topk, generator=g, device=DEV), dim=1)
        if op == "combine":
            s["y"] = torch.empty(n, m, dtype=TORCH[c["y"]], device=DEV)
        else:
            s["dy"] = _randn(g, n, m, dtype=c["x"])
            s["dx"] = torch.zeros(n * topk, m, dtype=TORCH[c["x"]], device=DEV)
            s["dweights"] = torch.empty(n, topk, dtype=torch.float32, device=DEV)
    else:
        k, groups = c["k"], -(-c["k"] // c["group"])
        s["w"] = torch.randint(0, 256, (m, k // 2), generator=g, device=DEV).to(torch.uint8)
        s["x"] = _randn(g, n, k, dtype=c["x"])
        s["zeros"] = None
        if c["w"] == "e2m1":
            s["scales"] = torch.randint(116, 124, (m, groups), generator=g, device=DEV).to(torch.uint8)
        else:
            s["scales"] = (0.005 + 0.01 * torch.rand(m, groups, generator=g, device=DEV)).to(TORCH[c["x"]])
            if c["w"] == "u4":
                s["zeros"] = torch.randint(4, 12, (m, groups), generator=g, device=DEV).to(torch.uint8)
        s["bias"] = _randn(g, m, dtype=c["x"]) if c["bias"] else None
        s["d"] = torch.empty(n, m, dtype=TORCH[c["x"]], device=DEV)
    return s


# ------------------------------------------------------------------ plain forms

def _blocks(v, kind):
    """v (n, m) as MX blocks of 32: the elements before rounding, and the E8M0 scale codes."""
    n, m = v.shape
    nb = -(-m // 32)
    b = torch.nn.functional.pad(v, (0, 32 * nb - m)).reshape(n, nb, 32)
    amax = b.abs().amax(dim=2)
    x = torch.clamp(torch.frexp(amax).exponent - 1 - EMAX[kind], -127, 127)
    code = torch.where(amax > 0, x + 127, 0)
    e = torch.ldexp(b, (127 - code)[:, :, None].to(b.dtype))
    return torch.clamp(e, -TOP[kind], TOP[kind]).reshape(n, 32 * nb)[:, :m], code.to(torch.uint8)


def _norm(s, f):
    """The norm in the floating type f: (x + residual, the normalised rows)."""
    v = s["x"].to(f) if s["res"] is None else s["x"].to(f) + s["res"].to(f)
    return v, v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS) * s["w"].to(f)


def _norm_grad(s, f):
    x, dy, w = s["x"].to(f), s["dy"].to(f), s["w"].to(f)
    r = torch.rsqrt(x.square().mean(dim=1, keepdim=True) + EPS)
    h = x * r
    t = dy * w
    dx = r * (t - h * (t * h).mean(dim=1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].to(f)
    return dx, (dy * h).sum(dim=0)


def _combine(s, f):
    rows = s["rows"].long()
    w = torch.where(rows < 0, 0.0, s["weights"]).to(f)
    return (s["x"].to(f)[rows.clamp(min=0)] * w[:, :, None]).sum(dim=1)


def _combine_grad(s, f):
    rows, dy = s["rows"].long(), s["dy"].to(f)
    kept = rows >= 0
    dots = (s["x"].to(f)[rows.clamp(min=0)] * dy[:, None, :]).sum(dim=2)
    token = torch.arange(rows.shape[0], device=DEV)[:, None].expand_as(rows)
    return rows[kept], dy[token[kept]] * s["weights"].to(f)[kept][:, None], torch.where(kept, dots, 0.0)


def _w4(s, f):
    c, w = s["case"], s["w"]
    m, half = w.shape
    codes = torch.stack([w & 15, w >> 4], dim=2).reshape(m, 2 * half)
    if c["w"] == "e2m1":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=f, device=DEV)
        v = table[codes.int()]
        scales = torch.ldexp(torch.ones((), dtype=f, device=DEV), s["scales"].to(f) - 127)
        zeros = None
    else:
        v = codes.to(f)
        if c["w"] == "i4":
            v = torch.where(v >= 8, v - 16, v)
        scales, zeros = s["scales"].to(f), s["zeros"]
    groups = scales.shape[1]
    pad = groups * c["group"] - c["k"]
    v = torch.nn.functional.pad(v, (0, pad)).reshape(m, groups, c["group"])
    if zeros is not None:
        v = v - zeros.to(f)[:, :, None]
    v = (v * scales[:, :, None]).reshape(m, groups * c["group"])[:, :c["k"]]
    y = s["x"].to(f) @ v.t()
    return y if s["bias"] is None else y + s["bias"].to(f)


def _plain(s):
    c, f = s["case"], torch.float32
    op = c["op"]
    if op == "norm":
        v, y = _norm(s, f)
        total = None if s["res"] is None else v.to(s["res"].dtype)
        kind = _mx(c["y"])
        if kind:
            y, code = _blocks(y, kind)
            sf = s["sf"].clone()
            sf[:, :code.shape[1]] = code
            return total, y.to(TORCH[kind]), sf.view(torch.float8_e8m0fnu)
        if c["y"] in TOP:
            y = torch.clamp(y / s["scale"], -TOP[c["y"]], TOP[c["y"]])
        return total, y.to(TORCH[c["y"]])
    if op == "norm_grad":
        dx, dw = _norm_grad(s, f)
        return dx.to(s["dx"].dtype), dw
    if op == "dispatch":
        flat = s["ids"].reshape(-1)
        kept = flat >= 0
        place = torch.argsort(torch.where(kept, flat, 1 << 30), stable=True)
        inverse = torch.empty_like(place)
        inverse[place] = torch.arange(flat.numel(), device=DEV)
        rows = torch.where(kept, inverse, -1).to(torch.int32).reshape(s["ids"].shape)
        counts = (flat[:, None] == torch.arange(c["experts"], device=DEV)).sum(dim=0)
        offsets = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)]).to(torch.int32)
        live = torch.arange(flat.numel(), device=DEV) < offsets[-1]
        order = torch.where(live, place, s["order"].long()).to(torch.int32)
        token = place // c["topk"]
        bits = s["x"].view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[s["x"].element_size()])
        y = torch.where(live[:, None], bits[token], 0).view(s["x"].dtype)
        if s["sf"] is None:
            return rows, offsets, order, y
        sf = torch.zeros_like(s["sf_y"])
        nb = -(-c["m"] // 32)
        sf[:, :nb] = torch.where(live[:, None], s["sf"][token, :nb], 0)
        return rows, offsets, order, y, sf.view(torch.float8_e8m0fnu)
    if op == "combine":
        return _combine(s, f).to(s["y"].dtype)
    if op == "combine_grad":
        at, values, dweights = _combine_grad(s, f)
        dx = torch.zeros_like(s["dx"])
        dx[at] = values.to(dx.dtype)
        return dx, dweights
    return _w4(s, f).to(s["d"].dtype)


# ------------------------------------------------------------------ the framework's kernels

def _kernels(s):
    import tile_hierarchy_linear_amd as thl

    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        thl.rmsnorm(s["x"], s["w"], s["y"], eps=EPS, residual=s["res"], residual_out=s["sum"],
                    scale=s["scale"] if c["y"] in TOP else 1.0, sf=s["sf"])
        if s["sf"] is None:
            return s["sum"], s["y"]
        return s["sum"], s["y"], s["sf"].view(torch.float8_e8m0fnu)
    if op == "norm_grad":
        thl.rmsnorm_backward(s["x"], s["dy"], s["w"], s["dx"], s["dw"], eps=EPS, dres=s["dres"])
        return s["dx"], s["dw"]
    if op == "dispatch":
        thl.moe_sort(s["ids"], c["experts"], s["rows"], s["offsets"], order=s["order"])
        thl.moe_gather(s["x"], s["rows"], s["y"], sf=s["sf"], sf_y=s["sf_y"])
        if s["sf"] is None:
            return s["rows"], s["offsets"], s["order"], s["y"]
        return s["rows"], s["offsets"], s["order"], s["y"], s["sf_y"].view(torch.float8_e8m0fnu)
    if op == "combine":
        thl.moe_combine(s["x"], s["rows"], s["y"], weights=s["weights"])
        return s["y"]
    if op == "combine_grad":
        thl.moe_combine_backward(s["dy"], s["x"], s["rows"], s["weights"], s["dx"], s["dweights"])
        return s["dx"], s["dweights"]
    thl.gemm_w4(s["w"], s["x"], s["d"], type_w=c["w"], scales=s["scales"], group=c["group"], zeros=s["zeros"],
                bias=s["bias"])
    return s["d"]


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits, and the work

def exact(case, seed):
    """From the definitions, in fp64.  None for block scales and copied bits (no computed numbers there)."""
    s, d = prepare(case, seed), torch.float64
    c, op = s["case"], s["case"]["op"]
    n, m = c["n"], c["m"]
    if op == "norm":
        x = s["x"].to(d)
        if s["res"] is not None:
            x += s["res"].to(d)
        y = x / torch.sqrt((x * x).sum(dim=1, keepdim=True) / m + EPS) * s["w"].to(d)
        total = None if s["res"] is None else x
        kind = _mx(c["y"])
        if not kind:
            return total, torch.clamp(y / s["scale"], -TOP[c["y"]], TOP[c["y"]]) if c["y"] in TOP else y
        block = torch.arange(m, device=DEV) // 32
        amax = torch.zeros(n, -(-m // 32), dtype=d, device=DEV)
        amax.scatter_reduce_(1, block.expand(n, m), y.abs(), "amax")
        e = torch.clamp(torch.floor(torch.log2(amax)) - EMAX[kind], -127, 127)
        return total, torch.clamp(y / torch.pow(2.0, e)[:, block], -TOP[kind], TOP[kind]), None
    if op == "norm_grad":
        x, dy, w = s["x"].to(d), s["dy"].to(d), s["w"].to(d)
        ms = (x * x).sum(dim=1, keepdim=True) / m + EPS
        along = (dy * w * x).sum(dim=1, keepdim=True)
        dx = dy * w / torch.sqrt(ms) - x * along / (m * ms * torch.sqrt(ms))
        if s["dres"] is not None:
            dx += s["dres"].to(d)
        return dx, (dy * x / torch.sqrt(ms)).sum(dim=0)
    if op == "dispatch":
        return None
    if op in ("combine", "combine_grad"):
        rows, wt = s["rows"].long(), s["weights"].to(d)
        if op == "combine":
            y = torch.zeros(n, m, dtype=d, device=DEV)
            for t in range(c["topk"]):
                at = torch.nonzero(rows[:, t] >= 0).reshape(-1)
                y[at] += wt[at, t, None] * s["x"][rows[at, t]].to(d)
            return y
        dx = torch.zeros(s["dx"].shape, dtype=d, device=DEV)
        dwt = torch.zeros(n, c["topk"], dtype=d, device=DEV)
        for t in range(c["topk"]):
            at = torch.nonzero(rows[:, t] >= 0).reshape(-1)
            dy = s["dy"][at].to(d)
            dx[rows[at, t]] = wt[at, t, None] * dy
            dwt[at, t] = (dy * s["x"][rows[at, t]].to(d)).sum(dim=1)
        return dx, dwt
    k, group = c["k"], c["group"]
    y = torch.zeros(n, m, dtype=d, device=DEV)
    values = torch.tensor([v if i < 8 else v - 16 for i, v in enumerate(range(16))] if c["w"] == "i4" else
                          list(range(16)) if c["w"] == "u4" else list(E2M1) + [-v for v in E2M1], dtype=d, device=DEV)
    x, w = s["x"].to(d), s["w"].long()
    even, odd = x[:, 0::2], x[:, 1::2]
    for b in range(0, k, group):
        h = slice(b // 2, min(k, b + group) // 2)
        lo, hi = values[w[:, h] & 15], values[w[:, h] >> 4]
        if s["zeros"] is not None:
            z = s["zeros"][:, b // group, None].to(d)
            lo, hi = lo - z, hi - z
        sc = s["scales"][:, b // group].to(d)
        y += (even[:, h] @ lo.t() + odd[:, h] @ hi.t()) * (torch.pow(2.0, sc - 127) if c["w"] == "e2m1" else sc)
    return y if s["bias"] is None else y + s["bias"].to(d)


def work(case):
    c, op = case, case["op"]
    size = {"f32": 4, "f16": 2, "bf16": 2}
    n, m = c["n"], c["m"]
    if op == "norm":
        x, y = size[c["x"]], size.get(c["y"], 1)
        b = n * m * (x + y) + m * size[c["x"]]
        if c["res"] != "none":
            b += 2 * n * m * size[c["res"]]
        if _mx(c["y"]):
            b += n * -(-m // 32)
        return {"bytes": b, "flops": 5 * n * m}
    if op == "norm_grad":
        return {"bytes": n * m * (size[c["x"]] + size[c["g"]] * (3 if c["dres"] else 2)) + m * (size[c["x"]] + 4),
                "flops": 10 * n * m}
    if op == "w4":
        groups = -(-c["k"] // c["group"])
        b = m * c["k"] // 2 + m * groups * (1 if c["w"] == "e2m1" else 3 if c["w"] == "u4" else 2)
        return {"bytes": b + 2 * n * (c["k"] + m) + (2 * m if c["bias"] else 0), "flops": 2 * n * m * c["k"]}
    topk = c["topk"]
    kept = 1.0 - c["drop"]
    if op == "dispatch":
        row = m + -(-m // 32) if _mx(c["x"]) else m * size[c["x"]]
        return {"bytes": n * row * (1 + topk * kept) + n * topk * (8 + 4 + 4) + 4 * c["experts"], "flops": 0}
    x = size[c["x"]]
    if op == "combine":
        return {"bytes": n * m * (topk * kept * x + size[c["y"]]) + 8 * n * topk, "flops": 2 * n * m * topk}
    return {"bytes": n * m * x * (1 + 2 * topk * kept) + 12 * n * topk, "flops": 3 * n * m * topk}
