"""Plain fp64 forms of the operators around the products (CPU, torch), with
the bounds their fp32 kernels stay within: each bound counts the roundings of
the sums and products it names, U = 2^-24 each."""
from __future__ import annotations

import torch

U = 2.0 ** -24
TOP = {"e4m3": 448.0, "e5m2": 57344.0, "e2m1": 6.0}
EMAX = {"e4m3": 8, "e5m2": 15, "e2m1": 2}
MANT = {"e4m3": 3, "e5m2": 2, "e2m1": 1}
EMIN = {"e4m3": -6, "e5m2": -14, "e2m1": 0}  # the smallest normal exponent
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def f64(t):
    return t.detach().cpu().double()


def half_step(v, dtype):
    """Half a step of a float type at |v| (subnormals included)."""
    fi = torch.finfo(dtype)
    return torch.clamp(v.abs(), min=fi.tiny) * (fi.eps / 2)


def narrow_half_step(v, kind):
    """Half a step of e4m3, e5m2 or e2m1 at |v|."""
    e = torch.floor(torch.log2(torch.clamp(v.abs(), min=2.0 ** EMIN[kind])))
    return torch.pow(2.0, e - MANT[kind] - 1)


def e2m1_values(codes, m):
    """(n, ceil(m/2)) bytes of two codes, the even feature in the low nibble, as (n, m) values."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64)
    c = codes.cpu().to(torch.int64)
    return table[torch.stack([c & 15, c >> 4], dim=2).reshape(c.shape[0], -1)[:, :m]]


def rmsnorm(x, r, w, eps):
    """(s, y) and y's relative error in fp32: the sum of squares (at most 64 terms a lane of the up to 16,384
    features held in registers, six adds across a wavefront and sixteen across them; longer tokens add
    m / 8192 terms), halved by the root; the division, the reciprocal root and two products; and x + r."""
    s = f64(x) if r is None else f64(x) + f64(r)
    rho = 1.0 / torch.sqrt((s * s).mean(dim=1, keepdim=True) + eps)
    terms = 64 + s.shape[1] / 8192 + 6 + 16
    return s, s * rho * f64(w), (terms / 2 + 8) * U


def rmsnorm_backward(s, dy, w, dr, eps):
    """(dx, dw, bound of dx, bound of dw) of the fp32 kernel, before the outputs' roundings."""
    s, dy, w = f64(s), f64(dy), f64(w)
    n, m = s.shape
    rho = 1.0 / torch.sqrt((s * s).mean(dim=1, keepdim=True) + eps)
    h, t = rho * s, w * dy
    mean = (t * h).mean(dim=1, keepdim=True)
    dx = rho * (t - h * mean)
    # sums of up to 64 + m/8192 + 22 terms; rho enters dx to the third power
    c = 3 * ((64 + m / 8192 + 22) + 8) * U
    bx = c * rho * (t.abs() + h.abs() * (t * h).abs().mean(dim=1, keepdim=True))
    if dr is not None:
        dx = dx + f64(dr)
        bx = bx + U * (f64(dr).abs() + dx.abs())
    # tokens add up one after another in at most n steps, then 32 + 32 across workgroups
    bw = (n + 64 + 64) * U * (dy * h).abs().sum(dim=0)
    return dx, (dy * h).sum(dim=0), bx, bw


def moe_sort(ids, experts):
    """(rows, offsets, order) of the stable sort, plain loops."""
    n, topk = ids.shape
    flat = ids.reshape(-1).tolist()
    by = [[f for f, e in enumerate(flat) if e == x] for x in range(experts)] if len(flat) * experts < 4_000_000 else None
    if by is None:
        by = [[] for _ in range(experts)]
        for f, e in enumerate(flat):
            if 0 <= e < experts:
                by[e].append(f)
    order = [f for fs in by for f in fs]
    rows = [-1] * len(flat)
    for p, f in enumerate(order):
        rows[f] = p
    offsets = [0]
    for fs in by:
        offsets.append(offsets[-1] + len(fs))
    return (torch.tensor(rows, dtype=torch.int32).reshape(n, topk), torch.tensor(offsets, dtype=torch.int32),
            torch.tensor(order, dtype=torch.int32))


def moe_combine(x, rows, weights, n, m):
    """(y, bound): topk products and adds."""
    x, rows = f64(x), rows.cpu().tolist()
    y, a = torch.zeros(n, m, dtype=torch.float64), torch.zeros(n, m, dtype=torch.float64)
    for j in range(n):
        for t, p in enumerate(rows[j]):
            if 0 <= p < x.shape[0]:
                v = x[p] * (1.0 if weights is None else float(weights[j, t]))
                y[j] += v
                a[j] += v.abs()
    return y, (len(rows[0]) if rows else 0) * 2 * U * a


def moe_combine_backward(dy, x, rows, weights):
    """({place: row of dx}, dweights, bound of dweights)."""
    dy, x = f64(dy), f64(x)
    n, topk = rows.shape
    m = dy.shape[1]
    dx, dw, bw = {}, torch.zeros(n, topk, dtype=torch.float64), torch.zeros(n, topk, dtype=torch.float64)
    for j in range(n):
        for t in range(topk):
            p = int(rows[j, t])
            if 0 <= p < x.shape[0]:
                dx[p] = dy[j] * float(weights[j, t])
                dw[j, t] = (dy[j] * x[p]).sum()
                # a lane adds 8 products of each of m / 512 (long tokens: 2,048) runs; then 6 + 4 adds
                bw[j, t] = (8 * (m / 512 + 1) + 10) * U * (dy[j] * x[p]).abs().sum()
    return dx, dw, bw


def w4_values(codes, type_w, k):
    """(m, ldw/2) bytes as (m, k) code values."""
    c = codes.cpu().to(torch.int64)
    q = torch.stack([c & 15, c >> 4], dim=2).reshape(c.shape[0], -1)[:, :k]
    if type_w == "e2m1":
        return torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64)[q]
    return torch.where(q >= 8, q - 16, q).double() if type_w == "i4" else q.double()


def gemm_w4(codes, type_w, scales, group, zeros, x, k):
    """(products (n, m) before the epilogue, bound).  Within a group both the sum of (16 + q) x and that of
    (16 + z) x take group additions (counted at a whole step of fp32 each, matrix cores not always rounding to
    nearest) of terms up to 31 |x|; then three roundings a group, and the groups' own sum over up to
    groups + 8 additions."""
    v, x = w4_values(codes, type_w, k), f64(x)
    m, groups = v.shape[0], -(-k // group)
    s = (torch.pow(2.0, scales.cpu().double() - 127) if type_w == "e2m1" else f64(scales))[:, :groups]
    y = torch.zeros(x.shape[0], m, dtype=torch.float64)
    b = torch.zeros_like(y)
    for q in range(groups):
        cut = slice(q * group, min(k, (q + 1) * group))
        z = f64(zeros)[:, q:q + 1] if zeros is not None else 0.0
        y += (x[:, cut] @ (v[:, cut] - z).t()) * s[:, q]
        size = x[:, cut].abs().sum(dim=1, keepdim=True) * s[:, q].abs()
        # a group longer than 256 leaves in pieces of 256
        length = min(cut.stop - cut.start, 256)
        pieces = -(-(cut.stop - cut.start) // 256)
        b += size * (2 * (length + 4) * 2 * U * (31.0 if type_w != "e2m1" else 6.0) + (groups * pieces + 8 + 4) * U * 31.0)
    return y, b


def _terms(m):
    """Additions that a term of a sum over m features takes part in (as counted in rmsnorm)."""
    return 64 + m / 8192 + 6 + 16


def layernorm(x, r, w, b, eps):
    """(s, y, bound of y before its rounding).  The mean is off by its sum's additions, and every difference from it
    by that and the rounding of s; the squares of the differences sum to the variance, in which a shift of all
    differences counts squared only, as they sum to zero."""
    s = f64(x) if r is None else f64(x) + f64(r)
    m = s.shape[1]
    d = s - s.mean(dim=1, keepdim=True)
    rho = 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + eps)
    h, e_h = _centred(s, d, rho, m)
    W = torch.ones(m, dtype=torch.float64) if w is None else f64(w)
    B = torch.zeros(m, dtype=torch.float64) if b is None else f64(b)
    y = h * W + B
    return s, y, W.abs() * e_h + 3 * U * ((h * W).abs() + B.abs())


def _centred(s, d, rho, m):
    """The normalised features and their bound."""
    shift = (_terms(m) + 3) * U * s.abs().mean(dim=1, keepdim=True)
    rel = (_terms(m) / 2 + 8) * U + (rho * shift) ** 2 + rho * rho * U * (d * s).abs().mean(dim=1, keepdim=True)
    h = d * rho
    return h, rho * (shift + 2 * U * s.abs()) + h.abs() * rel


def layernorm_backward(s, dy, w, dr, eps):
    """(dx, dw, db, and their bounds) of the fp32 kernel, before the outputs' roundings."""
    s, dy = f64(s), f64(dy)
    n, m = s.shape
    W = torch.ones(m, dtype=torch.float64) if w is None else f64(w)
    d = s - s.mean(dim=1, keepdim=True)
    rho = 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + eps)
    h, e_h = _centred(s, d, rho, m)
    t = W * dy
    level, along = t.mean(dim=1, keepdim=True), (t * h).mean(dim=1, keepdim=True)
    c = (_terms(m) + 4) * U
    e_along = c * (t * h).abs().mean(dim=1, keepdim=True) + (t.abs() * e_h).mean(dim=1, keepdim=True)
    part = t - level - h * along
    # rho is off by its share of h's bound: a relative e_h / |h| at most terms / 2 + 8 roundings and the shifts'
    shift = (_terms(m) + 3) * U * s.abs().mean(dim=1, keepdim=True)
    rel = (_terms(m) / 2 + 8) * U + (rho * shift) ** 2 + rho * rho * U * (d * s).abs().mean(dim=1, keepdim=True)
    bx = rho * (4 * U * (t.abs() + level.abs() + (h * along).abs()) + c * t.abs().mean(dim=1, keepdim=True)
                + h.abs() * e_along + e_h * along.abs() + rel * part.abs())
    dx = rho * part
    if dr is not None:
        dx = dx + f64(dr)
        bx = bx + U * (f64(dr).abs() + dx.abs())
    steps = (n + 64 + 64) * U  # as in rmsnorm_backward
    bw = steps * (dy * h).abs().sum(dim=0) + (dy.abs() * (e_h + U * h.abs())).sum(dim=0)
    return dx, (dy * h).sum(dim=0), dy.sum(dim=0), bx, bw, steps * dy.abs().sum(dim=0)


def mx_quantize(x, kind):
    """(elements (n, m) as fp64 values before the block scale, scale codes (n, blocks)) of an (n, m) array: exact.  A
    block with a NaN: scale 255, elements of zero."""
    v = f64(x)
    n, m = v.shape
    nb = -(-m // 32)
    b = torch.nn.functional.pad(v, (0, 32 * nb - m)).reshape(n, nb, 32)
    bad = torch.isnan(b).any(dim=2)
    b = torch.where(bad[:, :, None], 0.0, b)
    amax = b.abs().amax(dim=2)
    finite = torch.where(torch.isinf(amax), 2.0 ** 128, amax)
    e = (torch.frexp(finite).exponent.double() - 1 - EMAX[kind]).clamp(-127, 127)
    code = torch.where(amax > 0, e + 127, 0.0)
    q = (b / torch.pow(2.0, code - 127)[:, :, None]).clamp(-TOP[kind], TOP[kind])
    a = q.abs()
    low = torch.floor(torch.log2(a.clamp(min=2.0 ** EMIN[kind])))
    low = torch.where(torch.pow(2.0, low) > a.clamp(min=2.0 ** EMIN[kind]), low - 1, low)  # (log2 next to a power)
    step = torch.pow(2.0, low - MANT[kind])
    r = torch.round(a / step) * step  # half to even
    r = torch.copysign(r.clamp(max=TOP[kind]), q)
    return r.reshape(n, 32 * nb)[:, :m], torch.where(bad, 255.0, code).to(torch.uint8)


def moe_route(logits, topk, score, renorm, scale, bias=None):
    """(ids, weights, p, values that were compared), plain loops."""
    l = f64(logits)
    n, experts = l.shape
    live = l > -torch.inf  # False for NaN
    top = torch.where(live, l, -torch.inf).amax(dim=1, keepdim=True)
    p = torch.where(live, torch.exp(l - torch.where(live.any(dim=1, keepdim=True), top, 0.0)), 0.0)
    if score == "softmax":
        p = p / p.sum(dim=1, keepdim=True).clamp(min=1e-300)  # (a row of masks alone: zeros)
    else:
        p = torch.where(live, torch.sigmoid(l), 0.0)
    by = torch.where(live, l if bias is None else p + f64(bias), -torch.inf)
    ids = torch.full((n, topk), -1, dtype=torch.int32)
    for j in range(n):
        order = sorted((e for e in range(experts) if by[j, e] > -torch.inf), key=lambda e: (-float(by[j, e]), e))
        for t, e in enumerate(order[:topk]):
            ids[j, t] = e
    chosen = torch.where(ids >= 0, p.gather(1, ids.long().clamp(min=0)), 0.0)
    total = chosen.sum(dim=1, keepdim=True) if renorm else torch.ones(n, 1, dtype=torch.float64)
    return ids, torch.where(total > 0, scale * chosen / total, 0.0), p, by


def moe_route_backward(logits, ids, dweights, score, renorm, scale):
    """dlogits by autograd in fp64."""
    l = f64(logits).requires_grad_()
    live = l.detach() > -torch.inf
    with torch.enable_grad():
        if score == "softmax":
            p = torch.softmax(torch.where(live, l, -1e300), dim=1)
        else:
            p = torch.where(live, torch.sigmoid(l), 0.0)
        ok = (ids >= 0) & (ids < l.shape[1])
        at = torch.where(ok, ids, 0).long()
        w = torch.where(ok, p.gather(1, at), 0.0)
        if renorm:
            w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
        (scale * w * f64(dweights)).sum().backward()
    return l.grad


def moe_layer(x, ids, weights, w1, w2, gated, act, b1=None, b2=None):
    """(y, bound before y's rounding) for matrices of fp64 values (experts, rows, k).  Sums of K products are counted at
    K + 8 whole steps of fp32, activations at a slope of 1.13 and four roundings, u's planes at 2^-16."""
    x, wt = f64(x), f64(weights)
    n, m = x.shape
    experts, hidden = w1.shape[0], w2.shape[2]
    y, b = torch.zeros(n, m, dtype=torch.float64), torch.zeros(n, m, dtype=torch.float64)
    fn = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu,
          "gelu": torch.nn.functional.gelu}[act]
    for j in range(n):
        for t in range(ids.shape[1]):
            e = int(ids[j, t])
            if not 0 <= e < experts:
                continue
            u = w1[e] @ x[j]
            eu = (m + 8) * 2 * U * (w1[e].abs() @ x[j].abs())
            if b1 is not None:
                u = u + f64(b1[e])
                eu = eu + U * (u.abs() + f64(b1[e]).abs())
            if act != "none":
                g, eg = fn(u[:hidden]), 1.13 * eu[:hidden]
                eg = eg + 4 * U * (g.abs() + u[:hidden].abs())
            else:
                g, eg = u[:hidden], eu[:hidden]
            if gated:
                up, e_up = u[hidden:], eu[hidden:]
                eg = g.abs() * e_up + (up.abs() + e_up) * eg + U * (g * up).abs()
                g = g * up
            eg = eg + 2.0 ** -16 * g.abs()
            z = w2[e] @ g
            ez = (hidden + 8) * 4 * U * (w2[e].abs() @ g.abs()) + w2[e].abs() @ eg
            if b2 is not None:
                z = z + f64(b2[e])
                ez = ez + U * (z.abs() + f64(b2[e]).abs())
            y[j] += wt[j, t] * z
            b[j] += wt[j, t].abs() * (ez + 2 * (ids.shape[1] + 1) * U * z.abs())
    return y, b
