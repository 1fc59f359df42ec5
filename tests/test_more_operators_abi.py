"""Layer norm, MX quantization, the router and the layer of experts reject bad calls before any HIP call, and take
empty ones without a launch (no GPU needed)."""
import ctypes

import pytest

import tile_hierarchy_linear_amd as thl

INVALID, UNSUPPORTED, MISALIGNED, OK = (thl.THL_ERR_INVALID, thl.THL_ERR_UNSUPPORTED, thl.THL_ERR_MISALIGNED,
                                        thl.THL_OK)
D = thl.DTYPES
# Fake (never dereferenced) device addresses, 256-byte aligned and far apart.
P = [0x10000000 * i for i in range(1, 14)]
B16 = ("bf16", "bf16", "bf16", "bf16")
FP8 = ("bf16", "bf16", "bf16", "e4m3")
FP4 = ("bf16", "bf16", "bf16", "e2m1")


def norm(m=64, n=4, x=P[0], ldx=64, r=None, ldr=64, s=None, lds=64, w=P[3], b=P[6], eps=1e-6, scale=1.0, y=P[4],
         ldy=64, sf=None, ld_sf=16, types=B16):
    t = thl.thl_norm_types(*(D[v] for v in types)) if types else None
    return thl.thl_layernorm(m, n, x, ldx, r, ldr, s, lds, w, b, eps, scale, y, ldy, sf, ld_sf, t)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(types=None), INVALID),
    (dict(ldx=63), INVALID), (dict(ldy=63), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(s=P[2]), INVALID), (dict(r=P[1], ldr=63), INVALID), (dict(r=P[1], s=P[2], lds=63), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(scale=0.0, types=FP8), INVALID), (dict(scale=1e-45, types=FP8), INVALID),
    (dict(scale=2.0), UNSUPPORTED), (dict(scale=2.0, sf=P[5], types=FP8), UNSUPPORTED), (dict(sf=P[5]), UNSUPPORTED),
    (dict(types=FP4), UNSUPPORTED), (dict(types=FP4, sf=P[5], ldy=65), INVALID),
    (dict(types=FP8, sf=P[5], ld_sf=1), INVALID), (dict(types=("i8", "i8", "bf16", "bf16")), UNSUPPORTED),
    (dict(types=("bf16", "bf16", "e4m3", "bf16")), UNSUPPORTED),
    (dict(types=("bf16", "bf16", "e4m3", "bf16"), w=None), UNSUPPORTED),  # the bias's type
    (dict(types=("bf16", "bf16", "bf16", "i8")), UNSUPPORTED),
    (dict(r=P[1], types=("bf16", "f16", "bf16", "bf16")), UNSUPPORTED),
    (dict(m=1 << 27, ldx=1 << 27, ldy=1 << 27), UNSUPPORTED), (dict(n=1 << 31), UNSUPPORTED),
    (dict(x=P[0] + 1), MISALIGNED), (dict(w=P[3] + 1), MISALIGNED), (dict(b=P[6] + 1), MISALIGNED),
    (dict(y=P[4] + 1), MISALIGNED), (dict(r=P[1] + 1), MISALIGNED), (dict(r=P[1], s=P[2] + 1), MISALIGNED),
    (dict(y=P[0] + 2), INVALID), (dict(y=P[0], ldy=72), INVALID), (dict(y=P[3]), INVALID), (dict(y=P[6]), INVALID),
    (dict(y=P[0], types=FP8), INVALID), (dict(r=P[1], s=P[1], lds=80), INVALID), (dict(r=P[1], y=P[1]), INVALID),
    (dict(r=P[1], s=P[6]), INVALID), (dict(r=P[1], s=P[3]), INVALID), (dict(r=P[1], s=P[0], y=P[0]), INVALID),
    (dict(types=FP8, sf=P[4]), INVALID), (dict(types=FP8, sf=P[0]), INVALID), (dict(types=FP8, sf=P[6]), INVALID),
    (dict(m=0), OK), (dict(n=0), OK), (dict(m=0, x=None, w=None, b=None, y=None), OK),
])
def test_layernorm_refusals(kw, want):
    assert norm(**kw) == want


def grad(m=64, n=4, s=P[0], lds=64, dy=P[1], lddy=64, dr=None, lddr=64, w=P[3], eps=1e-6, dx=P[4], lddx=64, dw=P[5],
         db=P[7], ws=P[6], size=1 << 20, types=("bf16", "bf16", "bf16", "f32")):
    t = thl.thl_norm_grad_types(*(D[v] for v in types)) if types else None
    return thl.thl_layernorm_backward(m, n, s, lds, dy, lddy, dr, lddr, w, eps, dx, lddx, dw, db, ws, size, t)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(types=None), INVALID), (dict(lds=1), INVALID),
    (dict(lddy=1), INVALID), (dict(lddx=1), INVALID), (dict(dr=P[2], lddr=1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(s=None), INVALID), (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(ws=None), INVALID),
    (dict(size=64 * 8 - 1), INVALID), (dict(dw=None, size=64 * 8 - 1), INVALID), (dict(ws=P[6] + 2), MISALIGNED),
    (dict(types=("e4m3", "bf16", "bf16", "f32")), UNSUPPORTED), (dict(types=("bf16", "bf16", "i8", "f32")), UNSUPPORTED),
    (dict(types=("bf16", "bf16", "bf16", "f16")), UNSUPPORTED),
    (dict(types=("bf16", "bf16", "bf16", "bf16"), w=None), UNSUPPORTED),  # no weight whose type it could be
    (dict(dx=P[0] + 2), INVALID), (dict(dx=P[1], lddx=80), INVALID), (dict(dx=P[3]), INVALID),
    (dict(dx=P[0], types=("f32", "bf16", "bf16", "f32")), INVALID), (dict(dw=P[0]), INVALID), (dict(dw=P[4]), INVALID),
    (dict(db=P[5]), INVALID), (dict(db=P[4]), INVALID), (dict(db=P[6]), INVALID), (dict(db=P[5] + 4, n=0), INVALID),
    (dict(ws=P[4]), INVALID), (dict(ws=P[1]), INVALID), (dict(ws=P[5]), INVALID), (dict(dx=P[4] + 1), MISALIGNED),
    (dict(dw=P[5] + 2), MISALIGNED), (dict(db=P[7] + 2), MISALIGNED), (dict(m=0), OK),
    (dict(n=0, dw=None, db=None), OK),
])
def test_layernorm_backward_refusals(kw, want):
    assert grad(**kw) == want


def mx(m=64, n=96, x=P[0], ldx=64, y=P[1], ldy=64, sf=P[2], ld_sf=2, yt=P[3], ldyt=96, sft=P[4], ld_sft=3, tx="bf16",
       ty="e2m1"):
    return thl.thl_mx_quantize(m, n, x, ldx, y, ldy, sf, ld_sf, yt, ldyt, sft, ld_sft, tx, ty)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(ldx=63), INVALID), (dict(ldy=63), INVALID),
    (dict(ldy=65), INVALID), (dict(ldyt=95), INVALID), (dict(ldyt=97), INVALID), (dict(ld_sf=1), INVALID),
    (dict(ld_sft=2), INVALID), (dict(sf=None), INVALID), (dict(y=None), INVALID), (dict(sft=None), INVALID),
    (dict(yt=None), INVALID), (dict(y=None, sf=None, yt=None, sft=None), INVALID), (dict(x=None), INVALID),
    (dict(tx="e4m3"), UNSUPPORTED), (dict(ty="bf16"), UNSUPPORTED), (dict(ty="e2m3"), UNSUPPORTED),
    (dict(m=1 << 27, ldx=1 << 27), UNSUPPORTED), (dict(n=1 << 31), UNSUPPORTED), (dict(x=P[0] + 1), MISALIGNED),
    (dict(y=P[0]), INVALID), (dict(sf=P[0]), INVALID), (dict(yt=P[1]), INVALID), (dict(sft=P[3]), INVALID),
    (dict(sft=P[2]), INVALID), (dict(ty="e4m3", ldy=65, ldyt=97, m=0), OK), (dict(m=0), OK), (dict(n=0), OK),
])
def test_mx_quantize_refusals(kw, want):
    assert mx(**kw) == want


def route(n=8, topk=2, experts=16, l=P[0], ld=16, bias=None, ids=P[1], weights=P[2], type="f32", score=0, renorm=1,
          scale=1.0, how=True):
    h = thl.thl_route(D[type], score, renorm, scale) if how else None
    return thl.thl_moe_route(n, topk, experts, l, ld, bias, h, ids, weights)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(topk=-1), INVALID), (dict(experts=0), INVALID), (dict(how=False), INVALID),
    (dict(ld=15), INVALID), (dict(experts=1025, ld=1025), UNSUPPORTED), (dict(topk=65), UNSUPPORTED),
    (dict(type="e4m3"), UNSUPPORTED), (dict(score=2), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(l=None), INVALID), (dict(ids=None), INVALID),
    (dict(weights=None), INVALID), (dict(l=P[0] + 2), MISALIGNED), (dict(ids=P[1] + 2), MISALIGNED),
    (dict(weights=P[2] + 1), MISALIGNED), (dict(bias=P[3] + 2), MISALIGNED), (dict(ids=P[0]), INVALID),
    (dict(weights=P[1]), INVALID), (dict(bias=P[2]), INVALID), (dict(n=1 << 31), UNSUPPORTED), (dict(n=0), OK),
    (dict(topk=0), OK),
])
def test_moe_route_refusals(kw, want):
    assert route(**kw) == want


def route_grad(n=8, topk=2, experts=16, l=P[0], ld=16, ids=P[1], dw=P[2], dl=P[3], lddl=16, type="f32", score=0,
               renorm=1, scale=1.0):
    return thl.thl_moe_route_backward(n, topk, experts, l, ld, thl.thl_route(D[type], score, renorm, scale), ids, dw,
                                      dl, lddl)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(ld=15), INVALID), (dict(lddl=15), INVALID), (dict(lddl=1 << 31), UNSUPPORTED),
    (dict(l=None), INVALID), (dict(ids=None), INVALID), (dict(dw=None), INVALID), (dict(dl=None), INVALID),
    (dict(dl=P[3] + 2), MISALIGNED), (dict(dw=P[2] + 2), MISALIGNED), (dict(dl=P[0] + 4), INVALID),
    (dict(dl=P[0], lddl=20), INVALID), (dict(dl=P[1]), INVALID), (dict(dl=P[2]), INVALID), (dict(n=0), OK),
])
def test_moe_route_backward_refusals(kw, want):
    assert route_grad(**kw) == want


def matrix(w, rows, k, type="bf16", sf=None, ld=None, stride=None, ld_sf=None, stride_sf=None, bias=None,
           type_bias="none"):
    b = -(-k // 32)
    return thl.thl_expert_matrix(w, k if ld is None else ld, rows * k if stride is None else stride, sf,
                                 b if ld_sf is None else ld_sf, rows * b if stride_sf is None else stride_sf, bias, rows,
                                 D[type], D[type_bias])


def layer(m=64, hidden=32, n=4, topk=2, experts=8, x=P[0], ldx=64, ids=P[1], ld_ids=2, size_ids=4, weights=P[2],
          flags=thl.THL_MOE_GATED | thl.THL_MOE_SILU, y=P[3], ldy=64, tx="bf16", ty="bf16", ws=P[4], size=1 << 20,
          w1=P[5], w2=P[6], up={}, down={}, both={}, structs=True):
    a = matrix(w1, 2 * hidden if flags & 1 else hidden, m, **{**both, **up})
    b = matrix(w2, m, hidden, **{**both, **down})
    return thl.thl_moe_layer(m, hidden, n, topk, experts, x, ldx, ids, ld_ids, size_ids, weights, a if structs else None,
                             b if structs else None, flags, y, ldy, tx, ty, ws, size)


MX = dict(type="e2m1", sf=P[7])


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(hidden=-1), INVALID), (dict(n=-1), INVALID), (dict(topk=-1), INVALID),
    (dict(experts=0), INVALID), (dict(structs=False), INVALID), (dict(ldx=63), INVALID), (dict(ldy=63), INVALID),
    (dict(ld_ids=1), INVALID), (dict(hidden=0), INVALID), (dict(topk=0), INVALID), (dict(n=513), UNSUPPORTED),
    (dict(topk=1025, ld_ids=1025), UNSUPPORTED), (dict(size_ids=2), UNSUPPORTED), (dict(tx="f32"), UNSUPPORTED),
    (dict(ty="e4m3"), UNSUPPORTED), (dict(flags=16), INVALID),
    (dict(flags=thl.THL_MOE_RELU | thl.THL_MOE_SILU), INVALID), (dict(both=dict(type="f16")), UNSUPPORTED),
    (dict(both=dict(type="e5m2", sf=P[7])), UNSUPPORTED), (dict(both=dict(type="e2m1")), INVALID),
    (dict(up=dict(sf=P[7])), INVALID),  # block scales of 16-bit weights
    (dict(up=MX, down=dict(MX, ld_sf=0)), INVALID), (dict(up=dict(MX, ld=65)), INVALID),
    (dict(up=dict(MX, stride=65)), INVALID), (dict(up=dict(ld=63)), INVALID), (dict(up=dict(stride=-1)), INVALID),
    (dict(down=dict(ld=31)), INVALID), (dict(up=dict(bias=P[8], type_bias="i32")), UNSUPPORTED),
    (dict(up=dict(bias=P[8] + 2, type_bias="f32")), MISALIGNED), (dict(w1=None), INVALID), (dict(w2=None), INVALID),
    (dict(x=None), INVALID), (dict(ids=None), INVALID), (dict(weights=None), INVALID), (dict(y=None), INVALID),
    (dict(ws=None), INVALID), (dict(size=8 * 4 * (64 + 64) - 1), INVALID), (dict(ws=P[4] + 2), MISALIGNED),
    (dict(x=P[0] + 1), MISALIGNED), (dict(y=P[3] + 1), MISALIGNED), (dict(ids=P[1] + 2), MISALIGNED),
    (dict(ids=P[1] + 4, size_ids=8), MISALIGNED), (dict(w1=P[5] + 1), MISALIGNED), (dict(y=P[0]), INVALID),
    (dict(y=P[1]), INVALID), (dict(y=P[2]), INVALID), (dict(y=P[4]), INVALID), (dict(y=P[5]), INVALID),
    (dict(y=P[6]), INVALID), (dict(y=P[7], up=MX), INVALID), (dict(y=P[8], up=dict(bias=P[8], type_bias="f32")), INVALID),
    (dict(ws=P[0]), INVALID), (dict(ws=P[6]), INVALID), (dict(m=0), OK), (dict(n=0), OK),
    (dict(m=1 << 27, ldx=1 << 27, ldy=1 << 27), UNSUPPORTED), (dict(up=dict(stride=1 << 41)), UNSUPPORTED),
    (dict(experts=1 << 30, up=dict(stride=1 << 33)), UNSUPPORTED),  # byte offsets past 64 bits
    (dict(experts=1 << 30, up=MX, down=dict(MX, stride_sf=1 << 34)), UNSUPPORTED),
])
def test_moe_layer_refusals(kw, want):
    assert layer(**kw) == want


def test_workspace_sizes():
    assert thl.thl_layernorm_backward_workspace(600, 4) == 2 * 4 * 600 * 4  # two partial rows a token
    assert thl.thl_layernorm_backward_workspace(64, 0) == thl.thl_layernorm_backward_workspace(0, 4) == 0
    assert thl.thl_layernorm_backward_workspace(64, 1 << 20) <= 2 * 64 * 4 * 4096  # bounded in the tokens
    assert thl.thl_moe_layer_workspace(64, 100, 3, 2) >= 6 * 4 * (100 + 64)
    assert thl.thl_moe_layer_workspace(64, 100, 1025, 1) == thl.thl_moe_layer_workspace(64, 100, 0, 1) == 0
    assert thl.thl_moe_layer_workspace(64, 100, 1 << 40, 1 << 40) == 0


def test_structures_match_the_header():
    assert ctypes.sizeof(thl.thl_route) == 16
    assert ctypes.sizeof(thl.thl_expert_matrix) == 72


def test_torch_forms_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    u = torch.zeros(4, 4, dtype=torch.uint8)
    for call in (lambda: thl.layernorm(x, x[0], x[0], x), lambda: thl.layernorm_backward(x, x, x[0], x),
                 lambda: thl.mx_quantize(x, u, u), lambda: thl.moe_route(x, i, x[:, :2]),
                 lambda: thl.moe_route_backward(x, i, x[:, :2], x),
                 lambda: thl.moe_layer(x, i, x[:, :2], x[None], x[None], x)):
        with pytest.raises(ValueError):
            call()
