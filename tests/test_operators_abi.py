"""The operators around the products reject bad calls before any HIP call, and
take empty ones without a launch (no GPU needed)."""
import ctypes

import pytest

import tile_hierarchy_linear_amd as thl

INVALID, UNSUPPORTED, MISALIGNED, OK = (thl.THL_ERR_INVALID, thl.THL_ERR_UNSUPPORTED, thl.THL_ERR_MISALIGNED,
                                        thl.THL_OK)
D = thl.DTYPES
# Fake (never dereferenced) device addresses, 256-byte aligned and far apart.
P = [0x10000000 * i for i in range(1, 10)]


def norm(m=64, n=4, x=P[0], ldx=64, r=None, ldr=64, s=None, lds=64, w=P[3], eps=1e-6, scale=1.0, y=P[4], ldy=64,
         sf=None, ld_sf=16, types=("bf16", "bf16", "bf16", "bf16")):
    t = thl.thl_norm_types(*(D[v] for v in types)) if types else None
    return thl.thl_rmsnorm(m, n, x, ldx, r, ldr, s, lds, w, eps, scale, y, ldy, sf, ld_sf, t)


FP8 = ("bf16", "bf16", "bf16", "e4m3")
FP4 = ("bf16", "bf16", "bf16", "e2m1")


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(types=None), INVALID),
    (dict(ldx=63), INVALID), (dict(ldy=63), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(y=None), INVALID), (dict(s=P[2]), INVALID),  # a sum without a residual
    (dict(r=P[1], ldr=63), INVALID), (dict(r=P[1], s=P[2], lds=63), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(scale=0.0, types=FP8), INVALID), (dict(scale=float("inf"), types=FP8), INVALID),
    (dict(scale=1e-45, types=FP8), INVALID), (dict(scale=float("nan"), types=FP8), INVALID),
    (dict(scale=2.0), UNSUPPORTED), (dict(scale=2.0, sf=P[5], types=FP8), UNSUPPORTED),
    (dict(sf=P[5]), UNSUPPORTED),  # block scales of a 16-bit output
    (dict(types=FP4), UNSUPPORTED), (dict(types=FP4, sf=P[5], ldy=65), INVALID),
    (dict(types=FP8, sf=P[5], ld_sf=1), INVALID),
    (dict(types=("i8", "i8", "bf16", "bf16")), UNSUPPORTED), (dict(types=("bf16", "bf16", "e4m3", "bf16")), UNSUPPORTED),
    (dict(types=("bf16", "bf16", "bf16", "i8")), UNSUPPORTED),
    (dict(r=P[1], types=("bf16", "f16", "bf16", "bf16")), UNSUPPORTED),
    (dict(m=1 << 27, ldx=1 << 27, ldy=1 << 27), UNSUPPORTED), (dict(n=1 << 31), UNSUPPORTED),
    (dict(x=P[0] + 1), MISALIGNED), (dict(w=P[3] + 1), MISALIGNED), (dict(y=P[4] + 1), MISALIGNED),
    (dict(r=P[1] + 1), MISALIGNED), (dict(r=P[1], s=P[2] + 1), MISALIGNED),
    (dict(y=P[0] + 2), INVALID), (dict(y=P[0], ldy=72), INVALID), (dict(y=P[3]), INVALID),
    (dict(y=P[0], types=FP8), INVALID),  # y over x in another type
    (dict(r=P[1], s=P[1], lds=80), INVALID), (dict(r=P[1], y=P[1]), INVALID), (dict(r=P[1], s=P[0], y=P[0]), INVALID),
    (dict(r=P[1], s=P[0], types=("bf16", "f32", "bf16", "bf16")), INVALID),
    (dict(types=FP8, sf=P[4]), INVALID), (dict(types=FP8, sf=P[0]), INVALID), (dict(types=FP8, sf=P[3]), INVALID),
    (dict(m=0), OK), (dict(n=0), OK), (dict(m=0, x=None, w=None, y=None), OK),
])
def test_rmsnorm_refusals(kw, want):
    assert norm(**kw) == want


def grad(m=64, n=4, s=P[0], lds=64, dy=P[1], lddy=64, dr=None, lddr=64, w=P[3], eps=1e-6, dx=P[4], lddx=64, dw=P[5],
         ws=P[6], size=1 << 20, types=("bf16", "bf16", "bf16", "f32")):
    t = thl.thl_norm_grad_types(*(D[v] for v in types)) if types else None
    return thl.thl_rmsnorm_backward(m, n, s, lds, dy, lddy, dr, lddr, w, eps, dx, lddx, dw, ws, size, t)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(types=None), INVALID), (dict(lds=1), INVALID),
    (dict(lddy=1), INVALID), (dict(lddx=1), INVALID), (dict(dr=P[2], lddr=1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(s=None), INVALID), (dict(dy=None), INVALID), (dict(w=None), INVALID), (dict(dx=None), INVALID),
    (dict(ws=None), INVALID), (dict(size=64 * 4 - 1), INVALID), (dict(ws=P[6] + 2), MISALIGNED),
    (dict(types=("e4m3", "bf16", "bf16", "f32")), UNSUPPORTED), (dict(types=("bf16", "bf16", "i8", "f32")), UNSUPPORTED),
    (dict(types=("bf16", "bf16", "bf16", "f16")), UNSUPPORTED),
    (dict(dx=P[0] + 2), INVALID), (dict(dx=P[1], lddx=80), INVALID), (dict(dx=P[3]), INVALID),
    (dict(dx=P[0], types=("f32", "bf16", "bf16", "f32")), INVALID),
    (dict(dw=P[0]), INVALID), (dict(dw=P[4]), INVALID), (dict(ws=P[4]), INVALID), (dict(ws=P[1]), INVALID),
    (dict(ws=P[5]), INVALID), (dict(dx=P[4] + 1), MISALIGNED), (dict(dw=P[5] + 2), MISALIGNED),
    (dict(m=0), OK), (dict(n=0, dw=None), OK),
])
def test_rmsnorm_backward_refusals(kw, want):
    assert grad(**kw) == want


def test_workspace_sizes():
    assert thl.thl_rmsnorm_backward_workspace(600, 4) == 4 * 600 * 4  # a partial row a token
    assert thl.thl_rmsnorm_backward_workspace(64, 5) == 2 * 64 * 4  # of four short tokens
    assert thl.thl_rmsnorm_backward_workspace(64, 0) == thl.thl_rmsnorm_backward_workspace(0, 4) == 0
    assert thl.thl_rmsnorm_backward_workspace(64, 1 << 20) <= 64 * 4 * 4096  # bounded in the tokens
    assert thl.thl_moe_sort_workspace(512, 8, 64) == 0
    assert thl.thl_moe_sort_workspace(513, 8, 64) > 0
    assert thl.thl_moe_sort_workspace(1 << 26, 8, 64) <= 256 * 64 * 4
    assert thl.thl_gemm_w4_workspace(4096, 2, 4096) == thl.thl_gemm_w4_workspace(4096, 40, 0) == 0
    assert thl.thl_gemm_w4_workspace(64, 17, 256) == 0  # one pair of units: nothing to split
    assert thl.thl_gemm_w4_workspace(64, 17, 4096) == 8 * 17 * 64 * 4
    assert thl.thl_gemm_w4_workspace(1 << 20, 17, 4096) == 0  # enough features
    assert thl.thl_moe_sort_workspace(-1, 8, 64) == thl.thl_moe_sort_workspace(513, 8, 1 << 20) == 0


def sort(n=8, topk=2, experts=4, ids=P[0], ld=2, size_ids=8, rows=P[1], offsets=P[2], order=P[3], ws=None, size=0):
    return thl.thl_moe_sort(n, topk, experts, ids, ld, size_ids, rows, offsets, order, ws, size)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(topk=-1), INVALID), (dict(experts=0), INVALID), (dict(experts=1025), UNSUPPORTED),
    (dict(ld=1), INVALID), (dict(size_ids=2), UNSUPPORTED), (dict(ids=None), INVALID), (dict(rows=None), INVALID),
    (dict(offsets=None), INVALID), (dict(ids=P[0] + 4), MISALIGNED), (dict(rows=P[1] + 2), MISALIGNED),
    (dict(n=1 << 30), UNSUPPORTED), (dict(n=4096), INVALID),  # more than one workgroup without a workspace
    (dict(n=4096, ws=P[4], size=8), INVALID), (dict(n=4096, ws=P[4] + 1, size=1 << 20), MISALIGNED),
    (dict(rows=P[0]), INVALID), (dict(offsets=P[1] + 4), INVALID), (dict(order=P[1]), INVALID),
    (dict(n=4096, ws=P[1], size=1 << 20), INVALID),
])
def test_moe_sort_refusals(kw, want):
    assert sort(**kw) == want


def gather(m=64, n=8, topk=2, x=P[0], ldx=64, sfx=None, ld_sfx=2, rows=P[1], rows_y=16, y=P[2], ldy=64, sfy=None,
           ld_sfy=2, type="bf16"):
    return thl.thl_moe_gather(m, n, topk, x, ldx, sfx, ld_sfx, rows, rows_y, y, ldy, sfy, ld_sfy, type)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(rows_y=-1), INVALID), (dict(ldx=63), INVALID),
    (dict(ldy=63), INVALID), (dict(type="none"), UNSUPPORTED), (dict(type=99), UNSUPPORTED),
    (dict(type="e2m1", ldx=65), INVALID), (dict(type="e2m3", ldx=66, ldy=68), INVALID), (dict(sfx=P[3]), INVALID),
    (dict(sfx=P[3], sfy=P[4], ld_sfy=1), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(rows=None), INVALID), (dict(rows=P[1] + 2), MISALIGNED), (dict(y=P[0]), INVALID), (dict(y=P[1]), INVALID),
    (dict(sfx=P[3], sfy=P[3]), INVALID), (dict(sfx=P[3], sfy=P[2]), INVALID), (dict(sfx=P[3], sfy=P[0]), INVALID),
    (dict(m=0), OK), (dict(n=0), OK), (dict(topk=0), OK), (dict(rows_y=0), OK),
])
def test_moe_gather_refusals(kw, want):
    assert gather(**kw) == want


def combine(m=64, n=8, topk=2, x=P[0], ldx=64, rows_x=16, rows=P[1], weights=P[2], y=P[3], ldy=64, tx="bf16",
            ty="bf16"):
    return thl.thl_moe_combine(m, n, topk, x, ldx, rows_x, rows, weights, y, ldy, tx, ty)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(topk=-1), INVALID), (dict(ldx=63), INVALID), (dict(ldy=63), INVALID),
    (dict(tx="e4m3"), UNSUPPORTED), (dict(ty="i32"), UNSUPPORTED), (dict(x=None), INVALID), (dict(rows=None), INVALID),
    (dict(y=None), INVALID), (dict(x=P[0] + 1), MISALIGNED), (dict(weights=P[2] + 2), MISALIGNED),
    (dict(y=P[0]), INVALID), (dict(y=P[1]), INVALID), (dict(y=P[2]), INVALID), (dict(m=0), OK), (dict(n=0), OK),
])
def test_moe_combine_refusals(kw, want):
    assert combine(**kw) == want


def cgrad(m=64, n=8, topk=2, dy=P[0], lddy=64, x=P[1], ldx=64, rows_x=16, rows=P[2], weights=P[3], dx=P[4], lddx=64,
          dw=P[5], tdy="bf16", tx="bf16"):
    return thl.thl_moe_combine_backward(m, n, topk, dy, lddy, x, ldx, rows_x, rows, weights, dx, lddx, dw, tdy, tx)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(lddy=1), INVALID), (dict(ldx=1), INVALID),
    (dict(lddx=1), INVALID), (dict(tdy="e4m3"), UNSUPPORTED), (dict(tx="i32"), UNSUPPORTED), (dict(dy=None), INVALID),
    (dict(x=None), INVALID), (dict(rows=None), INVALID), (dict(weights=None), INVALID), (dict(dx=P[4] + 1), MISALIGNED),
    (dict(dw=P[5] + 2), MISALIGNED), (dict(dx=P[0]), INVALID), (dict(dx=P[1]), INVALID),
    (dict(dx=P[1], lddx=72), INVALID), (dict(dx=P[2]), INVALID), (dict(dx=P[3]), INVALID), (dict(dw=P[0]), INVALID),
    (dict(dw=P[1]), INVALID), (dict(dw=P[4]), INVALID), (dict(dw=P[3]), INVALID), (dict(dx=None, dw=None), OK),
    (dict(n=0), OK), (dict(topk=0), OK),
])
def test_moe_combine_backward_refusals(kw, want):
    assert cgrad(**kw) == want


def w4(m=64, n=4, k=256, w=P[0], ldw=256, scales=P[1], ld_s=2, zeros=P[2], ld_z=2, group=128, ts="f16", x=P[3],
       ldx=256, c=None, ldc=64, d=P[4], ldd=64, beta=0.0, types=("u4", "f16", "f16", "f16", "none"), flags=0,
       bias=None, acc="f32", gs=True, ws=None, size=0):
    ta, tb, tc, td, tbias = types
    dts = thl.make_dtypes(ta, tb, tc, td, tbias, acc)
    sc = thl.thl_group_scales(scales, ld_s, zeros, ld_z, group, D[ts]) if gs else None
    return thl.thl_gemm_w4(m, n, k, w, ldw, sc, x, ldx, c, ldc, d, ldd, 1.0, beta, dts,
                           thl.thl_epilogue(flags, bias, None, 0), ws, size)


LONG = dict(n=17, k=4096, ldw=4096, ldx=4096, ld_s=32, ld_z=32)  # needs a workspace
I4 = ("i4", "bf16", "f32", "f32", "none")
E2 = ("e2m1", "bf16", "f32", "f32", "none")


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(k=-1), INVALID), (dict(gs=False), INVALID),
    (dict(ldw=255), INVALID), (dict(ldw=254), INVALID), (dict(ldx=255), INVALID), (dict(ldd=63), INVALID),
    (dict(beta=1.0, c=P[5], ldc=63), INVALID), (dict(beta=1.0), INVALID), (dict(ld_s=1), INVALID),
    (dict(ld_z=1), INVALID), (dict(zeros=None), INVALID), (dict(w=None), INVALID), (dict(x=None), INVALID),
    (dict(scales=None), INVALID), (dict(d=None), INVALID), (dict(flags=thl.THL_EPI_RELU | thl.THL_EPI_GELU), INVALID),
    (dict(flags=8), INVALID), (dict(flags=thl.THL_EPI_BIAS, types=("u4", "f16", "f16", "f16", "f16")), INVALID),
    (dict(group=0), INVALID), (dict(group=16), UNSUPPORTED), (dict(group=96), UNSUPPORTED),
    (dict(types=I4), UNSUPPORTED),  # signed codes with zero points
    (dict(types=I4, zeros=None, ts="e8m0"), UNSUPPORTED), (dict(types=E2, zeros=None), UNSUPPORTED),
    (dict(ts="f32"), UNSUPPORTED),
    (dict(types=E2, zeros=None, ts="e8m0", group=64), UNSUPPORTED),
    (dict(types=("e4m3", "f16", "f16", "f16", "none")), UNSUPPORTED),
    (dict(types=("u4", "f32", "f16", "f16", "none")), UNSUPPORTED),
    (dict(types=("u4", "f16", "f16", "e4m3", "none")), UNSUPPORTED), (dict(acc="i32"), UNSUPPORTED),
    (dict(m=1 << 27), UNSUPPORTED), (dict(n=1 << 22), UNSUPPORTED),
    (dict(LONG), INVALID), (dict(LONG, ws=P[6], size=8 * 17 * 64 * 4 - 1), INVALID),
    (dict(LONG, ws=P[6] + 2, size=1 << 20), MISALIGNED), (dict(LONG, ws=P[4], size=1 << 20), INVALID),
    (dict(LONG, ws=P[0], size=1 << 20), INVALID), (dict(LONG, ws=P[3], size=1 << 20), INVALID),
    (dict(x=P[3] + 1), MISALIGNED), (dict(d=P[4] + 1), MISALIGNED), (dict(scales=P[1] + 1), MISALIGNED),
    (dict(d=P[0]), INVALID), (dict(d=P[1]), INVALID), (dict(d=P[2]), INVALID), (dict(d=P[3]), INVALID),
    (dict(beta=1.0, c=P[4], ldc=80), INVALID), (dict(m=0), OK), (dict(n=0), OK),
])
def test_gemm_w4_refusals(kw, want):
    assert w4(**kw) == want


@pytest.mark.parametrize("fmt", ["i4", "u4"])
def test_gemm_refuses_integer_nibbles(fmt):
    dts = thl.make_dtypes(fmt, fmt, "f32", "f32")
    assert thl.thl_gemm(64, 64, 64, P[0], 64, "T", P[1], 64, "N", None, 64, P[2], 64, 1.0, 0.0, dts) == UNSUPPORTED


def test_structures_match_the_header():
    assert ctypes.sizeof(thl.thl_group_scales) == 48
    assert ctypes.sizeof(thl.thl_norm_types) == ctypes.sizeof(thl.thl_norm_grad_types) == 16
    assert (D["i4"], D["u4"]) == (12, 13)


def test_torch_forms_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        thl.rmsnorm(x, x[0], x)
    with pytest.raises(ValueError):
        thl.rmsnorm_backward(x, x, x[0], x)
    with pytest.raises(ValueError):
        thl.moe_sort(i, 4, i, i[0])
    with pytest.raises(ValueError):
        thl.moe_gather(x, i, x)
    with pytest.raises(ValueError):
        thl.moe_combine(x, i, x)
    with pytest.raises(ValueError):
        thl.moe_combine_backward(x, x, i, x)
    with pytest.raises(ValueError):
        thl.gemm_w4(x.to(torch.uint8), x, x, scales=x, group=32)
