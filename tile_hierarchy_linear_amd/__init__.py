"""Python binding of libthl.so: the MI355X tiled GEMM with a fused epilogue,
the operators around a layer's products (norm, tokens by expert, 4-bit
weights), and the Shape:Stride layout module.

Argument marshalling only: every step of the GEMM and of the operators runs
in the library's HIP kernels, and the layout algebra in its C++.  The names
match the C entry points of ``include/thl.h``.  Importing this module fails
loudly when the built library is missing, and the torch-tensor forms when the
host module behind them does not load; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libthl.so")

THL_OK, THL_ERR_INVALID, THL_ERR_UNSUPPORTED, THL_ERR_MISALIGNED, THL_ERR_HIP, THL_ERR_UNDEFINED = (
    0, -1, -2, -3, -4, -5)
THL_ERR_SCRATCH = -6
THL_OP_N, THL_OP_T = 0, 1
DTYPES = {"f32": 0, "f16": 1, "bf16": 2, "i8": 3, "i32": 4, "e4m3": 5, "e2m1": 6, "e8m0": 7, "none": 8, "e5m2": 9,
          "e2m3": 10, "e3m2": 11, "i4": 12, "u4": 13}
THL_EPI_NONE, THL_EPI_BIAS, THL_EPI_RELU, THL_EPI_GELU = 0, 1, 2, 4


class ThlError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {thl_status_string(status)} ({status})" if what else thl_status_string(status))


class thl_dtypes(ctypes.Structure):
    _fields_ = [("a", ctypes.c_int), ("b", ctypes.c_int), ("c", ctypes.c_int), ("d", ctypes.c_int),
                ("bias", ctypes.c_int), ("acc", ctypes.c_int)]


class thl_epilogue(ctypes.Structure):
    _fields_ = [("flags", ctypes.c_uint), ("bias", ctypes.c_void_p), ("sfd", ctypes.c_void_p),
                ("ld_sfd", ctypes.c_int64)]


class thl_scales(ctypes.Structure):
    _fields_ = [("a_scale", ctypes.c_float), ("b_scale", ctypes.c_float), ("sfa", ctypes.c_void_p),
                ("ld_sfa", ctypes.c_int64), ("sfb", ctypes.c_void_p), ("ld_sfb", ctypes.c_int64)]


class thl_group_problem(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("A", ctypes.c_void_p), ("lda", ctypes.c_int64), ("B", ctypes.c_void_p), ("ldb", ctypes.c_int64),
                ("C", ctypes.c_void_p), ("ldc", ctypes.c_int64), ("D", ctypes.c_void_p), ("ldd", ctypes.c_int64),
                ("bias", ctypes.c_void_p), ("sfa", ctypes.c_void_p), ("ld_sfa", ctypes.c_int64),
                ("sfb", ctypes.c_void_p), ("ld_sfb", ctypes.c_int64)]


class thl_norm_types(ctypes.Structure):
    _fields_ = [("x", ctypes.c_int), ("r", ctypes.c_int), ("w", ctypes.c_int), ("y", ctypes.c_int)]


class thl_norm_grad_types(ctypes.Structure):
    _fields_ = [("s", ctypes.c_int), ("w", ctypes.c_int), ("g", ctypes.c_int), ("dw", ctypes.c_int)]


class thl_group_scales(ctypes.Structure):
    _fields_ = [("scales", ctypes.c_void_p), ("ld_scales", ctypes.c_int64), ("zeros", ctypes.c_void_p),
                ("ld_zeros", ctypes.c_int64), ("group", ctypes.c_int64), ("type", ctypes.c_int)]


def _load():
    # One HIP runtime per process.  torch ships its own libamdhip64 and asks
    # for it by its unversioned name, so loading libthl first (which pulls in
    # the system libamdhip64.so.7) would leave two runtimes in the process and
    # device pointers from one invalid in the other.  Importing torch first
    # makes libthl bind to torch's runtime.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                          "or python tile_hierarchy_linear_amd/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    i64, vp, cp, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_char_p, ctypes.c_size_t
    p64 = ctypes.POINTER(ctypes.c_int64)
    lib.thl_gemm.argtypes = [i64, i64, i64, vp, i64, ctypes.c_int, vp, i64, ctypes.c_int, vp, i64, vp, i64,
                             ctypes.c_float, ctypes.c_float, ctypes.POINTER(thl_dtypes),
                             ctypes.POINTER(thl_epilogue), ctypes.POINTER(thl_scales), vp]
    lib.thl_gemm.restype = ctypes.c_int
    lib.thl_gemm_noalloc.argtypes = lib.thl_gemm.argtypes
    lib.thl_gemm_noalloc.restype = ctypes.c_int
    lib.thl_gemm_batched.argtypes = [i64, i64, i64, i64, vp, i64, i64, ctypes.c_int, vp, i64, i64, ctypes.c_int,
                                     vp, i64, i64, vp, i64, i64, ctypes.c_float, ctypes.c_float,
                                     ctypes.POINTER(thl_dtypes), ctypes.POINTER(thl_epilogue), i64,
                                     ctypes.POINTER(thl_scales), i64, i64, vp]
    lib.thl_gemm_batched.restype = ctypes.c_int
    lib.thl_gemm_grouped.argtypes = [i64, ctypes.POINTER(thl_group_problem), vp, ctypes.c_int, ctypes.c_int,
                                     ctypes.c_float, ctypes.c_float, ctypes.POINTER(thl_dtypes),
                                     ctypes.POINTER(thl_epilogue), ctypes.POINTER(thl_scales), vp]
    lib.thl_gemm_grouped.restype = ctypes.c_int
    f32, i32 = ctypes.c_float, ctypes.c_int
    lib.thl_rmsnorm.argtypes = [i64, i64, vp, i64, vp, i64, vp, i64, vp, f32, f32, vp, i64, vp, i64,
                                ctypes.POINTER(thl_norm_types), vp]
    lib.thl_rmsnorm_backward_workspace.argtypes = [i64, i64]
    lib.thl_rmsnorm_backward.argtypes = [i64, i64, vp, i64, vp, i64, vp, i64, vp, f32, vp, i64, vp, vp, sz,
                                         ctypes.POINTER(thl_norm_grad_types), vp]
    lib.thl_moe_sort_workspace.argtypes = [i64, i64, i64]
    lib.thl_moe_sort.argtypes = [i64, i64, i64, vp, i64, i32, vp, vp, vp, vp, sz, vp]
    lib.thl_moe_gather.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, vp]
    lib.thl_moe_combine.argtypes = [i64, i64, i64, vp, i64, i64, vp, vp, vp, i64, i32, i32, vp]
    lib.thl_moe_combine_backward.argtypes = [i64, i64, i64, vp, i64, vp, i64, i64, vp, vp, vp, i64, vp, i32, i32, vp]
    lib.thl_gemm_w4.argtypes = [i64, i64, i64, vp, i64, ctypes.POINTER(thl_group_scales), vp, i64, vp, i64, vp, i64,
                                f32, f32, ctypes.POINTER(thl_dtypes), ctypes.POINTER(thl_epilogue), vp, sz, vp]
    lib.thl_gemm_w4_workspace.argtypes = [i64, i64, i64]
    for name in ("rmsnorm", "rmsnorm_backward", "moe_sort", "moe_gather", "moe_combine", "moe_combine_backward",
                 "gemm_w4"):
        getattr(lib, "thl_" + name).restype = ctypes.c_int
    for name in ("rmsnorm_backward_workspace", "moe_sort_workspace", "gemm_w4_workspace"):
        getattr(lib, "thl_" + name).restype = sz
    lib.thl_status_string.argtypes = [ctypes.c_int]
    lib.thl_status_string.restype = cp
    lib.thl_last_variant.restype = cp
    lib.thl_last_splits.restype = ctypes.c_int
    lib.thl_variant_count.restype = ctypes.c_int
    lib.thl_variant_name.argtypes = [ctypes.c_int]
    lib.thl_variant_name.restype = cp
    lib.thl_kernel_index_map.argtypes = [cp, p64, i64, p64, p64]
    lib.thl_kernel_index_map.restype = ctypes.c_int
    lib.thl_kernel_index_map_names.restype = cp
    for name in ("coalesce",):
        getattr(lib, "thl_layout_" + name).argtypes = [cp, ctypes.c_char_p, sz]
    for name in ("composition", "logical_divide", "zipped_divide", "tiled_divide", "flat_divide"):
        getattr(lib, "thl_layout_" + name).argtypes = [cp, cp, ctypes.c_char_p, sz]
    lib.thl_layout_complement.argtypes = [cp, i64, ctypes.c_char_p, sz]
    lib.thl_layout_local_tile.argtypes = [cp, cp, i64, p64, ctypes.c_char_p, sz]
    lib.thl_layout_local_partition.argtypes = [cp, cp, i64, p64, ctypes.c_char_p, sz]
    lib.thl_layout_eval.argtypes = [cp, p64, i64, p64]
    lib.thl_layout_eval_coord.argtypes = [cp, cp, p64]
    lib.thl_layout_info.argtypes = [cp, p64, p64, p64]
    lib.thl_layout_mode.argtypes = [cp, i64, ctypes.c_char_p, sz]
    lib.thl_swizzle_eval.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, cp, p64, i64, p64]
    return lib


_lib = _load()


def library():
    """The loaded ctypes library (for symbol checks)."""
    return _lib


# ------------------------------------------------------------------ status

def thl_status_string(status: int) -> str:
    return _lib.thl_status_string(int(status)).decode()


def thl_last_variant() -> str:
    return _lib.thl_last_variant().decode()


def thl_last_splits() -> int:
    return int(_lib.thl_last_splits())


def thl_variant_count() -> int:
    return int(_lib.thl_variant_count())


def thl_variant_name(i: int) -> str | None:
    r = _lib.thl_variant_name(int(i))
    return r.decode() if r else None


def variants() -> list[str]:
    return [thl_variant_name(i) for i in range(thl_variant_count())]


# ------------------------------------------------------------------ GEMM

def _dt(x) -> int:
    return DTYPES[x] if isinstance(x, str) else int(x)


def make_dtypes(a, b=None, c="f32", d="f32", bias="none", acc=None) -> thl_dtypes:
    b = a if b is None else b
    if acc is None:
        acc = "i32" if _dt(a) == DTYPES["i8"] else "f32"
    return thl_dtypes(_dt(a), _dt(b), _dt(c), _dt(d), _dt(bias), _dt(acc))


def thl_gemm(m, n, k, A, lda, opA, B, ldb, opB, C, ldc, D, ldd, alpha, beta, dtypes, epilogue=None,
             scales=None, stream=None) -> int:
    """Direct call of the C entry point.  Pointers are integers (device
    addresses) or None; opA/opB are THL_OP_N/THL_OP_T or 'N'/'T'; `stream` is
    a hipStream_t as an integer (torch: ``torch.cuda.current_stream().cuda_stream``).
    Returns the thl_status code."""
    opa = THL_OP_T if opA in ("T", THL_OP_T) else (THL_OP_N if opA in ("N", THL_OP_N) else int(opA))
    opb = THL_OP_T if opB in ("T", THL_OP_T) else (THL_OP_N if opB in ("N", THL_OP_N) else int(opB))
    return int(_lib.thl_gemm(int(m), int(n), int(k), A, int(lda), opa, B, int(ldb), opb, C, int(ldc), D,
                             int(ldd), float(alpha), float(beta), ctypes.byref(dtypes),
                             ctypes.byref(epilogue) if epilogue is not None else None,
                             ctypes.byref(scales) if scales is not None else None, stream))


def bind_thl_gemm(m, n, k, A, lda, opA, B, ldb, opB, C, ldc, D, ldd, alpha, beta, dtypes, epilogue=None,
                  scales=None, stream=None, entry="thl_gemm"):
    """The arguments of one thl_gemm (or thl_gemm_noalloc) call, marshalled
    once: returns a callable that issues exactly that call and returns its
    status.  For loops that repeat one call (timing), where rebuilding the
    ctypes arguments each time would cost more host time than a small
    kernel runs."""
    opa = THL_OP_T if opA in ("T", THL_OP_T) else (THL_OP_N if opA in ("N", THL_OP_N) else int(opA))
    opb = THL_OP_T if opB in ("T", THL_OP_T) else (THL_OP_N if opB in ("N", THL_OP_N) else int(opB))
    fn = getattr(_lib, entry)
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    args = (i64(m), i64(n), i64(k), vp(A), i64(lda), ctypes.c_int(opa), vp(B), i64(ldb), ctypes.c_int(opb), vp(C),
            i64(ldc), vp(D), i64(ldd), ctypes.c_float(alpha), ctypes.c_float(beta), ctypes.byref(dtypes),
            ctypes.byref(epilogue) if epilogue is not None else None,
            ctypes.byref(scales) if scales is not None else None, vp(stream))
    keep = (dtypes, epilogue, scales)

    def call() -> int:
        return fn(*args)

    call.keep = keep  # the structures the byref arguments point into
    return call


def thl_gemm_noalloc(m, n, k, A, lda, opA, B, ldb, opB, C, ldc, D, ldd, alpha, beta, dtypes, epilogue=None,
                     scales=None, stream=None) -> int:
    """Direct call of the no-allocation C entry point (arguments as for thl_gemm)."""
    opa = THL_OP_T if opA in ("T", THL_OP_T) else (THL_OP_N if opA in ("N", THL_OP_N) else int(opA))
    opb = THL_OP_T if opB in ("T", THL_OP_T) else (THL_OP_N if opB in ("N", THL_OP_N) else int(opB))
    return int(_lib.thl_gemm_noalloc(int(m), int(n), int(k), A, int(lda), opa, B, int(ldb), opb, C, int(ldc), D,
                                     int(ldd), float(alpha), float(beta), ctypes.byref(dtypes),
                                     ctypes.byref(epilogue) if epilogue is not None else None,
                                     ctypes.byref(scales) if scales is not None else None, stream))


def thl_gemm_batched(batch, m, n, k, A, lda, stride_a, opA, B, ldb, stride_b, opB, C, ldc, stride_c, D, ldd,
                     stride_d, alpha, beta, dtypes, epilogue=None, stride_bias=0, scales=None, stride_sfa=0,
                     stride_sfb=0, stream=None) -> int:
    """Direct call of the batched C entry point (arguments as for thl_gemm,
    plus the batch count and per-array strides in elements)."""
    opa = THL_OP_T if opA in ("T", THL_OP_T) else (THL_OP_N if opA in ("N", THL_OP_N) else int(opA))
    opb = THL_OP_T if opB in ("T", THL_OP_T) else (THL_OP_N if opB in ("N", THL_OP_N) else int(opB))
    return int(_lib.thl_gemm_batched(int(batch), int(m), int(n), int(k), A, int(lda), int(stride_a), opa, B,
                                     int(ldb), int(stride_b), opb, C, int(ldc), int(stride_c), D, int(ldd),
                                     int(stride_d), float(alpha), float(beta), ctypes.byref(dtypes),
                                     ctypes.byref(epilogue) if epilogue is not None else None, int(stride_bias),
                                     ctypes.byref(scales) if scales is not None else None, int(stride_sfa),
                                     int(stride_sfb), stream))


def thl_gemm_grouped(count, problems, problems_dev, opA, opB, alpha, beta, dtypes, epilogue=None, scales=None,
                     stream=None) -> int:
    """Direct call of the grouped C entry point: `problems` is a ctypes array
    of thl_group_problem (host), `problems_dev` the device address of a copy
    of the same bytes."""
    opa = THL_OP_T if opA in ("T", THL_OP_T) else THL_OP_N
    opb = THL_OP_T if opB in ("T", THL_OP_T) else THL_OP_N
    return int(_lib.thl_gemm_grouped(int(count), problems, problems_dev, opa, opb, float(alpha), float(beta),
                                     ctypes.byref(dtypes), ctypes.byref(epilogue) if epilogue is not None else None,
                                     ctypes.byref(scales) if scales is not None else None, stream))


def gemm(A, B, D, *, m, n, k, lda, ldb, ldd, op_a="T", op_b="N", C=None, ldc=0, alpha=1.0, beta=0.0,
         type_ab="bf16", type_c="f32", type_d="f32", bias=None, type_bias="none", act="none",
         a_scale=1.0, b_scale=1.0, sfa=None, ld_sfa=0, sfb=None, ld_sfb=0, stream=None, type_b=None,
         sfd=None, ld_sfd=0) -> str:
    """Torch-tensor convenience around thl_gemm: takes device tensors holding
    the stored bits, issues on the current stream, raises ThlError on a
    non-OK status and returns the name of the kernel variant launched.
    type_ab is A's format and B's unless type_b is given; sfd / ld_sfd take
    the generated scales of an MX-format D."""
    import torch

    def ptr(t):
        return None if t is None else t.data_ptr()

    flags = (THL_EPI_BIAS if bias is not None else 0) | {"none": 0, "relu": THL_EPI_RELU,
                                                         "gelu": THL_EPI_GELU}[act]
    epi = thl_epilogue(flags, ptr(bias), ptr(sfd), int(ld_sfd))
    sc = thl_scales(float(a_scale), float(b_scale), ptr(sfa), int(ld_sfa), ptr(sfb), int(ld_sfb))
    dts = make_dtypes(type_ab, type_b or type_ab, type_c, type_d, type_bias)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    st = thl_gemm(m, n, k, ptr(A), lda, op_a, ptr(B), ldb, op_b, ptr(C), ldc or max(1, m), ptr(D), ldd,
                  alpha, beta, dts, epi, sc, stream)
    if st != THL_OK:
        raise ThlError(st, "thl_gemm")
    return thl_last_variant()


def thl_kernel_index_map(name: str, points, params=()) -> list[tuple[int, int]]:
    """Evaluate a kernel index map at (x, y) points on the host."""
    pts = list(points)
    n = len(pts)
    arr_in = (ctypes.c_int64 * (2 * max(n, 1)))()
    for t, (x, y) in enumerate(pts):
        arr_in[2 * t], arr_in[2 * t + 1] = int(x), int(y)
    arr_out = (ctypes.c_int64 * (2 * max(n, 1)))()
    par = (ctypes.c_int64 * max(len(params), 1))(*[int(p) for p in params]) if params else None
    st = _lib.thl_kernel_index_map(name.encode(), par, n, arr_in, arr_out)
    if st != THL_OK:
        raise ThlError(st, f"thl_kernel_index_map({name})")
    return [(arr_out[2 * t], arr_out[2 * t + 1]) for t in range(n)]


def thl_kernel_index_map_names() -> list[str]:
    return _lib.thl_kernel_index_map_names().decode().split(",")


# ------------------------------------------------------------------ operators around the products
# Direct calls of the C entry points, arguments as in include/thl.h (pointers
# are integers or None, the types structures objects, formats names or codes).

def _ref(structure):
    return ctypes.byref(structure) if structure is not None else None


def thl_rmsnorm(m, n, X, ldx, R, ldr, S, lds, W, eps, y_scale, Y, ldy, sfy, ld_sfy, types, stream=None) -> int:
    return _lib.thl_rmsnorm(m, n, X, ldx, R, ldr, S, lds, W, eps, y_scale, Y, ldy, sfy, ld_sfy, _ref(types), stream)


def thl_rmsnorm_backward_workspace(m, n) -> int:
    return _lib.thl_rmsnorm_backward_workspace(m, n)


def thl_rmsnorm_backward(m, n, S, lds, DY, lddy, DR, lddr, W, eps, DX, lddx, DW, workspace, workspace_bytes, types,
                         stream=None) -> int:
    return _lib.thl_rmsnorm_backward(m, n, S, lds, DY, lddy, DR, lddr, W, eps, DX, lddx, DW, workspace,
                                     workspace_bytes, _ref(types), stream)


def thl_moe_sort_workspace(n, topk, experts) -> int:
    return _lib.thl_moe_sort_workspace(n, topk, experts)


def thl_moe_sort(n, topk, experts, ids, ld_ids, ids_bytes, rows, offsets, order, workspace, workspace_bytes,
                 stream=None) -> int:
    return _lib.thl_moe_sort(n, topk, experts, ids, ld_ids, ids_bytes, rows, offsets, order, workspace,
                             workspace_bytes, stream)


def thl_moe_gather(m, n, topk, X, ldx, sfx, ld_sfx, rows, rows_y, Y, ldy, sfy, ld_sfy, type, stream=None) -> int:
    return _lib.thl_moe_gather(m, n, topk, X, ldx, sfx, ld_sfx, rows, rows_y, Y, ldy, sfy, ld_sfy, _dt(type), stream)


def thl_moe_combine(m, n, topk, X, ldx, rows_x, rows, weights, Y, ldy, type_x, type_y, stream=None) -> int:
    return _lib.thl_moe_combine(m, n, topk, X, ldx, rows_x, rows, weights, Y, ldy, _dt(type_x), _dt(type_y), stream)


def thl_moe_combine_backward(m, n, topk, DY, lddy, X, ldx, rows_x, rows, weights, DX, lddx, dweights, type_dy, type_x,
                             stream=None) -> int:
    return _lib.thl_moe_combine_backward(m, n, topk, DY, lddy, X, ldx, rows_x, rows, weights, DX, lddx, dweights,
                                         _dt(type_dy), _dt(type_x), stream)


def thl_gemm_w4_workspace(m, n, k) -> int:
    return _lib.thl_gemm_w4_workspace(m, n, k)


def thl_gemm_w4(m, n, k, W, ldw, scales, X, ldx, C, ldc, D, ldd, alpha, beta, dtypes, epilogue=None, workspace=None,
                workspace_bytes=0, stream=None) -> int:
    return _lib.thl_gemm_w4(m, n, k, W, ldw, _ref(scales), X, ldx, C, ldc, D, ldd, alpha, beta, _ref(dtypes),
                            _ref(epilogue), workspace, workspace_bytes, stream)


# Torch-tensor forms.  An array of tokens is a (tokens, features) tensor whose
# features are contiguous (rows may be pitched); outputs are tensors that the
# caller made, so that serving loops and graphs reuse them.  They issue on the
# current stream of the tensors' device, take their workspaces from torch on
# that stream, and raise ValueError for a tensor of the wrong shape, type or
# device, ThlError for what the library refuses and torch.OutOfMemoryError
# where a workspace does not fit.  Autograd does not see them: a tensor that
# requires a gradient raises ValueError where gradients are recorded (call them
# under torch.no_grad() or inside a torch.autograd.Function, with the *_backward
# forms as its backward), and outputs count as written in place.  The tensors are read and checked in
# csrc/torch_ops.cpp: in Python that took as long as the launch.


class _NoTorchForms:
    """In place of the host module where it does not load: each form raises."""

    def __init__(self, reason):
        self._reason = reason

    def __getattr__(self, name):
        raise ImportError(f"thl.{name} takes torch tensors through {os.path.join(_HERE, '_torch_ops.so')}, which does "
                          "not load; run __graft_entry__.build() or python tile_hierarchy_linear_amd/build.py "
                          f"({self._reason})")


try:
    from . import _torch_ops as _ops
except ImportError as e:  # not built, or for another torch; the C entry points above do not need it
    _ops = _NoTorchForms(str(e))


def rmsnorm(x, w, y, *, eps=1e-6, residual=None, residual_out=None, scale=1.0, sf=None):
    """y = the root-mean-square norm of x (+ residual) times w, in y's format; the sum goes to residual_out.
    An fp8 y holds y * (1 / scale), or MX blocks when sf takes their E8M0 scales; a uint8 y of ceil(features / 2)
    columns holds E2M1 MX blocks.  Returns y."""
    status = _ops.rmsnorm(x, w, y, eps, residual, residual_out, scale, sf)
    if status:
        raise ThlError(status, "thl_rmsnorm")
    return y


def rmsnorm_backward(s, dy, w, dx, dw=None, *, eps=1e-6, dres=None):
    """The gradients of rmsnorm for the s it normalised: dx (of x and residual alike; dres, the gradient that
    reaches s past the norm, is added) and, if wanted, dw."""
    status = _ops.rmsnorm_backward(s, dy, w, dx, dw, eps, dres)
    if status:
        raise ThlError(status, "thl_rmsnorm_backward")


def moe_sort(ids, experts, rows, offsets, *, order=None):
    """The stable order of (tokens, choices) int32 or int64 expert ids: each choice's row (int32, -1 when its id is
    outside 0 .. experts-1), each expert's first row (experts + 1 of them), and each row's flat choice.  A grouped
    product over the experts takes the offsets on the host (offsets.tolist() waits for them)."""
    status = _ops.moe_sort(ids, experts, rows, offsets, order)
    if status:
        raise ThlError(status, "thl_moe_sort")


def moe_gather(x, rows, y, *, sf=None, sf_y=None, type_x=None):
    """y[rows[j, t]] = x[j], bit for bit, with the rows of block scales sf likewise into sf_y.  type_x: "e2m1", "i4" or
    "u4" (two codes a byte), "e4m3", "e5m2" or "i8" where a one-byte tensor's type does not say it; fp6 rows go through
    thl_moe_gather.  Returns y."""
    status = _ops.moe_gather(x, rows, y, sf, sf_y, type_x)
    if status:
        raise ThlError(status, "thl_moe_gather")
    return y


def moe_combine(x, rows, y, *, weights=None):
    """y[j] = the sum over t of weights[j, t] * x[rows[j, t]] (fp32 weights, ones without).  Returns y."""
    status = _ops.moe_combine(x, rows, y, weights)
    if status:
        raise ThlError(status, "thl_moe_combine")
    return y


def moe_combine_backward(dy, x, rows, weights, dx=None, dweights=None):
    """moe_combine's gradients: dx (x's type; rows that no choice has are left as they were) and dweights (fp32),
    each if wanted.  Without dweights x may be None (dx gives the rows)."""
    status = _ops.moe_combine_backward(dy, x, rows, weights, dx, dweights)
    if status:
        raise ThlError(status, "thl_moe_combine_backward")


def gemm_w4(w, x, d, *, scales, group, type_w="u4", zeros=None, c=None, alpha=1.0, beta=0.0, bias=None, act="none"):
    """d = act(alpha * x @ W^T + beta * c + bias) for (features, K / 2) uint8 weights of two codes a byte ("u4" with
    uint8 zero points, "i4", or "e2m1" with E8M0 scales), (features, groups) scales and (tokens, K) x.  Returns d."""
    status = _ops.gemm_w4(w, x, d, scales, group, type_w, zeros, c, alpha, beta, bias, act)
    if status:
        raise ThlError(status, "thl_gemm_w4")
    return d


# ------------------------------------------------------------------ layouts

_CAP = 4096


def _text_call(fn, *args) -> str:
    buf = ctypes.create_string_buffer(_CAP)
    st = fn(*args, buf, _CAP)
    if st != THL_OK:
        raise ThlError(st, fn.__name__)
    return buf.value.decode()


def _enc(x) -> bytes:
    return x.encode() if isinstance(x, str) else x


def _tiler(t) -> bytes:
    return _enc(t if isinstance(t, str) else ";".join(t))


def thl_layout_coalesce(a: str) -> str:
    return _text_call(_lib.thl_layout_coalesce, _enc(a))


def thl_layout_composition(a: str, b) -> str:
    return _text_call(_lib.thl_layout_composition, _enc(a), _tiler(b))


def thl_layout_complement(a: str, cotarget: int) -> str:
    return _text_call(_lib.thl_layout_complement, _enc(a), int(cotarget))


def thl_layout_logical_divide(a: str, b) -> str:
    return _text_call(_lib.thl_layout_logical_divide, _enc(a), _tiler(b))


def thl_layout_zipped_divide(a: str, tiler) -> str:
    return _text_call(_lib.thl_layout_zipped_divide, _enc(a), _tiler(tiler))


def thl_layout_tiled_divide(a: str, tiler) -> str:
    return _text_call(_lib.thl_layout_tiled_divide, _enc(a), _tiler(tiler))


def thl_layout_flat_divide(a: str, tiler) -> str:
    return _text_call(_lib.thl_layout_flat_divide, _enc(a), _tiler(tiler))


def thl_layout_local_tile(a: str, tiler, tile: int) -> tuple[int, str]:
    off = ctypes.c_int64(0)
    s = _text_call(_lib.thl_layout_local_tile, _enc(a), _tiler(tiler), int(tile), ctypes.byref(off))
    return off.value, s


def thl_layout_local_partition(a: str, threads: str, tid: int) -> tuple[int, str]:
    off = ctypes.c_int64(0)
    s = _text_call(_lib.thl_layout_local_partition, _enc(a), _enc(threads), int(tid), ctypes.byref(off))
    return off.value, s


def thl_layout_eval(a: str, coords) -> list[int]:
    cs = [int(c) for c in coords]
    n = len(cs)
    arr = (ctypes.c_int64 * max(n, 1))(*cs)
    out = (ctypes.c_int64 * max(n, 1))()
    st = _lib.thl_layout_eval(_enc(a), arr, n, out)
    if st != THL_OK:
        raise ThlError(st, "thl_layout_eval")
    return list(out[:n])


def thl_layout_eval_coord(a: str, coord: str) -> int:
    out = ctypes.c_int64(0)
    st = _lib.thl_layout_eval_coord(_enc(a), _enc(coord), ctypes.byref(out))
    if st != THL_OK:
        raise ThlError(st, "thl_layout_eval_coord")
    return out.value


def thl_layout_info(a: str) -> tuple[int, int, int]:
    s, c, r = ctypes.c_int64(0), ctypes.c_int64(0), ctypes.c_int64(0)
    st = _lib.thl_layout_info(_enc(a), ctypes.byref(s), ctypes.byref(c), ctypes.byref(r))
    if st != THL_OK:
        raise ThlError(st, "thl_layout_info")
    return s.value, c.value, r.value


def thl_layout_mode(a: str, i: int) -> str:
    return _text_call(_lib.thl_layout_mode, _enc(a), int(i))


def thl_swizzle_eval(b: int, m: int, s: int, a: str, coords) -> list[int]:
    cs = [int(c) for c in coords]
    n = len(cs)
    arr = (ctypes.c_int64 * max(n, 1))(*cs)
    out = (ctypes.c_int64 * max(n, 1))()
    st = _lib.thl_swizzle_eval(int(b), int(m), int(s), _enc(a), arr, n, out)
    if st != THL_OK:
        raise ThlError(st, "thl_swizzle_eval")
    return list(out[:n])
