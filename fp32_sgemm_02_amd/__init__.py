"""fp32_sgemm_02_amd -- single-precision GEMM for AMD Instinct MI355X (gfx950).

C = alpha * (A * B) + beta * C on row-major fp32 matrices, computed by the
hand-written HIP kernels of ``libfp32sgemm.so`` (C ABI: include/fp32_sgemm.h).
This module only marshals arguments: every step of the product runs in the
library's GPU kernels.  PyTorch supplies device memory and streams.

The operation is the SGEMM of "a CUDA matmul" (plasmient.com labs) section 00
and "The GEMM Scrapbook" introduction: A is M x K, B is K x N, C is M x N, and
every cell of C is the dot product of a row of A and a column of B.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

__all__ = [
    "sgemm", "sgemm_ex", "sgemm_op", "sgemm_op_noalloc", "sgemm_cblas", "sgemm_epilogue", "sgemm_strided_batched",
    "sgemm_mixed", "gemm", "gemm_batched", "gemm_mixed", "linear", "linear_backward", "moe",
    "sgemm_linear", "sgemm_linear_backward", "sgemm_moe", "select", "tile_count", "tile_info", "status_string",
    "version", "workspace_release", "plan", "SgemmConfig", "TileDesc", "SgemmError", "LIB_PATH",
    "VARIANT_AUTO", "VARIANT_MFMA", "VARIANT_VALU", "VARIANT_SKINNY", "VARIANT_MFMA16",
    "VARIANT_GENERIC16", "VARIANT_SMALL", "DTYPE_F32", "DTYPE_BF16", "DTYPE_F16", "FLAG_SCALAR_IO", "FLAG_UNTUNED", "FLAG_STREAMK",
    "TILE_WHOLE", "TILE_DIRECT", "TILE_TRANS_B", "TILE_TRANS_A", "TILE_STREAMK",
    "ACT_NONE", "ACT_RELU", "ACT_SILU", "ACT_GELU_ERF", "ACT_GELU_TANH",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp32sgemm.so")

VARIANT_AUTO, VARIANT_MFMA, VARIANT_VALU, VARIANT_SKINNY = 0, 1, 2, 3
VARIANT_MFMA16, VARIANT_GENERIC16, VARIANT_SMALL = 4, 5, 6
DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2
FLAG_SCALAR_IO = 0x1
FLAG_UNTUNED = 0x2
FLAG_STREAMK = 0x4
TILE_WHOLE = 0x1
TILE_DIRECT = 0x2
TILE_TRANS_B = 0x4
TILE_TRANS_A = 0x8
TILE_STREAMK = 0x10
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU_ERF, ACT_GELU_TANH = 0, 1, 2, 3, 4


class SgemmConfig(ctypes.Structure):
    """Mirror of ``sgemm_config``."""
    _fields_ = [("variant", ctypes.c_int), ("tile", ctypes.c_int),
                ("flags", ctypes.c_int), ("group_m", ctypes.c_int)]


class TileDesc(ctypes.Structure):
    """Mirror of ``sgemm_tile_desc``."""
    _fields_ = [(n, ctypes.c_int) for n in
                ("bm", "bn", "bk", "wm", "wn", "tm", "tn", "threads", "lds_bytes", "stages", "flags")]

    def as_dict(self) -> dict:
        return {n: getattr(self, n) for n, _ in self._fields_}


class SgemmError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(f"sgemm status {status}: {status_string(status)}")


_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -m fp32_sgemm_02_amd.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    i, f, p = ctypes.c_int, ctypes.c_float, ctypes.c_void_p
    lib.sgemm.restype = i
    lib.sgemm.argtypes = [i, i, i, f, p, i, p, i, f, p, i, p]
    lib.sgemm_ex.restype = i
    lib.sgemm_ex.argtypes = [i, i, i, f, p, i, p, i, f, p, i, p, ctypes.POINTER(SgemmConfig)]
    lib.sgemm_op.restype = i
    lib.sgemm_op.argtypes = [i, i, i, i, i, f, p, i, p, i, f, p, i, p]
    lib.sgemm_op_ex.restype = i
    lib.sgemm_op_ex.argtypes = [i, i, i, i, i, f, p, i, p, i, f, p, i, p,
                                ctypes.POINTER(SgemmConfig)]
    lib.sgemm_op_ex_noalloc.restype = i
    lib.sgemm_op_ex_noalloc.argtypes = lib.sgemm_op_ex.argtypes
    lib.sgemm_select.restype = i
    lib.sgemm_select.argtypes = [i, i, i, p, i, p, i, p, i, ctypes.POINTER(SgemmConfig)]
    ll = ctypes.c_longlong
    lib.sgemm_epilogue.restype = i
    lib.sgemm_epilogue.argtypes = [i, i, i, i, i, f, p, i, p, i, f, p, i, p, i, p]
    lib.sgemm_epilogue_ex.restype = i
    lib.sgemm_epilogue_ex.argtypes = lib.sgemm_epilogue.argtypes + [ctypes.POINTER(SgemmConfig)]
    lib.sgemm_strided_batched.restype = i
    lib.sgemm_strided_batched.argtypes = [i, i, i, i, i, f, p, i, ll, p, i, ll, f, p, i, ll, i, p]
    lib.sgemm_strided_batched_ex.restype = i
    lib.sgemm_strided_batched_ex.argtypes = (lib.sgemm_strided_batched.argtypes +
                                             [ctypes.POINTER(SgemmConfig)])
    lib.sgemm_mixed.restype = i
    lib.sgemm_mixed.argtypes = [i, i, i, i, i, i, f, p, i, p, i, f, p, i, p]
    lib.sgemm_mixed_ex.restype = i
    lib.sgemm_mixed_ex.argtypes = lib.sgemm_mixed.argtypes + [ctypes.POINTER(SgemmConfig)]
    lib.sgemm_linear.restype = i
    lib.sgemm_linear.argtypes = [i, i, i, i, p, i, p, i, p, p, i, i, p, i, p, i, p]
    lib.sgemm_linear_backward.restype = i
    lib.sgemm_linear_backward.argtypes = [i, i, i, i, p, i, p, i, i, p, i, p, i, p, i, p, i, p, p]
    lib.sgemm_moe.restype = i
    lib.sgemm_moe.argtypes = [i, i, i, i, i, i, i, i, i, p, i, p, i, p, i, ll, p, i, ll, p, i, p, p, p]
    lib.sgemm_cblas.restype = i
    lib.sgemm_cblas.argtypes = [i, i, i, i, i, i, f, p, i, p, i, f, p, i, p]
    lib.sgemm_op_plan.restype = i
    lib.sgemm_op_plan.argtypes = [i, i, i, i, i, p, i, p, i, p, i, ctypes.POINTER(SgemmConfig),
                                  ctypes.POINTER(i), ctypes.POINTER(i)]
    lib.sgemm_plan.restype = i
    lib.sgemm_plan.argtypes = [i, i, i, p, i, p, i, p, i, ctypes.POINTER(SgemmConfig),
                               ctypes.POINTER(i), ctypes.POINTER(i)]
    lib.sgemm_tile_count.restype = i
    lib.sgemm_tile_count.argtypes = [i]
    lib.sgemm_tile_info.restype = i
    lib.sgemm_tile_info.argtypes = [i, i, ctypes.POINTER(TileDesc)]
    lib.sgemm_status_string.restype = ctypes.c_char_p
    lib.sgemm_status_string.argtypes = [i]
    lib.sgemm_version.restype = i
    lib.sgemm_version.argtypes = []
    lib.sgemm_workspace_release.restype = i
    lib.sgemm_workspace_release.argtypes = []
    _lib = lib
    return lib


def sgemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> int:
    """Raw C-ABI call: A, B, C are device addresses (int) or None; returns the status."""
    return _load().sgemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def sgemm_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None,
             cfg: SgemmConfig | None = None) -> int:
    """Raw C-ABI call with an explicit configuration (None = automatic)."""
    return _load().sgemm_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream,
                            ctypes.byref(cfg) if cfg is not None else None)


def sgemm_op(trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None,
             cfg: SgemmConfig | None = None) -> int:
    """Raw C-ABI call of sgemm_op (cfg given: sgemm_op_ex)."""
    if cfg is None:
        return _load().sgemm_op(trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                                stream)
    return _load().sgemm_op_ex(trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                               stream, ctypes.byref(cfg))


def sgemm_op_noalloc(trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                     stream=None, cfg: SgemmConfig | None = None) -> int:
    """Raw C-ABI call of sgemm_op_ex_noalloc (partial sums in the library's
    static scratch array; no device allocation)."""
    return _load().sgemm_op_ex_noalloc(trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C,
                                       ldc, stream,
                                       ctypes.byref(cfg) if cfg is not None else None)


def sgemm_epilogue(trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act,
                   stream=None, cfg: SgemmConfig | None = None) -> int:
    """Raw C-ABI call of sgemm_epilogue (cfg given: sgemm_epilogue_ex)."""
    args = (trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act, stream)
    if cfg is None:
        return _load().sgemm_epilogue(*args)
    return _load().sgemm_epilogue_ex(*args, ctypes.byref(cfg))


def sgemm_strided_batched(trans_a, trans_b, M, N, K, alpha, A, lda, stride_a, B, ldb, stride_b,
                          beta, C, ldc, stride_c, batch, stream=None,
                          cfg: SgemmConfig | None = None) -> int:
    """Raw C-ABI call of sgemm_strided_batched (cfg given: the _ex form)."""
    args = (trans_a, trans_b, M, N, K, alpha, A, lda, stride_a, B, ldb, stride_b, beta, C, ldc,
            stride_c, batch, stream)
    if cfg is None:
        return _load().sgemm_strided_batched(*args)
    return _load().sgemm_strided_batched_ex(*args, ctypes.byref(cfg))


def sgemm_mixed(dtype, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                stream=None, cfg: SgemmConfig | None = None) -> int:
    """Raw C-ABI call of sgemm_mixed (cfg given: sgemm_mixed_ex)."""
    args = (dtype, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)
    if cfg is None:
        return _load().sgemm_mixed(*args)
    return _load().sgemm_mixed_ex(*args, ctypes.byref(cfg))


def sgemm_cblas(order, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                stream=None) -> int:
    """Raw C-ABI call with cblas_sgemm's conventions (order 101 row-major /
    102 column-major; trans 111 / 112 / 113)."""
    return _load().sgemm_cblas(order, trans_a, trans_b, M, N, K, alpha, A, lda, B, ldb, beta, C,
                               ldc, stream)


def sgemm_linear(dtype, M, N, K, X, ldx, W, ldw, bias, R, ldr, act, Y, ldy, Z, ldz,
                 stream=None) -> int:
    """Raw C-ABI call: device addresses (int) or None; returns the status."""
    return _load().sgemm_linear(dtype, M, N, K, X, ldx, W, ldw, bias, R, ldr, act, Y, ldy, Z, ldz,
                                stream)


def sgemm_linear_backward(dtype, M, N, K, dY, lddy, Z, ldz, act, X, ldx, W, ldw, dX, lddx, dW,
                          lddw, db, stream=None) -> int:
    """Raw C-ABI call: device addresses (int) or None; returns the status."""
    return _load().sgemm_linear_backward(dtype, M, N, K, dY, lddy, Z, ldz, act, X, ldx, W, ldw, dX,
                                         lddx, dW, lddw, db, stream)


def sgemm_moe(dtype, T, D, F, E, top_k, gated, renormalize, act, X, ldx, Wr, ldr, W1, ld1, stride1,
              W2, ld2, stride2, Y, ldy, ids=None, weights=None, stream=None) -> int:
    """Raw C-ABI call: device addresses (int) or None; returns the status."""
    return _load().sgemm_moe(dtype, T, D, F, E, top_k, gated, renormalize, act, X, ldx, Wr, ldr, W1,
                             ld1, stride1, W2, ld2, stride2, Y, ldy, ids, weights, stream)


def select(M, N, K, A=None, lda=None, B=None, ldb=None, C=None, ldc=None, *,
           trans_a=False, trans_b=False) -> SgemmConfig:
    """The configuration sgemm() (sgemm_op() with transposition flags) picks
    for this shape (and these addresses); with edge strips, the main part's."""
    return plan(M, N, K, A, lda, B, ldb, C, ldc, trans_a=trans_a, trans_b=trans_b)[0]


def plan(M, N, K, A=None, lda=None, B=None, ldb=None, C=None, ldc=None, *,
         trans_a=False, trans_b=False):
    """(main-part configuration, edge rows, edge columns) of the automatic
    plan for this shape (and these addresses).  Leading dimensions default to
    the tight ones of the stored operands."""
    out = SgemmConfig()
    rows, cols = ctypes.c_int(0), ctypes.c_int(0)
    lda = lda or max(M if trans_a else K, 1)
    ldb = ldb or max(K if trans_b else N, 1)
    st = _load().sgemm_op_plan(int(trans_a), int(trans_b), M, N, K, A, lda, B, ldb, C,
                               ldc or max(N, 1), ctypes.byref(out), ctypes.byref(rows),
                               ctypes.byref(cols))
    if st != 0:
        raise SgemmError(st)
    return out, rows.value, cols.value


def tile_count(variant: int) -> int:
    return _load().sgemm_tile_count(variant)


def tile_info(variant: int, tile: int) -> dict:
    d = TileDesc()
    st = _load().sgemm_tile_info(variant, tile, ctypes.byref(d))
    if st != 0:
        raise SgemmError(st)
    return d.as_dict()


def status_string(status: int) -> str:
    return _load().sgemm_status_string(status).decode()


def version() -> int:
    return _load().sgemm_version()


def workspace_release() -> None:
    """Synchronise the current device and free the workspaces the library
    keeps for it (stream-K and split-K partial sums, one per stream)."""
    st = _load().sgemm_workspace_release()
    if st != 0:
        raise SgemmError(st)


def _ld(t) -> int:
    """Leading dimension of a 2-D row-major tensor view, in elements."""
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError("rows must be contiguous (stride(1) == 1)")
    ld = t.stride(0)
    if rows <= 1 or cols == 0:
        ld = max(ld, cols, 1)
    return ld


def _check_tensor(name, t, torch, device=None):
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be float32")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _on_device(device, torch):
    """A context that makes `device` current: a no-op when it already is
    (the common case, and the switch costs host time on every call)."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _stream_handle(stream, device, torch):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def gemm(A, B, C=None, alpha: float = 1.0, beta: float = 0.0, *, trans_a: bool = False,
         trans_b: bool = False, bias=None, act: int = ACT_NONE, variant: int = VARIANT_AUTO,
         tile: int = -1, flags: int = 0, group_m: int = 0, stream=None, noalloc: bool = False):
    """C = act(alpha * op(A) @ op(B) + beta * C + bias) for 2-D float32 CUDA
    tensors (row-major views with unit column stride; padded rows are used
    through their leading dimension).  op(X) is X, or X transposed when
    trans_x: A is then stored K x M and B N x K (e.g. a linear layer's weight,
    C = X W^T with B = W, trans_b=True).  bias (N floats, one per column) and
    act (ACT_*) are optional (sgemm_epilogue).  C is updated in place when
    given; otherwise a new tensor is returned (beta must then be 0).  Runs
    asynchronously on ``stream`` (default: the current stream of A's
    device).  noalloc: run through sgemm_op_ex_noalloc (no bias or act)."""
    import torch

    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    M, K = A.shape[::-1] if trans_a else A.shape
    K2, N = B.shape[::-1] if trans_b else B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: A is {tuple(A.shape)}, B is {tuple(B.shape)}")
    _check_tensor("A", A, torch)
    _check_tensor("B", B, torch, A.device)
    if bias is not None:
        _check_tensor("bias", bias, torch, A.device)
        if bias.dim() != 1 or bias.shape[0] != N or (N > 1 and bias.stride(0) != 1):
            raise ValueError(f"bias must be a contiguous vector of {N} floats")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs an input C")
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    else:
        if C.dtype != torch.float32 or C.device != A.device or tuple(C.shape) != (M, N):
            raise ValueError(f"C must be float32 ({M}, {N}) on {A.device}")
    with _on_device(A.device, torch):
        s = _stream_handle(stream, A.device, torch)
        ptr = lambda t: t.data_ptr() if t.numel() else None
        args = (M, N, K, float(alpha), ptr(A), _ld(A), ptr(B), _ld(B), float(beta), ptr(C),
                _ld(C))
        explicit = not (variant == VARIANT_AUTO and tile < 0 and flags == 0 and group_m == 0)
        cfg = SgemmConfig(variant, tile, flags, group_m) if explicit else None
        if noalloc:
            if bias is not None or act != ACT_NONE:
                raise ValueError("noalloc: no bias or activation")
            st = sgemm_op_noalloc(int(trans_a), int(trans_b), *args, s, cfg=cfg)
        elif bias is not None or act != ACT_NONE:
            st = sgemm_epilogue(int(trans_a), int(trans_b), *args,
                                None if bias is None else ptr(bias), int(act), s, cfg=cfg)
        elif trans_a or trans_b:
            st = sgemm_op(int(trans_a), int(trans_b), *args, s, cfg=cfg)
        elif explicit:
            st = sgemm_ex(*args, s, cfg=cfg)
        else:
            st = sgemm(*args, s)
    if st != 0:
        raise SgemmError(st)
    return C


def gemm_mixed(A, B, C=None, alpha: float = 1.0, beta: float = 0.0, *, trans_a: bool = False,
               trans_b: bool = False, variant: int = VARIANT_AUTO, tile: int = -1, group_m: int = 0,
               stream=None):
    """C = alpha * op(A) @ op(B) + beta * C for 2-D bfloat16 or float16 CUDA
    tensors A and B (the same dtype) and a float32 C (sgemm_mixed: fp32
    accumulation).  Layout and stream handling as gemm()."""
    import torch

    codes = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
    if A.dtype not in codes or B.dtype != A.dtype:
        raise ValueError("A and B must both be bfloat16 or both float16")
    if not A.is_cuda or B.device != A.device:
        raise ValueError("A and B must be GPU tensors on one device")
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    M, K = A.shape[::-1] if trans_a else A.shape
    K2, N = B.shape[::-1] if trans_b else B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: A is {tuple(A.shape)}, B is {tuple(B.shape)}")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs an input C")
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _check_tensor("C", C, torch, A.device)
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C must be ({M}, {N})")
    with _on_device(A.device, torch):
        s = _stream_handle(stream, A.device, torch)
        ptr = lambda t: t.data_ptr() if t.numel() else None
        explicit = not (variant == VARIANT_AUTO and tile < 0 and group_m == 0)
        cfg = SgemmConfig(variant, tile, 0, group_m) if explicit else None
        st = sgemm_mixed(codes[A.dtype], int(trans_a), int(trans_b), M, N, K, float(alpha),
                         ptr(A), _ld(A), ptr(B), _ld(B), float(beta), ptr(C), _ld(C), s, cfg=cfg)
    if st != 0:
        raise SgemmError(st)
    return C


def _batch_view(name, t, torch):
    """(batch, rows, cols, leading dimension, batch stride) of a 3-D stack of
    row-major matrices, or of a 2-D matrix shared by the batch (stride 0)."""
    if t.dim() == 2:
        rows, cols = t.shape
        return None, rows, cols, _ld(t), 0
    if t.dim() != 3:
        raise ValueError(f"{name} must be 2-D or 3-D")
    nb, rows, cols = t.shape
    if cols > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: rows must be contiguous (stride(2) == 1)")
    ld = t.stride(1) if rows > 1 else max(t.stride(1), cols, 1)
    return nb, rows, cols, max(ld, cols, 1), t.stride(0) if nb > 1 else 0


def gemm_batched(A, B, C=None, alpha: float = 1.0, beta: float = 0.0, *, trans_a: bool = False,
                 trans_b: bool = False, variant: int = VARIANT_AUTO, tile: int = -1,
                 flags: int = 0, group_m: int = 0, stream=None):
    """C[b] = alpha * op(A[b]) @ op(B[b]) + beta * C[b] for every b
    (sgemm_strided_batched).  A and B are 3-D float32 CUDA tensors (batch,
    rows, cols) with unit column stride, or 2-D matrices shared by the whole
    batch (batch stride 0); C is a 3-D tensor (batch, M, N), updated in place
    when given (otherwise a new one; beta must then be 0)."""
    import torch

    _check_tensor("A", A, torch)
    _check_tensor("B", B, torch, A.device)
    na, ar, ac, lda, sa = _batch_view("A", A, torch)
    nb, br, bc, ldb, sb = _batch_view("B", B, torch)
    M, K = (ac, ar) if trans_a else (ar, ac)
    K2, N = (bc, br) if trans_b else (br, bc)
    if K != K2:
        raise ValueError(f"inner dimensions differ: A is {tuple(A.shape)}, B is {tuple(B.shape)}")
    sizes = {n for n in (na, nb) if n is not None}
    if len(sizes) > 1:
        raise ValueError(f"batch sizes differ: {sorted(sizes)}")
    batch = sizes.pop() if sizes else (C.shape[0] if C is not None and C.dim() == 3 else 1)
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs an input C")
        C = torch.empty((batch, M, N), dtype=torch.float32, device=A.device)
    _check_tensor("C", C, torch, A.device)
    if C.dim() != 3 or tuple(C.shape) != (batch, M, N):
        raise ValueError(f"C must be ({batch}, {M}, {N})")
    _, _, _, ldc, sc = _batch_view("C", C, torch)
    with _on_device(A.device, torch):
        s = _stream_handle(stream, A.device, torch)
        ptr = lambda t: t.data_ptr() if t.numel() else None
        explicit = not (variant == VARIANT_AUTO and tile < 0 and flags == 0 and group_m == 0)
        cfg = SgemmConfig(variant, tile, flags, group_m) if explicit else None
        st = sgemm_strided_batched(int(trans_a), int(trans_b), M, N, K, float(alpha), ptr(A), lda,
                                   sa, ptr(B), ldb, sb, float(beta), ptr(C), ldc, sc, batch, s,
                                   cfg=cfg)
    if st != 0:
        raise SgemmError(st)
    return C


# ---- the feed-forward operators ------------------------------------------------
#
# Small calls take a few microseconds on the GPU, so the checks below use the
# cheapest forms torch has for them (device indexes instead of device objects,
# one read of each property): with the helpers above a linear layer took 12 us of
# host time, with these 9, of which 4 are the library's call and launch.

_torch = _raw_stream = _get_device = None
_codes: dict = {}


def _import_torch():
    global _torch, _raw_stream, _get_device
    import torch

    _codes.update({torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16})
    _raw_stream, _get_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _torch = torch
    return torch


def _rows(name, t, dtype, dev):
    """(rows, columns, address, leading dimension) of a row-major matrix."""
    try:
        r, c = t.shape
    except ValueError:
        raise ValueError(f"{name} must be 2-D") from None
    if t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} on GPU {dev}")
    ld, one = t.stride()
    if one != 1 and c > 1:
        raise ValueError(f"{name}: rows must be contiguous (stride(1) == 1)")
    if ld < c or ld < 1:
        if r > 1 and c > 0:
            raise ValueError(f"{name}: rows must not overlap")
        ld = c if c > 1 else 1
    if ld > 0x7fffffff or r > 0x7fffffff:
        raise ValueError(f"{name}: sizes and strides must fit 32 bits")
    return r, c, t.data_ptr() or None, ld


def _matrix(name, t, rows, cols, dtype, dev):
    """(address, leading dimension) of a row-major rows x cols matrix."""
    r, c, p, ld = _rows(name, t, dtype, dev)
    if r != rows or c != cols:
        raise ValueError(f"{name} must be ({rows}, {cols}), got ({r}, {c})")
    return p, ld


def _vector(name, t, n, dtype, dev):
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n} values")
    if t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} on GPU {dev}")
    return t.data_ptr() or None


def _first(name, t):
    """(dtype code, dtype, device index) that the call's other arrays share."""
    dtype = t.dtype
    code = _codes.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    dev = t.get_device()
    if dev < 0:
        if t.dim() != 2:
            raise ValueError(f"{name} must be 2-D")
        raise ValueError(f"{name} must be a GPU tensor")
    return code, dtype, dev


def _call(dev, stream, entry, args):
    """entry(*args, stream) with the arrays' device current."""
    if stream is None:
        stream = _raw_stream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if _get_device() == dev:
        st = entry(*args, stream)
    else:
        with _torch.cuda.device(dev):
            st = entry(*args, stream)
    if st != 0:
        raise SgemmError(st)


def linear(X, W, bias=None, *, act: int = ACT_NONE, residual=None, keep_pre: bool = False,
           out=None, pre=None, stream=None):
    """act(X @ W.T + bias) + residual for 2-D float32, bfloat16 or float16 CUDA
    tensors of one type (sgemm_linear): a linear layer with its whole epilogue,
    computed in fp32 and rounded once.  X is M x K, W N x K, bias N values,
    residual M x N; rows contiguous, padded rows are used through their leading
    dimension.  keep_pre also returns X @ W.T + bias, the activation's input,
    for linear_backward: (Y, Z).  out and pre receive Y and Z when given (out
    may be residual itself).  Runs asynchronously on ``stream`` (default: the
    current stream of X's device)."""
    _torch or _import_torch()
    code, dtype, dev = _first("X", X)
    M, K, x, ldx = _rows("X", X, dtype, dev)
    N, cols, w, ldw = _rows("W", W, dtype, dev)
    if cols != K:
        raise ValueError(f"inner dimensions differ: X is ({M}, {K}), W is ({N}, {cols})")
    b = r = z = None
    ldr = ldz = 0
    if bias is not None:
        b = _vector("bias", bias, N, dtype, dev)
    if residual is not None:
        r, ldr = _matrix("residual", residual, M, N, dtype, dev)
    if out is None:
        out = X.new_empty((M, N))
        y, ldy = out.data_ptr() or None, N or 1
    else:
        y, ldy = _matrix("out", out, M, N, dtype, dev)
    if pre is not None:
        z, ldz = _matrix("pre", pre, M, N, dtype, dev)
    elif keep_pre:
        pre = X.new_empty((M, N))
        z, ldz = pre.data_ptr() or None, N or 1
    _call(dev, stream, _load().sgemm_linear,
          (code, M, N, K, x, ldx, w, ldw, b, r, ldr, act, y, ldy, z, ldz))
    return (out, pre) if keep_pre else out


def linear_backward(dY, X, W, Z=None, *, act: int = ACT_NONE, need_x: bool = True,
                    need_w: bool = True, need_bias: bool = True, stream=None):
    """(dX, dW, db): the gradients of ``linear`` for the gradient dY of its
    result (sgemm_linear_backward); None in the place of one that is not
    needed.  Z is the activation's input that ``linear(keep_pre=True)`` returned
    (not needed for ACT_NONE); the gradient of a residual is dY itself.  Types,
    layout and stream handling as linear()."""
    _torch or _import_torch()
    code, dtype, dev = _first("dY", dY)
    M, N, g, ldg = _rows("dY", dY, dtype, dev)
    rows, K, x, ldx = _rows("X", X, dtype, dev)
    if rows != M:
        raise ValueError(f"dY has {M} rows, X {rows}")
    w, ldw = _matrix("W", W, N, K, dtype, dev)
    z, ldz = None, N or 1
    if act != ACT_NONE:
        if Z is None:
            raise ValueError("an activation's gradient needs its input Z")
        z, ldz = _matrix("Z", Z, M, N, dtype, dev)
    dX = dW = db = px = pw = pb = None
    ldk = K or 1
    if need_x:
        dX = dY.new_empty((M, K))
        px = dX.data_ptr() or None
    if need_w:
        dW = dY.new_empty((N, K))
        pw = dW.data_ptr() or None
    if need_bias:
        db = dY.new_empty((N,))
        pb = db.data_ptr() or None
    _call(dev, stream, _load().sgemm_linear_backward,
          (code, M, N, K, g, ldg, z, ldz, act, x, ldx, w, ldw, px, ldk, pw, ldk, pb))
    return dX, dW, db


def _stack(name, t, n, rows, cols, dtype, dev):
    """(address, leading dimension, matrix stride) of a stack of n matrices."""
    if t.shape != (n, rows, cols):
        raise ValueError(f"{name} must be ({n}, {rows}, {cols}), got {tuple(t.shape)}")
    if t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} on GPU {dev}")
    step, ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name}: rows must be contiguous (stride(2) == 1)")
    if ld > 0x7fffffff:
        raise ValueError(f"{name}: strides must fit 32 bits")
    return t.data_ptr() or None, ld if rows > 1 else max(ld, cols), step if n > 1 else 0


def moe(X, router, W1, W2, top_k: int, *, act: int = ACT_SILU, renormalize: bool = True, out=None,
        return_routing: bool = False, stream=None):
    """A whole mixture-of-experts layer for at most 64 tokens (sgemm_moe): X is
    T x D, router E x D, W2 E x D x F, and W1 E x 2F x D (gate rows, then up
    rows: h = act(gate) * up) or E x F x D (h = act(W1 x)); float32, bfloat16 or
    float16, one type, rows contiguous.  Each token goes through its top_k
    experts of largest logit (ties: the lowest index), weighted by the softmax
    over all experts, divided by the sum of the chosen with renormalize.
    Returns Y (T x D; ``out`` when given), with return_routing (Y, ids, weights),
    T x top_k int32 and float32.  Runs asynchronously on ``stream``
    (default: the current stream of X's device)."""
    torch = _torch or _import_torch()
    code, dtype, dev = _first("X", X)
    if W1.dim() != 3 or W2.dim() != 3:
        raise ValueError("W1 and W2 must be 3-D")
    T, D, x, ldx = _rows("X", X, dtype, dev)
    E, _, F = W2.shape
    rows = W1.shape[1]
    gated = int(rows == 2 * F)
    wr, ldr = _matrix("router", router, E, D, dtype, dev)
    w1, ld1, step1 = _stack("W1", W1, E, 2 * F if gated else F, D, dtype, dev)
    w2, ld2, step2 = _stack("W2", W2, E, D, F, dtype, dev)
    if not 1 <= top_k <= E:
        raise ValueError(f"top_k must be 1 to {E}")
    if out is None:
        out = X.new_empty((T, D))
        y, ldy = out.data_ptr() or None, D
    else:
        y, ldy = _matrix("out", out, T, D, dtype, dev)
    ids = weights = pi = pw = None
    if return_routing:
        ids = X.new_empty((T, top_k), dtype=torch.int32)
        weights = X.new_empty((T, top_k), dtype=torch.float32)
        pi, pw = ids.data_ptr() or None, weights.data_ptr() or None
    _call(dev, stream, _load().sgemm_moe,
          (code, T, D, F, E, top_k, gated, 1 if renormalize else 0, act, x, ldx, wr, ldr, w1, ld1,
           step1, w2, ld2, step2, y, ldy, pi, pw))
    return (out, ids, weights) if return_routing else out
