"""Products by expert of 16-bit operands: the rows of a layer of experts times
each expert's weights, and the gradients of the rows and of the weights.

The C calls of include/sgemm_mi355_experts.h under their own names, and
wrappers that take torch tensors on the GPU (argument marshalling only).
"""
from __future__ import annotations

import ctypes

from ._binding import MOST
from ._fp8 import _bind, _check, _empty, _F, _gpu, _I, _ints, _ld, _Library, _LL, _P, _result, _stream_of, _type_of, torch
from ._layer import _launch, _like, _matrix

EXPERTS_FORWARD, EXPERTS_DGRAD, EXPERTS_WGRAD = 0, 1, 2

_PRODUCT = [_I] * 6 + [_P, _I, _P, _I, _LL, _P, _P, _I, _P]
_SIGNATURES = {
    "sgemm_mi355_experts_gemm": _PRODUCT,
    "sgemm_mi355_experts_gemm_dgrad": _PRODUCT,
    "sgemm_mi355_experts_gemm_wgrad": [_I] * 6 + [_P, _I, _P, _I, _P, _F, _P, _I, _LL, _P],
}
for _name, _types in _SIGNATURES.items():
    globals()[_name] = _bind(_name, _types)
_kernel_name = _bind("sgemm_mi355_experts_kernel_name", [_I] * 5 + [_P, _I, _P, _I, _LL], ctypes.c_char_p)
_c = _Library(_SIGNATURES)


def sgemm_mi355_experts_kernel_name(form, rows, N, K, experts, A, lda, W, ldw, strideW=0) -> str | None:
    """Name of the kernel that a product with these arguments runs, or None."""
    r = _kernel_name(form, rows, N, K, experts, A, lda, W, ldw, strideW)
    return r.decode() if r is not None else None


def _result_of(C, shape, dtype, A, on, stream):
    """C, its type, address and row stride."""
    if C is None:
        kind = _type_of(dtype, "C")
        C = _empty(shape, dtype, A.device, stream)
        return C, kind, C.data_ptr(), shape[-1] or 1
    C = _result(C, shape, dtype, A, on, 0.0, stream)
    return C, _type_of(C.dtype, "C"), C.data_ptr(), _ld(C, "C")


def _stride(ld, rows):
    """The row stride to give for so many rows: of a single one, which may have any, one that direct loads take."""
    return ld + -ld % 8 if rows == 1 else ld


def _rows_by_expert(call, name, A, W, offsets, C, dtype, stream, inner, outer):
    sizes, strides = W.shape, W.stride()
    if len(sizes) != 3 or A.dim() != 2 or sizes[0] < 1:
        raise ValueError("A must be 2-D, W 3-D with the experts first")
    E, N, K = sizes
    on, kind, a, lda, (rows, columns) = _matrix(A, "A")
    if columns != sizes[inner]:
        raise ValueError("inner dimensions differ")
    if W.get_device() != on or W.dtype != A.dtype:
        _gpu(W, "W", A.dtype, on)
    ldw = strides[1] if strides[2] == 1 and 1 < N <= MOST >= strides[1] >= K > 0 else _ld(W[0], "W")
    off = _ints(offsets, "offsets", on, E + 1)
    C, c_kind, c, ldc = _result_of(C, (rows, sizes[outer]), dtype or A.dtype, A, on, stream)
    _check(_launch(call, on, kind, c_kind, rows, N, K, E, a, _stride(lda, rows), W.data_ptr(), _stride(ldw, N), strides[0], off, c, ldc,
                   _stream_of(on, stream)), name)
    return C


def gemm_experts(A, W, offsets, C=None, *, dtype=None, stream=None):
    """C[r] = A[r].W[e]^T for expert e's rows r, offsets[e] <= r < offsets[e + 1].

    A (rows x K) holds the rows sorted by expert, W is experts x N x K, both
    bfloat16 or float16; offsets (int32, experts + 1) as route_plan gives them.
    Rows from offsets[-1] on are set to zero. C (rows x N) is allocated with
    ``dtype`` (A's unless given, or float32) when omitted. Sums are float32.
    """
    return _rows_by_expert(_c.experts_gemm, "experts_gemm", A, W, offsets, C, dtype, stream, 2, 1)


def gemm_experts_dgrad(A, W, offsets, C=None, *, dtype=None, stream=None):
    """The gradient of gemm_experts' rows: C[r] = A[r].W[e] for the gradient A
    (rows x N) of its result; C is rows x K. The rest as in gemm_experts."""
    return _rows_by_expert(_c.experts_gemm_dgrad, "experts_gemm_dgrad", A, W, offsets, C, dtype, stream, 1, 2)


def gemm_experts_wgrad(A, B, offsets, C=None, *, beta: float = 0.0, dtype=None, stream=None):
    """The gradient of gemm_experts' weights: C[e] = sum over expert e's rows r
    of A[r]^T.B[r] + beta*C[e], for the gradient A (rows x N) of its result and
    its rows B (rows x K). C is experts x N x K, allocated with ``dtype``
    (float32 unless given, or A's) when omitted."""
    on, kind, a, lda, (rows, N) = _matrix(A, "A")
    if B.dim() != 2 or B.shape[0] != rows:
        raise ValueError("A and B must be 2-D with as many rows")
    K = B.shape[1]
    b, ldb = _like(B, "B", A.dtype, on, (rows, K))
    off = _ints(offsets, "offsets", on)
    E = offsets.numel() - 1
    if E < 1:
        raise ValueError("offsets must have experts + 1 values")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs an input C")
        dtype = dtype or torch.float32
        c_kind = _type_of(dtype, "C")
        C = _empty((E, N, K), dtype, A.device, stream)
        ldc, apart = K or 1, N * K
    else:
        C = _result(C, (E, N, K), dtype, A, on, beta, stream)
        c_kind, ldc, apart = _type_of(C.dtype, "C"), _ld(C[0], "C"), C.stride(0)
    _check(_launch(_c.experts_gemm_wgrad, on, kind, c_kind, rows, N, K, E, a, _stride(lda, rows), b, _stride(ldb, rows), off, beta,
                   C.data_ptr(), ldc, apart, _stream_of(on, stream)), "experts_gemm_wgrad")
    return C
