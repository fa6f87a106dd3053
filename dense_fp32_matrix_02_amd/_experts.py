"""Products by expert of 16-bit operands: the rows of a layer of experts times
each expert's weights, and the gradients of the rows and of the weights.

The C calls of include/sgemm_mi355_experts.h under their own names, and
wrappers that take torch tensors on the GPU (argument marshalling only).
"""
from __future__ import annotations

import ctypes

from ._fp8 import _bind, _check, _F, _gpu, _I, _ints, _ld, _Library, _LL, _P, _result, _stream_of, _type_of, torch
from ._layer import _launch

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


def _weights(W, A, on):
    """Address, row stride and stride of the experts' weights, of A's type."""
    _gpu(W, "W", A.dtype, on)
    if W.dim() != 3 or W.shape[0] < 1:
        raise ValueError("W must be experts x N x K")
    return W.data_ptr(), _ld(W[0], "W"), W.stride(0)


def _rows_by_expert(name, A, W, offsets, C, dtype, stream, inner, outer):
    if A.dim() != 2 or W.dim() != 3:
        raise ValueError("A must be 2-D, W 3-D with the experts first")
    E, N, K = W.shape
    rows = A.shape[0]
    if A.shape[1] != W.shape[inner]:
        raise ValueError("inner dimensions differ")
    on = _gpu(A, "A")
    w = _weights(W, A, on)
    off = _ints(offsets, "offsets", on, E + 1)
    C = _result(C, (rows, W.shape[outer]), dtype or A.dtype, A, on, 0.0, stream)
    _check(_launch(getattr(_c, name), on, _type_of(A.dtype, "A"), _type_of(C.dtype, "C"), rows, N, K, E, A.data_ptr(), _ld(A, "A"),
                   *w, off, C.data_ptr(), _ld(C, "C"), _stream_of(on, stream)), name)
    return C


def gemm_experts(A, W, offsets, C=None, *, dtype=None, stream=None):
    """C[r] = A[r].W[e]^T for expert e's rows r, offsets[e] <= r < offsets[e + 1].

    A (rows x K) holds the rows sorted by expert, W is experts x N x K, both
    bfloat16 or float16; offsets (int32, experts + 1) as route_plan gives them.
    Rows from offsets[-1] on are set to zero. C (rows x N) is allocated with
    ``dtype`` (A's unless given, or float32) when omitted. Sums are float32.
    """
    return _rows_by_expert("experts_gemm", A, W, offsets, C, dtype, stream, 2, 1)


def gemm_experts_dgrad(A, W, offsets, C=None, *, dtype=None, stream=None):
    """The gradient of gemm_experts' rows: C[r] = A[r].W[e] for the gradient A
    (rows x N) of its result; C is rows x K. The rest as in gemm_experts."""
    return _rows_by_expert("experts_gemm_dgrad", A, W, offsets, C, dtype, stream, 1, 2)


def gemm_experts_wgrad(A, B, offsets, C=None, *, beta: float = 0.0, dtype=None, stream=None):
    """The gradient of gemm_experts' weights: C[e] = sum over expert e's rows r
    of A[r]^T.B[r] + beta*C[e], for the gradient A (rows x N) of its result and
    its rows B (rows x K). C is experts x N x K, allocated with ``dtype``
    (float32 unless given, or A's) when omitted."""
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    (rows, N), (rows_b, K) = A.shape, B.shape
    if rows != rows_b:
        raise ValueError("A and B must have as many rows")
    on = _gpu(A, "A")
    _gpu(B, "B", A.dtype, on)
    off = _ints(offsets, "offsets", on)
    E = offsets.numel() - 1
    if E < 1:
        raise ValueError("offsets must have experts + 1 values")
    C = _result(C, (E, N, K), dtype or torch.float32, A, on, beta, stream)
    _check(_launch(_c.experts_gemm_wgrad, on, _type_of(A.dtype, "A"), _type_of(C.dtype, "C"), rows, N, K, E, A.data_ptr(),
                   _ld(A, "A"), B.data_ptr(), _ld(B, "B"), off, beta, C.data_ptr(), _ld(C[0], "C"), C.stride(0),
                   _stream_of(on, stream)), "experts_gemm_wgrad")
    return C
