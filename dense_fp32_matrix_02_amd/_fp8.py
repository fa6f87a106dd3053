"""FP8 products with a scale for each block of 128, and their quantisers.

The C calls of include/sgemm_mi355_fp8.h under their own names, and wrappers
that take torch tensors on the GPU (argument marshalling only; the arithmetic
runs in the library's HIP kernels, and there is no fallback).

A quantised matrix is a pair (Q, S): Q of dtype float8_e4m3fn, S float32 with
one column for each block of 128 columns of Q. Rows of Q are stored at a stride
that is a multiple of 16 bytes; the scales of rows are stored block by block
(S.stride() == (1, rows)), those of tiles row by row.
"""
from __future__ import annotations

import ctypes

from ._binding import MOST, OK, SgemmError, load
from ._binding import _ld as _any_ld

ERR_TYPE, ERR_ROUTE = -13, -14
F32, BF16, F16 = 0, 1, 2
FP32_SUMS = 0x100  # added to a product's type
FP8_DENSE, FP8_EXPERTS, FP8_WGRAD = 0, 1, 2

_P, _I, _LL, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
_SCALES = [_P, _LL, _LL]
_SIGNATURES = {
    "sgemm_mi355_fp8_quantize_rows": [_I, _I, _I, _P, _I, _P, _I, _P, _I, *_SCALES, _P],
    "sgemm_mi355_fp8_quantize_cols": [_I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _I, *_SCALES, _P],
    "sgemm_mi355_fp8_quantize_tiles": [_I, _I, _I, _P, _I, _P, _I, *_SCALES, _P],
    "sgemm_mi355_fp8_gemm": [_I] * 4 + [_P, _I, *_SCALES, _P, _I, *_SCALES, _I, _F, _P, _I, _P],
    "sgemm_mi355_fp8_gemm_experts": [_I] * 5 + [_P, _I, *_SCALES, _P, _I, _LL, *_SCALES, _LL, _I, _P, _P, _I, _P],
    "sgemm_mi355_fp8_gemm_experts_wgrad": [_I] * 5 + [_P, _I, *_SCALES, _P, _I, *_SCALES, _P, _F, _P, _I, _LL, _P],
}


def _bind(name, argtypes, restype=_I):
    """The C function `name`, looked up in the library at its first call."""
    found = []

    def call(*args):
        if not found:
            fn = getattr(load(), name)
            fn.argtypes, fn.restype = argtypes, restype
            found.append(fn)
        return found[0](*args)

    call.__name__ = call.__qualname__ = name
    call.__doc__ = f"C function {name}: device addresses and the stream as ints; returns its code."
    return call


for _name, _types in _SIGNATURES.items():
    globals()[_name] = _bind(_name, _types)


_kernel_name = _bind("sgemm_mi355_fp8_kernel_name", [_I] * 6 + [_P, _I, _P, _I, _LL], ctypes.c_char_p)


def sgemm_mi355_fp8_kernel_name(form, type, M, N, K, experts, A, lda, B, ldb, strideB=0) -> str | None:
    """Name of the kernel that a product with these arguments runs, or None."""
    r = _kernel_name(form, type, M, N, K, experts, A, lda, B, ldb, strideB)
    return r.decode() if r is not None else None


class _Library:
    """The same functions without the wrappers' own cost: attribute `x` is C function sgemm_mi355_x, looked up once."""

    def __init__(self, signatures, results=()):
        self._signatures, self._results = signatures, dict(results)

    def __getattr__(self, name):
        name_in_c = "sgemm_mi355_" + name
        fn = getattr(load(), name_in_c)
        fn.argtypes, fn.restype = self._signatures[name_in_c], self._results.get(name_in_c, _I)
        setattr(self, name, fn)
        return fn


_c = _Library(_SIGNATURES)

# The calls below are made for single tokens too, where the host's time counts:
# an import statement in each, or asking a tensor twice, shows.
_types = {}


class _Torch:
    """torch, imported at the first use of an attribute (the C calls work without it)."""

    def __getattr__(self, name):
        import torch

        value = getattr(torch, name)
        setattr(self, name, value)
        return value


torch = _Torch()


def _ld(x, name):
    """Row stride of a 2-D tensor with contiguous rows."""
    strides, shape = x.stride(), x.shape
    if len(strides) == 2 and strides[1] == 1 and 1 < shape[0] <= MOST >= strides[0] >= shape[1] > 0:
        return strides[0]
    return _any_ld(x, name)


def _type_of(dtype, name):
    code = _types.get(dtype)
    if code is None:
        _types.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})
        code = _types.get(dtype)
        if code is None:
            raise TypeError(f"{name} must be float32, bfloat16 or float16")
    return code


def _stream_of(device, stream):
    if stream is None:  # the handle of torch.cuda.current_stream without a Stream object
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise ValueError(f"the stream is on GPU {stream.device_index}, the call's tensors on GPU {device}")
    return stream.cuda_stream


def _empty(shape, dtype, device, stream, strides=None):
    """A tensor from torch's caching allocator, allocated on the stream the
    call runs on, so that the allocator hands its memory out again only after
    that stream's work."""
    if strides is None:
        strides = (shape[1] or 1, 1) if len(shape) == 2 else (1,) if len(shape) == 1 else (shape[1] * shape[2], shape[2], 1)
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)  # cheaper than torch.empty here
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)


def _gpu(x, name, dtype=None, device=None):
    """The number of x's GPU, which has to be `device` where that is given."""
    at = x.get_device()  # -1: on the host
    if at < 0 or (dtype is not None and x.dtype != dtype):
        raise TypeError(f"{name} must be a {'' if dtype is None else str(dtype).replace('torch.', '') + ' '}GPU tensor")
    if device is not None and at != device:
        raise ValueError(f"{name} is on GPU {at}, other tensors of the call on GPU {device}")
    return at


def _ints(x, name, device, length=None):
    """Address of a dense 1-D int32 tensor on this GPU."""
    _gpu(x, name, torch.int32, device)
    if x.dim() != 1 or (x.numel() > 1 and x.stride(0) != 1) or (length is not None and x.numel() != length):
        raise ValueError(f"{name} must be a dense 1-D tensor" + ("" if length is None else f" of {length} values"))
    if x.numel() > MOST:
        raise ValueError(f"{name} has more than 2^31 - 1 values")
    return x.data_ptr()


def _check(rc, where):
    if rc != OK:
        raise SgemmError(rc, "sgemm_mi355_" + where)


def _blocks(n):
    return (n + 127) // 128


def _bytes_out(rows, cols, device, stream):
    """An uninitialised e4m3 matrix whose row stride is a multiple of 16 bytes, and that stride."""
    ld = max(cols + -cols % 16, 1)
    return _empty((rows, cols), torch.float8_e4m3fn, device, stream, (ld, 1)), ld


def quantize_fp8(X, *, index=None, blocks: bool = False, stream=None):
    """(Q, S): the rows of X (float32, bfloat16 or float16, rows may be padded)
    in e4m3 with a scale for each block of 128 columns.

    ``index`` (int32): row i of Q is row index[i] of X; an index outside X
    gives zeros. ``blocks``: one scale for each 128 x 128 tile instead, for
    weights; S then has a row for each 128 rows of X.
    """
    on = _gpu(X, "X")
    kind, ldx = _type_of(X.dtype, "X"), _ld(X, "X")
    rows, cols = X.shape
    s = _stream_of(on, stream)
    if blocks:
        if index is not None:
            raise ValueError("tiles are quantised without an index")
        Q, ldq = _bytes_out(rows, cols, X.device, stream)
        tiles = _blocks(cols)
        S = _empty((_blocks(rows), tiles), torch.float32, X.device, stream)
        _check(_c.fp8_quantize_tiles(kind, rows, cols, X.data_ptr(), ldx, Q.data_ptr(), ldq, S.data_ptr(), max(tiles, 1), 1, s),
               "fp8_quantize_tiles")
        return Q, S
    n = rows if index is None else index.numel()
    at = None if index is None else _ints(index, "index", on)
    Q, ldq = _bytes_out(n, cols, X.device, stream)
    S = _empty((n, _blocks(cols)), torch.float32, X.device, stream, (1, max(n, 1)))  # block by block
    if at is not None and n == 0:
        return Q, S
    _check(_c.fp8_quantize_rows(kind, rows, cols, X.data_ptr(), ldx, at, n, Q.data_ptr(), ldq, S.data_ptr(), 1, max(n, 1), s),
           "fp8_quantize_rows")
    return Q, S


def quantize_fp8_cols(X, *, index=None, offsets=None, stream=None):
    """(Q, S): the columns of X in e4m3, stored transposed (row c of Q is
    column c of X) with a scale for each block of 128 rows of X, for products
    that sum over X's rows.

    ``index`` (int32): the rows of X to take, in their order. ``offsets``
    (int32, experts + 1): the rows are sorted by expert and every expert's rows
    begin a block, expert e's block offsets[e] // 128 + e; Q then has
    128 * (n // 128 + experts) columns, zero where no row is.
    """
    on = _gpu(X, "X")
    kind, ldx = _type_of(X.dtype, "X"), _ld(X, "X")
    rows, cols = X.shape
    n = rows if index is None else index.numel()
    at = None if index is None else _ints(index, "index", on)
    experts = 0 if offsets is None else offsets.numel() - 1
    if offsets is not None and experts < 1:
        raise ValueError("offsets must have experts + 1 values")
    off = None if offsets is None else _ints(offsets, "offsets", on)
    width = n if offsets is None else 128 * (n // 128 + experts)
    Q, ldq = _bytes_out(cols, width, X.device, stream)
    S = _empty((cols, _blocks(width)), torch.float32, X.device, stream, (1, max(cols, 1)))
    if at is not None and n == 0:
        at, rows = None, 0
    _check(_c.fp8_quantize_cols(kind, rows, cols, X.data_ptr(), ldx, at, n, off, experts, Q.data_ptr(), ldq, S.data_ptr(), 1,
                                max(cols, 1), _stream_of(on, stream)), "fp8_quantize_cols")
    return Q, S


def _operand(Q, S, name, rows, cols, device, either=False):
    """Address, row stride, scales' address and strides, and rows that share a
    scale, of a quantised matrix (2-D, or the last two axes of a 3-D one)."""
    if Q.get_device() != device or S.get_device() != device or Q.dtype != torch.float8_e4m3fn or S.dtype != torch.float32:
        _gpu(Q, name, torch.float8_e4m3fn, device)
        _gpu(S, f"the scales of {name}", torch.float32, device)
    sizes, strides, apart = S.shape, Q.stride(), S.stride()
    if len(sizes) != len(strides):
        raise ValueError(f"{name} and its scales must have as many axes")
    per, blocks = sizes[-2:]
    if blocks != _blocks(cols) or not (per == rows or (either and per == _blocks(rows))):
        raise ValueError(f"the scales of {name} must be {rows}{f' or {_blocks(rows)}' if either else ''} x {_blocks(cols)}, "
                         f"not {per} x {blocks}")
    ld, step = strides[-2:]
    if step != 1 or not 1 < rows <= MOST >= ld >= cols:
        ld = _ld(Q if len(strides) == 2 else Q[0], name)
    by_row, by_block = apart[-2:]
    return Q.data_ptr(), ld or 1, S.data_ptr(), by_row, by_block, 1 if per == rows else 128


def _result(C, shape, dtype, A, on, beta, stream):
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs an input C")
        return _empty(shape, dtype, A.device, stream)
    if C.shape != shape:
        raise ValueError(f"C must be {' x '.join(map(str, shape))}")
    _gpu(C, "C", None, on)
    return C


def gemm_fp8(A, SA, B, SB, C=None, *, beta: float = 0.0, dtype=None, fp32_sums: bool = False, stream=None):
    """C = A.B^T + beta*C for quantised A (M x K) and B (N x K).

    SA has a scale for each block of a row of A (M x K/128), SB for each block
    of a row of B (N x K/128) or for each 128 x 128 tile (N/128 x K/128), as
    the quantisers give them. C is allocated with ``dtype`` (bfloat16 unless
    given) when omitted. ``fp32_sums``: the sums over a block's products are
    FP32 into a 16-bit C too, at up to twice the time (see the C header).
    """
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    (M, K), (N, K2) = A.shape, B.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    on = _gpu(A, "A")
    a = _operand(A, SA, "A", M, K, on)
    b = _operand(B, SB, "B", N, K, on, either=True)
    C = _result(C, (M, N), dtype or torch.bfloat16, A, on, beta, stream)
    kind = _type_of(C.dtype, "C") | (FP32_SUMS if fp32_sums else 0)
    _check(_c.fp8_gemm(kind, M, N, K, *a[:5], *b, beta, C.data_ptr(), _ld(C, "C"), _stream_of(on, stream)),
           "fp8_gemm")
    return C


def gemm_fp8_experts(A, SA, B, SB, offsets, C=None, *, dtype=None, fp32_sums: bool = False, stream=None):
    """C[r] = A[r].B[e]^T for expert e's rows r, offsets[e] <= r < offsets[e + 1].

    A (R x K) holds the rows sorted by expert, B is experts x N x K with scales
    for its rows (experts x N x K/128) or tiles (experts x N/128 x K/128).
    Rows from offsets[-1] on are set to zero. ``dtype`` and ``fp32_sums`` as in
    gemm_fp8.
    """
    if A.dim() != 2 or B.dim() != 3 or SB.dim() != 3 or SB.shape[0] != B.shape[0] or B.shape[0] < 1:
        raise ValueError("A must be 2-D, B and its scales 3-D with the experts first")
    (R, K), (E, N, K2) = A.shape, B.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    on = _gpu(A, "A")
    off = _ints(offsets, "offsets", on, E + 1)
    a = _operand(A, SA, "A", R, K, on)
    b = _operand(B, SB, "B", N, K, on, either=True)
    C = _result(C, (R, N), dtype or torch.bfloat16, A, on, 0.0, stream)
    kind = _type_of(C.dtype, "C") | (FP32_SUMS if fp32_sums else 0)
    _check(_c.fp8_gemm_experts(kind, R, N, K, E, *a[:5], *b[:2], B.stride(0), *b[2:5], SB.stride(0), b[5],
                               off, C.data_ptr(), _ld(C, "C"), _stream_of(on, stream)), "fp8_gemm_experts")
    return C


def gemm_fp8_experts_wgrad(A, SA, B, SB, offsets, C=None, *, beta: float = 0.0, dtype=None, fp32_sums: bool = False,
                           stream=None):
    """C[e] = sum over expert e's rows r of A[:, r].B[:, r]^T + beta*C[e].

    A (M x P) and B (N x P) as quantize_fp8_cols makes them with these
    ``offsets``; C is experts x M x N, allocated with ``dtype`` (float32 unless
    given) when omitted; ``fp32_sums`` as in gemm_fp8.
    """
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    (M, P), (N, P2) = A.shape, B.shape
    E = offsets.numel() - 1
    on = _gpu(A, "A")
    off = _ints(offsets, "offsets", on)
    if P != P2:
        raise ValueError("inner dimensions differ")
    if E < 1 or P % 128 != 0 or P < 128 * E:
        raise ValueError("A and B must be quantised by columns with these offsets")
    # P counts the blocks of rows, so the rows are known to a block: the most
    # that P has room for. The offsets end before that.
    rows = P - 128 * E + 127
    a = _operand(A, SA, "A", M, P, on)
    b = _operand(B, SB, "B", N, P, on)
    C = _result(C, (E, M, N), dtype or torch.float32, A, on, beta, stream)
    if C.dim() != 3:
        raise ValueError("C must be experts x M x N")
    ldc = _ld(C[0], "C")
    kind = _type_of(C.dtype, "C") | (FP32_SUMS if fp32_sums else 0)
    _check(_c.fp8_gemm_experts_wgrad(kind, rows, M, N, E, *a[:5], *b[:5], off, beta, C.data_ptr(), ldc,
                                     C.stride(0), _stream_of(on, stream)), "fp8_gemm_experts_wgrad")
    return C
