"""What stands around the products of a layer in 8 bits, forward and backward:
the root-mean-square norm with the residual's addition, gated activations, and
products with bias, activation and residual in their epilogue.

The C calls of include/sgemm_mi355_layer.h (and the product with an epilogue of
include/sgemm_mi355_fp8.h) under their own names, and wrappers that take torch
tensors on the GPU (argument marshalling only).
"""
from __future__ import annotations

import ctypes

from ._binding import MOST, run_on
from ._fp8 import (_bind, _blocks, _bytes_out, _check, _empty, _F, FP32_SUMS, _gpu, _I, _ld, _Library, _operand, _P,
                   _result, _SCALES, _stream_of, _type_of, _types, torch)

NONE, RELU, SILU, GELU, GELU_TANH = 0, 1, 2, 3, 4
MAX_NORM_COLS = 16384
_ACTIVATIONS = {None: NONE, "none": NONE, "relu": RELU, "silu": SILU, "gelu": GELU, "gelu_tanh": GELU_TANH}

_SIZE = ctypes.c_size_t
_SIGNATURES = {
    "sgemm_mi355_rms_norm": [_I, _I, _I, _P, _I, _P, _I, _P, _I, _F, _P, _I, _P, _P, _I, _P, _I, *_SCALES, _P],
    "sgemm_mi355_rms_norm_backward": [_I, _I, _I, _P, _I, _P, _I, _P, _P, _I, _P, _I, _P, _I, _P, _P, _SIZE, _P],
    "sgemm_mi355_rms_norm_backward_workspace_size": [_I, _I],
    "sgemm_mi355_gated": [_I, _I, _I, _I, _P, _I, _P, _I, _P, _I, *_SCALES, _P],
    "sgemm_mi355_gated_backward": [_I, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P],
    "sgemm_mi355_epilogue_backward": [_I, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _P, _SIZE, _P],
    "sgemm_mi355_epilogue_backward_workspace_size": [_I, _I],
    "sgemm_mi355_fp8_gemm_epilogue": [_I] * 4 + [_P, _I, *_SCALES, _P, _I, *_SCALES, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P],
}
_RESULTS = {"sgemm_mi355_rms_norm_backward_workspace_size": _SIZE, "sgemm_mi355_epilogue_backward_workspace_size": _SIZE}
for _name, _arguments in _SIGNATURES.items():
    globals()[_name] = _bind(_name, _arguments, _RESULTS.get(_name, _I))
_c = _Library(_SIGNATURES, _RESULTS)


_several = []  # whether there is more than one GPU, once that is known


def _launch(call, on, *args):
    if _several and not _several[0]:  # run_on's own first test, without the call
        return call(*args)
    return run_on(_several, call, on, *args)


def _act(name):
    code = _ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"unknown activation {name!r}")
    return code


def _vector(x, name, length, device, dtype=None):
    """Address of a dense 1-D tensor of `length` values on this GPU."""
    if x.get_device() != device or (dtype is not None and x.dtype != dtype):
        _gpu(x, name, dtype, device)
    if x.dim() != 1 or x.numel() != length or not x.is_contiguous():
        raise ValueError(f"{name} must be a dense 1-D tensor of {length} values")
    return x.data_ptr()


def _matrix(x, name):
    """(GPU, type, address, row stride, shape) of a 2-D tensor with contiguous rows."""
    on, kind = x.get_device(), _types.get(x.dtype)
    if on < 0 or kind is None:
        on, kind = _gpu(x, name), _type_of(x.dtype, name)
    shape, strides = x.shape, x.stride()
    # _ld's own first test, without the call: most matrices pass it
    if len(strides) == 2 and strides[1] == 1 and 1 < shape[0] <= MOST >= strides[0] >= shape[1] > 0:
        return on, kind, x.data_ptr(), strides[0], shape
    return on, kind, x.data_ptr(), _ld(x, name), shape


def _like(x, name, dtype, device, shape):
    """Address and row stride of a 2-D tensor of this dtype and shape on this GPU."""
    if x.get_device() != device or x.dtype != dtype:
        _gpu(x, name, dtype, device)
    sizes, strides = x.shape, x.stride()
    if sizes != shape:
        raise ValueError(f"{name} must be {' x '.join(map(str, shape))}")
    if strides[1] == 1 and 1 < sizes[0] <= MOST >= strides[0] >= sizes[1] > 0:
        return x.data_ptr(), strides[0]
    return x.data_ptr(), _ld(x, name)


def _room(need, device, stream):
    """Address of a workspace, or None, and the tensor that holds it."""
    if not need:
        return None, None
    room = _empty((need // 4,), torch.float32, device, stream)
    return room.data_ptr(), room


def _quantised_out(rows, cols, device, stream):
    if stream is None:  # _bytes_out and _empty without their calls
        ldq = max((cols + 15) & -16, 1)
        return (torch.empty_strided((rows, cols), (ldq, 1), dtype=torch.float8_e4m3fn, device=device), ldq,
                torch.empty_strided((rows, (cols + 127) // 128), (1, rows or 1), dtype=torch.float32, device=device))
    Q, ldq = _bytes_out(rows, cols, device, stream)
    return Q, ldq, _empty((rows, _blocks(cols)), torch.float32, device, stream, (1, rows or 1))


def _norm_input(X, weight, residual, H, stream):
    on, kind, x, ldx, shape = _matrix(X, "X")
    cols = shape[1]
    w = _vector(weight, "weight", cols, on)
    w_kind = _type_of(weight.dtype, "weight")
    if residual is None:
        if H is not None:
            raise ValueError("H needs a residual; without one it is X")
        return on, kind, (x, ldx, None, 0, w, w_kind), X, None, 0, shape
    dtype = X.dtype
    r, ldr = _like(residual, "residual", dtype, on, shape)
    if H is None:
        H = _empty(shape, dtype, X.device, stream)
        return on, kind, (x, ldx, r, ldr, w, w_kind), H, H.data_ptr(), cols or 1, shape
    return on, kind, (x, ldx, r, ldr, w, w_kind), H, *_like(H, "H", dtype, on, shape), shape


def rms_norm_fp8(X, weight, *, residual=None, eps: float = 1e-6, H=None, wide: bool = False, stream=None):
    """(Q, S, H, rstd): the rows of the norm of X + residual, in e4m3 with a
    scale for each block of 128 columns, as quantize_fp8 gives them.

    H = X + residual, rounded to X's dtype (X itself without a residual);
    rstd = 1 / sqrt(mean(H^2) + eps) of each row (float32); the norm is
    H * rstd * weight, quantised from its float32 values. X: float32, bfloat16
    or float16, up to 16384 columns; weight: float32 or X's dtype. ``H`` may be
    given, the residual itself for an update in place. ``wide``: the norm in
    X's dtype too, as a fifth result.
    """
    on, kind, x, H, h, ldh, (rows, cols) = _norm_input(X, weight, residual, H, stream)
    Q, ldq, S = _quantised_out(rows, cols, X.device, stream)
    rstd = _empty((rows,), torch.float32, X.device, stream)
    Y = _empty((rows, cols), X.dtype, X.device, stream) if wide else None
    _check(_launch(_c.rms_norm, on, kind, rows, cols, *x, eps, h, ldh, rstd.data_ptr(), None if Y is None else Y.data_ptr(), cols,
                       Q.data_ptr(), ldq, S.data_ptr(), 1, rows or 1, _stream_of(on, stream)), "rms_norm")
    return (Q, S, H, rstd, Y) if wide else (Q, S, H, rstd)


def rms_norm(X, weight, *, residual=None, eps: float = 1e-6, H=None, stream=None):
    """(Y, H, rstd): the norm of X + residual in X's dtype; the rest as in rms_norm_fp8."""
    on, kind, x, H, h, ldh, (rows, cols) = _norm_input(X, weight, residual, H, stream)
    Y = _empty((rows, cols), X.dtype, X.device, stream)
    rstd = _empty((rows,), torch.float32, X.device, stream)
    _check(_launch(_c.rms_norm, on, kind, rows, cols, *x, eps, h, ldh, rstd.data_ptr(), Y.data_ptr(), cols, None, 0, None, 0, 0,
                       _stream_of(on, stream)), "rms_norm")
    return Y, H, rstd


def rms_norm_backward(dY, H, rstd, weight, *, dH=None, stream=None):
    """(dX, dweight) of the norm for the gradient dY of its rows, from the H and
    rstd that the forward call returned. dX (of H's dtype) is the gradient of X
    and of the residual; ``dH``, the gradient of H from elsewhere, is added to
    it. dweight is float32."""
    on, kind, h, ldh, shape = _matrix(H, "H")
    rows, cols = shape
    dy = _like(dY, "dY", H.dtype, on, shape)
    a = _vector(rstd, "rstd", rows, on, torch.float32)
    w = _vector(weight, "weight", cols, on)
    d = (None, 0) if dH is None else _like(dH, "dH", H.dtype, on, shape)
    dX = _empty(shape, H.dtype, H.device, stream)
    dw = _empty((cols,), torch.float32, H.device, stream)
    need = _c.rms_norm_backward_workspace_size(rows, cols)
    at, room = _room(need, H.device, stream)
    _check(_launch(_c.rms_norm_backward, on, kind, rows, cols, *dy, h, ldh, a, w, _type_of(weight.dtype, "weight"), *d,
                                dX.data_ptr(), cols, dw.data_ptr(), at, need, _stream_of(on, stream)), "rms_norm_backward")
    if rows == 0:  # the C call writes nothing then
        _zero(dw, stream)
    return dX, dw


def _zero(x, stream):
    if stream is None:
        x.zero_()
    else:
        with torch.cuda.stream(stream):
            x.zero_()


def _halves(H):
    on, kind, h, ldh, (rows, cols) = _matrix(H, "H")
    if cols % 2:
        raise ValueError("H must have an even number of columns")
    return on, kind, h, ldh, rows, cols // 2


def gated_fp8(H, *, activation: str = "silu", wide: bool = False, stream=None):
    """(Q, S): z = act(g) * u in e4m3 with a scale for each block of 128
    columns, as quantize_fp8 gives them, from its float32 values; g is the
    first half of H's columns, u the second. ``wide``: z in H's dtype too, as a
    third result. Activations: "silu", "gelu", "gelu_tanh", "relu", "none"."""
    act = _act(activation)
    on, kind, h, ldh, rows, cols = _halves(H)
    Q, ldq, S = _quantised_out(rows, cols, H.device, stream)
    Z = _empty((rows, cols), H.dtype, H.device, stream) if wide else None
    _check(_launch(_c.gated, on, kind, act, rows, cols, h, ldh, None if Z is None else Z.data_ptr(), cols or 1,
                    Q.data_ptr(), ldq, S.data_ptr(), 1, rows or 1, _stream_of(on, stream)), "gated")
    return (Q, S, Z) if wide else (Q, S)


def gated(H, *, activation: str = "silu", stream=None):
    """z = act(g) * u in H's dtype; g is the first half of H's columns, u the second."""
    act = _act(activation)
    on, kind, h, ldh, rows, cols = _halves(H)
    Z = _empty((rows, cols), H.dtype, H.device, stream)
    _check(_launch(_c.gated, on, kind, act, rows, cols, h, ldh, Z.data_ptr(), cols or 1, None, 0, None, 0, 0,
                    _stream_of(on, stream)), "gated")
    return Z


def gated_backward(dZ, H, *, activation: str = "silu", stream=None):
    """dH = [act'(g) * u * dZ | act(g) * dZ], of H's dtype, for the gradient dZ of z."""
    act = _act(activation)
    on, kind, h, ldh, rows, cols = _halves(H)
    dz = _like(dZ, "dZ", H.dtype, on, (rows, cols))
    dH = _empty((rows, 2 * cols), H.dtype, H.device, stream)
    _check(_launch(_c.gated_backward, on, kind, act, rows, cols, *dz, h, ldh, dH.data_ptr(), 2 * cols or 1,
                             _stream_of(on, stream)), "gated_backward")
    return dH


def gemm_fp8_epilogue(A, SA, B, SB, C=None, *, bias=None, activation=None, residual=None, pre: bool = False, dtype=None,
                      fp32_sums: bool = False, stream=None):
    """C = act(A.B^T + bias) + residual for operands as in gemm_fp8.

    bias: float32, one for each row of B; activation: "relu", "silu", "gelu",
    "gelu_tanh" or None; residual: of C's shape and dtype, and may be C itself.
    ``pre``: returns (C, P), P the activation's argument in C's dtype, which
    epilogue_backward takes. C is allocated with ``dtype`` (the residual's, or
    bfloat16, unless given) when omitted; ``fp32_sums`` as in gemm_fp8.
    """
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    (M, K), (N, K2) = A.shape, B.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    act = _act(activation)
    on = _gpu(A, "A")
    a = _operand(A, SA, "A", M, K, on)
    b = _operand(B, SB, "B", N, K, on, either=True)
    if dtype is None:
        dtype = torch.bfloat16 if residual is None else residual.dtype
    if C is None:
        kind = _type_of(dtype, "C")
        C = _empty((M, N), dtype, A.device, stream)
        c, ldc = C.data_ptr(), N or 1
    else:
        C = _result(C, (M, N), dtype, A, on, 0.0, stream)
        kind, c, ldc = _type_of(C.dtype, "C"), C.data_ptr(), _ld(C, "C")
    v = None if bias is None else _vector(bias, "bias", N, on, torch.float32)
    r = (None, 0) if residual is None else _like(residual, "residual", C.dtype, on, (M, N))
    P = _empty((M, N), C.dtype, A.device, stream) if pre else None
    _check(_launch(_c.fp8_gemm_epilogue, on, kind | FP32_SUMS if fp32_sums else kind, M, N, K, *a[:5], *b, v, act, *r,
                   None if P is None else P.data_ptr(), N or 1, c, ldc, _stream_of(on, stream)), "fp8_gemm_epilogue")
    return (C, P) if pre else C


def epilogue_backward(dC, P, *, activation=None, bias: bool = True, stream=None):
    """(dP, dbias): dP = act'(P) * dC, the gradient of the product A.B^T, of P's
    dtype, and its sum over the rows, the bias' gradient (float32; None without
    ``bias``), for the gradient dC of gemm_fp8_epilogue's result. The
    residual's gradient is dC."""
    act = _act(activation)
    on, kind, p, ldp, shape = _matrix(P, "P")
    rows, cols = shape
    dc = _like(dC, "dC", P.dtype, on, shape)
    dP = _empty(shape, P.dtype, P.device, stream)
    db = _empty((cols,), torch.float32, P.device, stream) if bias else None
    need = _c.epilogue_backward_workspace_size(rows, cols) if bias else 0
    at, room = _room(need, P.device, stream)
    _check(_launch(_c.epilogue_backward, on, kind, act, rows, cols, *dc, p, ldp, dP.data_ptr(), cols or 1,
                                None if db is None else db.data_ptr(), at, need, _stream_of(on, stream)), "epilogue_backward")
    if bias and rows == 0:  # the C call writes nothing then
        _zero(db, stream)
    return dP, db
