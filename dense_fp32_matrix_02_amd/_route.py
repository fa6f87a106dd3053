"""Routing of tokens to experts, the order of the experts' rows, and the
weighted return of those rows.

The C calls of include/sgemm_mi355_route.h under their own names, and wrappers
that take torch tensors on the GPU (argument marshalling only).
"""
from __future__ import annotations

import ctypes

from ._binding import MOST, _launch
from ._fp8 import _bind, _check, _empty, _F, _gpu, _I, _ld, _Library, _P, _stream_of, _type_of, torch

SOFTMAX, SIGMOID = 0, 1
MAX_EXPERTS, MAX_CHOICES = 1024, 32

_SIZE = ctypes.c_size_t
_SIGNATURES = {
    "sgemm_mi355_route": [_I, _I, _I, _P, _I, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P],
    "sgemm_mi355_route_backward": [_I, _I, _I, _P, _I, _P, _P, _I, _I, _I, _F, _P, _I, _P],
    "sgemm_mi355_route_plan": [_I, _I, _I, _P, _P, _P, _P, _P, _SIZE, _P],
    "sgemm_mi355_route_combine": [_I, _I, _I, _I, _I, _P, _I, _P, _P, _P, _I, _P],
    "sgemm_mi355_route_combine_backward": [_I, _I, _I, _I, _I, _P, _I, _P, _I, _P, _P, _P, _I, _P, _P],
}
_SIGNATURES["sgemm_mi355_route_plan_workspace_size"] = [_I, _I, _I]
_RESULTS = {"sgemm_mi355_route_plan_workspace_size": _SIZE}
for _name, _types in _SIGNATURES.items():
    globals()[_name] = _bind(_name, _types, _RESULTS.get(_name, _I))
_c = _Library(_SIGNATURES, _RESULTS)


def _score(score):
    code = {"softmax": SOFTMAX, "sigmoid": SIGMOID}.get(score)
    if code is None:
        raise ValueError(f"unknown score {score!r}")
    return code


def _dense(x, name, dtype, shape, device):
    """Address of a dense tensor of this dtype and shape on this GPU."""
    _gpu(x, name, dtype, device)
    if x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{name} must be a dense {' x '.join(map(str, shape))} tensor")
    if shape[0] > MOST or shape[-1] > MOST:
        raise ValueError(f"{name} has a size over 2^31 - 1")
    return x.data_ptr()


def _bounded(x):
    """A count that the C calls refuse, inside an int's range."""
    return max(-1, min(x, MAX_EXPERTS + 1))


def route(logits, k: int, *, bias=None, score: str = "softmax", groups: int = 1, top_groups: int = 1,
          renorm: bool = True, scale: float = 1.0, stream=None):
    """(weights, experts): each token's k experts and their weights, tokens x k
    (float32 and int32), by descending choice value; of equal values the lower
    index comes first.

    logits: tokens x experts, float32, bfloat16 or float16. The scores are a
    softmax or a sigmoid of them; ``bias`` (float32, one for each expert) moves
    the choice and not the weights; with ``groups`` > 1 only the ``top_groups``
    groups with the largest sum of their two largest choice values take part;
    ``renorm`` divides the weights by their sum; ``scale`` multiplies them.
    """
    on = _gpu(logits, "logits")
    kind, ld, how = _type_of(logits.dtype, "logits"), _ld(logits, "logits"), _score(score)
    tokens, experts = logits.shape
    if not (0 <= k <= MAX_CHOICES and 1 <= top_groups <= groups <= MAX_EXPERTS):
        k, groups, top_groups = _bounded(k), _bounded(groups), _bounded(top_groups)
    at = None if bias is None else _dense(bias, "bias", torch.float32, (experts,), on)
    weights = _empty((tokens, max(k, 0)), torch.float32, logits.device, stream)
    ids = _empty((tokens, max(k, 0)), torch.int32, logits.device, stream)
    _check(_launch(_c.route, on, kind, tokens, experts, logits.data_ptr(), ld, at, how, groups, top_groups, k,
                             int(bool(renorm)), scale, weights.data_ptr(), ids.data_ptr(), _stream_of(on, stream)),
           "route")
    return weights, ids


def route_backward(logits, experts, dweights, *, score: str = "softmax", renorm: bool = True, scale: float = 1.0,
                   stream=None):
    """The gradient of the logits (float32) for given gradients of route's
    weights; ``experts`` are the ones it chose."""
    on = _gpu(logits, "logits")
    kind, ld, how = _type_of(logits.dtype, "logits"), _ld(logits, "logits"), _score(score)
    tokens, count = logits.shape
    k = experts.shape[-1]
    ids = _dense(experts, "experts", torch.int32, (tokens, k), on)
    dw = _dense(dweights, "dweights", torch.float32, (tokens, k), on)
    out = _empty((tokens, count), torch.float32, logits.device, stream)
    _check(_launch(_c.route_backward, on, kind, tokens, count, logits.data_ptr(), ld, ids, dw, how, k,
                                      int(bool(renorm)), scale, out.data_ptr(), max(count, 1), _stream_of(on, stream)),
           "route_backward")
    return out


def route_plan(experts, num_experts: int, *, stream=None):
    """(offsets, tokens, place): the tokens' rows sorted by expert.

    experts: tokens x k int32, as route gives them. Expert e's rows are
    offsets[e] .. offsets[e + 1] - 1 (offsets: num_experts + 1); row r is a row
    of token tokens[r]; choice j of token t has row place[t, j]. Ids outside
    the experts come after offsets[-1].
    """
    if experts.dim() != 2:
        raise ValueError("experts must be tokens x k")
    tokens, k = experts.shape
    on = _gpu(experts, "experts", torch.int32)
    ids = _dense(experts, "experts", torch.int32, (tokens, k), on)
    if not 1 <= num_experts <= MAX_EXPERTS:
        num_experts = _bounded(num_experts)
    need = _c.route_plan_workspace_size(tokens, k, num_experts)
    offsets = _empty((max(num_experts, 0) + 1,), torch.int32, experts.device, stream)
    rows = _empty((tokens * k,), torch.int32, experts.device, stream)
    place = _empty((tokens, k), torch.int32, experts.device, stream)
    room = _empty((need // 4,), torch.int32, experts.device, stream) if need else None
    _check(_launch(_c.route_plan, on, tokens, k, num_experts, ids, offsets.data_ptr(), rows.data_ptr(),
                                  place.data_ptr(), None if room is None else room.data_ptr(), need, _stream_of(on, stream)),
           "route_plan")
    return offsets, rows, place


def route_combine(Z, place, weights, Y=None, *, stream=None):
    """Y[t] = sum_j weights[t, j] * Z[place[t, j]], of Z's dtype; a place
    outside Z's rows adds nothing."""
    on = _gpu(Z, "Z")
    kind, ldz = _type_of(Z.dtype, "Z"), _ld(Z, "Z")
    rows, cols = Z.shape
    tokens, k = place.shape
    at, w = _dense(place, "place", torch.int32, (tokens, k), on), _dense(weights, "weights", torch.float32, (tokens, k), on)
    if Y is None:
        Y = _empty((tokens, cols), Z.dtype, Z.device, stream)
    _gpu(Y, "Y", Z.dtype, on)
    if tuple(Y.shape) != (tokens, cols):
        raise ValueError("Y must be tokens x cols")
    _check(_launch(_c.route_combine, on, kind, tokens, k, rows, cols, Z.data_ptr(), ldz, at, w, Y.data_ptr(), _ld(Y, "Y"),
                                     _stream_of(on, stream)), "route_combine")
    return Y


def route_combine_backward(dY, Z, place, weights, *, stream=None):
    """(dZ, dweights) of route_combine for the gradient dY of its result.

    place must name no row of Z twice (route_plan's names each once); the
    gradient of a row that it does not name is zero.
    """
    on = _gpu(Z, "Z")
    _gpu(dY, "dY", Z.dtype, on)
    kind, ldz, ldy = _type_of(Z.dtype, "Z"), _ld(Z, "Z"), _ld(dY, "dY")
    rows, cols = Z.shape
    tokens, k = place.shape
    if tuple(dY.shape) != (tokens, cols):
        raise ValueError("dY must be tokens x cols")
    at, w = _dense(place, "place", torch.int32, (tokens, k), on), _dense(weights, "weights", torch.float32, (tokens, k), on)
    dZ = _empty((rows, cols), Z.dtype, Z.device, stream)
    dw = _empty((tokens, k), torch.float32, Z.device, stream)
    _check(_launch(_c.route_combine_backward, on, kind, tokens, k, rows, cols, dY.data_ptr(), ldy, Z.data_ptr(), ldz, at, w,
                                              dZ.data_ptr(), max(cols, 1), dw.data_ptr(), _stream_of(on, stream)),
           "route_combine_backward")
    if tokens * k == 0 and dZ.numel() > 0:  # the C call writes nothing then
        with torch.cuda.stream(stream):
            dZ.zero_()
    return dZ, dw
