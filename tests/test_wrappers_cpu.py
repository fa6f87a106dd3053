"""What the torch wrappers refuse before any HIP call, with tensors that say they are on a GPU (no GPU needed)."""
from __future__ import annotations

import os

import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from dense_fp32_matrix_02_amd import _binding, _fp8, _route

FAR = 2 ** 32 + 304  # cut to 32 bits this is 304
E4M3 = torch.float8_e4m3fn


class _Stream:
    cuda_stream = 0
    device_index = 0


class OnGpu(torch.Tensor):
    """A tensor without memory that says it is on a GPU."""

    is_cuda = True
    at = 0

    def get_device(self):
        return self.at

    @property
    def device(self):
        return torch.device("cuda", self.at)


def gpu(shape, dtype=torch.float32, strides=None, at=0):
    x = torch.empty(shape, dtype=dtype, device="meta") if strides is None else \
        torch.empty_strided(shape, strides, dtype=dtype, device="meta")
    x = x.as_subclass(OnGpu)
    x.at = at
    return x


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(sg.LIB_PATH):
        from dense_fp32_matrix_02_amd import build
        build.build()
    return sg.load()


@pytest.fixture(autouse=True)
def no_allocation(monkeypatch):
    """Outputs without memory, on no stream."""
    for module in (_fp8, _route):
        monkeypatch.setattr(module, "_empty", lambda shape, dtype, device, stream, strides=None: gpu(shape, dtype, strides))


def q(rows, cols, strides=None):
    return gpu((rows, cols), E4M3, strides)


def s(rows, blocks):
    return gpu((rows, blocks))


def ints(*shape):
    return gpu(shape, torch.int32)


WIDE = [
    lambda: sg.quantize_fp8(gpu((2, 300), strides=(FAR, 1))),
    lambda: sg.quantize_fp8(gpu((2 ** 32 + 5, 1))),
    lambda: sg.quantize_fp8(gpu((5, 8)), index=ints(2 ** 32 + 5), stream=_Stream()),
    lambda: sg.quantize_fp8(gpu((2, 300), strides=(FAR, 1)), blocks=True),
    lambda: sg.quantize_fp8_cols(gpu((2, 300), strides=(FAR, 1))),
    lambda: sg.quantize_fp8_cols(gpu((5, 8)), offsets=ints(2 ** 32 + 5)),
    lambda: sg.gemm_fp8(q(2, 300, (FAR, 1)), s(2, 3), q(4, 300), s(4, 3)),
    lambda: sg.gemm_fp8(q(2, 300), s(2, 3), q(4, 300, (FAR, 1)), s(4, 3)),
    lambda: sg.gemm_fp8(q(2 ** 32 + 2, 8), s(2 ** 32 + 2, 1), q(4, 8), s(4, 1)),
    lambda: sg.gemm_fp8(q(2, 300), s(2, 3), q(4, 300), s(4, 3), gpu((2, 4), strides=(FAR, 1))),
    lambda: sg.gemm_fp8_experts(q(2, 300, (FAR, 1)), s(2, 3), gpu((1, 4, 300), E4M3), gpu((1, 4, 3)), ints(2)),
    lambda: sg.gemm_fp8_experts(q(2, 300), s(2, 3), gpu((1, 4, 300), E4M3, (0, FAR, 1)), gpu((1, 4, 3)), ints(2)),
    lambda: sg.gemm_fp8_experts_wgrad(q(2, 256, (FAR, 1)), s(2, 2), q(4, 256), s(4, 2), ints(2)),
    lambda: sg.route(gpu((2, 8), strides=(FAR, 1)), 2),
    lambda: sg.route(gpu((2 ** 32 + 2, 8)), 2),
    lambda: sg.route_backward(gpu((2, 8), strides=(FAR, 1)), ints(2, 2), gpu((2, 2))),
    lambda: sg.route_plan(ints(2 ** 32 + 2, 2), 4),
    lambda: sg.route_plan(ints(2, 2 ** 32 + 2), 4),
    lambda: sg.route_combine(gpu((4, 8), strides=(FAR, 1)), ints(2, 2), gpu((2, 2))),
    lambda: sg.route_combine(gpu((4, 8)), ints(2 ** 32 + 2, 1), gpu((2 ** 32 + 2, 1))),
    lambda: sg.route_combine_backward(gpu((2, 8), strides=(FAR, 1)), gpu((4, 8)), ints(2, 2), gpu((2, 2))),
    lambda: _binding._ld(gpu((2, 300), strides=(FAR, 1)), "A"),
    lambda: _binding._ld(gpu((1, 2 ** 32 + 300)), "A"),
    lambda: sg.gemm(gpu((2, 300), strides=(FAR, 1)), gpu((300, 4)), gpu((2, 4)), stream=_Stream()),
    lambda: sg.matmul(gpu((2, 300)), gpu((300, 4), strides=(FAR, 1)), gpu((2, 4)), stream=_Stream()),
    lambda: sg.gemm_strided_batched(gpu((2 ** 32 + 1, 1, 1)), gpu((1, 1, 1)), gpu((2 ** 32 + 1, 1, 1)), stream=_Stream()),
]


@pytest.mark.parametrize("call", WIDE, ids=range(len(WIDE)))
def test_sizes_and_strides_past_32_bits_are_refused(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("k,groups,top", [(2 ** 32 + 2, 1, 1), (-2 ** 32 + 2, 1, 1), (2, 2 ** 32 + 1, 1), (2, 1, 2 ** 32 + 1),
                                          (2, -2 ** 32 + 1, 1), (2, 1, -2 ** 32 + 1), (2, 2, 3)])
def test_counts_past_32_bits_are_refused(k, groups, top):
    with pytest.raises(sg.SgemmError) as e:
        sg.route(gpu((2, 8)), k, groups=groups, top_groups=top, stream=_Stream())
    assert e.value.code in (sg.ERR_ROUTE, sg.ERR_DIM)


@pytest.mark.parametrize("experts", [2 ** 32 + 4, -2 ** 32 + 4, 0, 1025])
def test_experts_past_32_bits_are_refused(experts):
    with pytest.raises(sg.SgemmError) as e:
        sg.route_plan(ints(2, 2), experts, stream=_Stream())
    assert e.value.code in (sg.ERR_ROUTE, sg.ERR_DIM)


def call_with(fn, far):
    """The call with tensor number `far` of `fn`'s list on another GPU."""
    made = []

    def on(shape, dtype=torch.float32):
        made.append(gpu(shape, dtype, at=1 if len(made) == far else 0))
        return made[-1]

    return fn(on)


TOGETHER = [  # the call and the number of its tensors
    (lambda t: sg.quantize_fp8(t((5, 8)), index=t((4,), torch.int32), stream=_Stream()), 2),
    (lambda t: sg.quantize_fp8_cols(t((5, 8)), index=t((4,), torch.int32), offsets=t((3,), torch.int32), stream=_Stream()), 3),
    (lambda t: sg.gemm_fp8(t((2, 300), E4M3), t((2, 3)), t((4, 300), E4M3), t((4, 3)), t((2, 4)), stream=_Stream()), 5),
    (lambda t: sg.gemm_fp8_experts(t((2, 300), E4M3), t((2, 3)), t((2, 4, 300), E4M3), t((2, 4, 3)), t((3,), torch.int32),
                                   t((2, 4)), stream=_Stream()), 6),
    (lambda t: sg.gemm_fp8_experts_wgrad(t((2, 256), E4M3), t((2, 2)), t((4, 256), E4M3), t((4, 2)), t((3,), torch.int32),
                                         t((2, 2, 4)), stream=_Stream()), 6),
    (lambda t: sg.route(t((2, 8)), 2, bias=t((8,)), stream=_Stream()), 2),
    (lambda t: sg.route_backward(t((2, 8)), t((2, 2), torch.int32), t((2, 2)), stream=_Stream()), 3),
    (lambda t: sg.route_plan(t((2, 2), torch.int32), 4, stream=_Stream()), 1),
    (lambda t: sg.route_combine(t((4, 8)), t((2, 2), torch.int32), t((2, 2)), t((2, 8)), stream=_Stream()), 4),
    (lambda t: sg.route_combine_backward(t((2, 8)), t((4, 8)), t((2, 2), torch.int32), t((2, 2)), stream=_Stream()), 4),
]


@pytest.mark.parametrize("fn,far", [(fn, far) for fn, count in TOGETHER for far in range(count)],
                         ids=[f"{i}-{far}" for i, (fn, count) in enumerate(TOGETHER) for far in range(count)])
def test_tensors_and_stream_have_to_be_on_one_gpu(fn, far):
    with pytest.raises(ValueError, match="GPU 1"):
        call_with(fn, far)
    with pytest.raises(sg.SgemmError):  # all together: the C call is reached, and refuses tensors without memory
        call_with(fn, None)


@pytest.mark.parametrize("call", [
    lambda: sg.gemm_fp8(q(2, 300), gpu((5, 2, 3)), q(4, 300), s(4, 3), stream=_Stream()),
    lambda: sg.gemm_fp8(q(2, 300), s(2, 3), q(4, 300), gpu((5, 4, 3)), stream=_Stream()),
    lambda: sg.gemm_fp8(q(2, 300), gpu((6,)), q(4, 300), s(4, 3), stream=_Stream()),
    lambda: sg.gemm_fp8_experts(q(2, 300), gpu((5, 2, 3)), gpu((2, 4, 300), E4M3), gpu((2, 4, 3)), ints(3), stream=_Stream()),
    lambda: sg.gemm_fp8_experts_wgrad(q(2, 256), gpu((5, 2, 2)), q(4, 256), s(4, 2), ints(3), stream=_Stream()),
    lambda: sg.gemm_fp8_experts_wgrad(q(2, 256), s(2, 2), q(4, 256), gpu((5, 4, 2)), ints(3), stream=_Stream())])
def test_scales_have_the_axes_of_their_operand(call):
    with pytest.raises(ValueError):
        call()


def test_messages_cover_the_calls_that_return_them():
    """route_plan returns ERR_WORKSPACE, too, and 2-byte types have no 4-byte alignment."""
    workspace = sg.strerror(sg.ERR_WORKSPACE)
    assert "workspace" in workspace and "splitk" not in workspace and "streamk" not in workspace
    assert "4-byte" not in sg.strerror(sg.ERR_ALIGN)
    for code, word in ((sg.ERR_ALIAS, "output"), (sg.ERR_STRIDE, "scales"), (sg.ERR_DIM, "experts"), (sg.ERR_OP, "option")):
        assert word in sg.strerror(code)
    codes = range(-14, 1)
    assert len({sg.strerror(c) for c in codes}) == len(codes)
