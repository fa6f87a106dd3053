"""Every wrapper makes its tensors' GPU the current one for its C call: a default stream is the current GPU's (no GPU needed)."""
from __future__ import annotations

import contextlib

import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from dense_fp32_matrix_02_amd import _binding, _experts, _fp8, _layer, _route
from tests.test_wrappers_cpu import E4M3, gpu


class Stream:
    cuda_stream = 0
    device_index = 1


def at_1(shape, dtype=torch.float32, strides=None):
    return gpu(shape, dtype, strides, 1)


def b8(*shape):
    return at_1(shape, E4M3)


def i32(*shape):
    return at_1(shape, torch.int32)


BF = torch.bfloat16
CALLS = [
    lambda s: sg.matmul(at_1((2, 3)), at_1((3, 4)), stream=s), lambda s: sg.matmul(at_1((2, 3)), at_1((3, 4)), kind="valu", stream=s),
    lambda s: sg.matmul(at_1((2, 3)), at_1((3, 4)), config=0, stream=s), lambda s: sg.gemm(at_1((2, 3)), at_1((3, 4)), stream=s),
    lambda s: sg.gemm(at_1((2, 3)), at_1((3, 4)), config=0, stream=s),
    lambda s: sg.gemm_strided_batched(at_1((2, 2, 3)), at_1((2, 3, 4)), stream=s),
    lambda s: sg.gemm_strided_batched(at_1((2, 2, 3)), at_1((2, 3, 4)), config=0, stream=s),
    lambda s: sg.gemm_splitk(at_1((2, 3)), at_1((3, 4)), splits=1, stream=s),
    lambda s: sg.gemm_splitk(at_1((2, 3)), at_1((3, 4)), splits=1, config=0, stream=s),
    lambda s: sg.gemm_streamk(at_1((2, 3)), at_1((3, 4)), stream=s), lambda s: sg.gemm_streamk(at_1((2, 3)), at_1((3, 4)), config=0, stream=s),
    lambda s: sg.quantize_fp8(at_1((2, 8)), stream=s), lambda s: sg.quantize_fp8(at_1((2, 8)), blocks=True, stream=s),
    lambda s: sg.quantize_fp8_cols(at_1((2, 8)), stream=s), lambda s: sg.gemm_fp8(b8(2, 8), at_1((2, 1)), b8(3, 8), at_1((3, 1)), stream=s),
    lambda s: sg.gemm_fp8_experts(b8(2, 8), at_1((2, 1)), b8(2, 3, 8), at_1((2, 3, 1)), i32(3), stream=s),
    lambda s: sg.gemm_fp8_experts_wgrad(b8(4, 256), at_1((4, 2)), b8(3, 256), at_1((3, 2)), i32(3), stream=s),
    lambda s: sg.route(at_1((2, 8)), 2, stream=s), lambda s: sg.route_backward(at_1((2, 8)), i32(2, 2), at_1((2, 2)), stream=s),
    lambda s: sg.route_plan(i32(2, 2), 8, stream=s), lambda s: sg.route_combine(at_1((4, 8)), i32(2, 2), at_1((2, 2)), stream=s),
    lambda s: sg.route_combine_backward(at_1((2, 8)), at_1((4, 8)), i32(2, 2), at_1((2, 2)), stream=s),
    lambda s: sg.rms_norm_fp8(at_1((2, 8)), at_1((8,)), stream=s), lambda s: sg.rms_norm(at_1((2, 8)), at_1((8,)), stream=s),
    lambda s: sg.rms_norm_backward(at_1((2, 8)), at_1((2, 8)), at_1((2,)), at_1((8,)), stream=s), lambda s: sg.gated_fp8(at_1((2, 8)), stream=s),
    lambda s: sg.gated(at_1((2, 8)), stream=s), lambda s: sg.gated_backward(at_1((2, 4)), at_1((2, 8)), stream=s),
    lambda s: sg.gemm_fp8_epilogue(b8(2, 8), at_1((2, 1)), b8(3, 8), at_1((3, 1)), stream=s),
    lambda s: sg.epilogue_backward(at_1((2, 8)), at_1((2, 8)), stream=s),
    lambda s: sg.gemm_experts(at_1((2, 8), BF), at_1((2, 4, 8), BF), i32(3), stream=s),
    lambda s: sg.gemm_experts_dgrad(at_1((2, 4), BF), at_1((2, 4, 8), BF), i32(3), stream=s),
    lambda s: sg.gemm_experts_wgrad(at_1((2, 4), BF), at_1((2, 8), BF), i32(3), stream=s),
]


@pytest.mark.parametrize("call", CALLS, ids=range(len(CALLS)))
def test_the_tensors_gpu_is_current(monkeypatch, call):
    now, seen = [0], []

    @contextlib.contextmanager
    def device(i):
        was, now[0] = now[0], i
        yield
        now[0] = was

    class Library:
        """C calls that note the current GPU; workspaces have some bytes."""

        def __getattr__(self, name):
            return (lambda *a: 64) if name.endswith("_size") else lambda *a: seen.append(now[0]) or 0

    for module in (_fp8, _route, _layer, _experts):
        monkeypatch.setattr(module, "_c", Library())
        monkeypatch.setattr(module, "_empty", lambda shape, dtype, device, stream, strides=None: at_1(shape, dtype, strides))
    for name in ("", "_valu", "_with_config", "_strided_batched", "_strided_batched_with_config", "_splitk", "_splitk_with_config", "_streamk",
                 "_streamk_with_config"):
        monkeypatch.setattr(_binding, "sgemm_mi355" + name, lambda *a: seen.append(now[0]) or 0)
    for name in ("_splitk", "_streamk"):
        monkeypatch.setattr(_binding, f"sgemm_mi355{name}_workspace_size", lambda *a: 64)
    monkeypatch.setattr(_binding, "_empty_on", lambda shape, device, stream: at_1(shape))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(_layer, "_several", [])
    kept = _binding._several[:]
    _binding._several.clear()
    try:
        call(Stream())
    finally:
        _binding._several[:] = kept
    assert seen == [1] and now == [0]
