"""The kernels that single rows, single experts and sums over nothing run, by name: what the wrappers pass to the C calls,
and what the C query says of it (no GPU needed)."""
from __future__ import annotations

import os

import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from dense_fp32_matrix_02_amd import _experts, _fp8
from tests.test_wrappers_cpu import _Stream, gpu

A, W = 0x100_0000_0000, 0x200_0000_0000  # never dereferenced
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(sg.LIB_PATH):
        from dense_fp32_matrix_02_amd import build
        build.build()
    return sg.load()


@pytest.fixture
def passed(monkeypatch):
    """The arguments of the C calls, instead of the calls."""
    calls = []
    for module in (_fp8, _experts):
        monkeypatch.setattr(module, "_empty", lambda shape, dtype, device, stream, strides=None: gpu(shape, dtype, strides))
    monkeypatch.setattr(_experts, "_launch", lambda call, on, *args: calls.append(args) or 0)
    return calls


def name(form, rows, N, K, experts, lda, ldw, strideW=0):
    return sg.sgemm_mi355_experts_kernel_name(form, rows, N, K, experts, A, lda, W, ldw, strideW)


def name_of(form, args):
    """Of the wrapper's arguments: types, rows, N, K, experts, A, lda, W (B), ldw, strideW (offsets in the weights' form)."""
    rows, N, K, E = args[2:6]
    return name(form, rows, N, K, E, args[7], args[9], 0 if form == 2 else args[10])


def ints(n):
    return gpu((n,), torch.int32)


def test_single_rows_are_loaded_directly_whatever_their_stride(passed):
    sg.gemm_experts_dgrad(gpu((1, 1001), BF), gpu((1, 1001, 512), BF), ints(2), stream=_Stream())
    sg.gemm_experts_dgrad(gpu((1, 300), BF), gpu((4, 300, 1000), BF), ints(5), stream=_Stream())
    sg.gemm_experts_wgrad(gpu((1, 1000), BF, (1001, 1)), gpu((1, 1000), BF, (1003, 1)), ints(2), stream=_Stream())
    assert [name_of(f, a) for f, a in zip((1, 1, 2), passed)] == ["tile_128x128"] * 3
    sg.gemm_experts(gpu((1, 1001), BF), gpu((1, 1, 1001), BF), ints(2), stream=_Stream())
    assert passed[-1][7] % 8 == 0 and passed[-1][9] % 8 == 0 and passed[-1][7] >= 1001 <= passed[-1][9]
    # a second row counts
    sg.gemm_experts_dgrad(gpu((2, 1001), BF), gpu((1, 1001, 512), BF), ints(2), stream=_Stream())
    assert passed[-1][7] == 1001 and name_of(1, passed[-1]) == "staged_128x128"


@pytest.mark.parametrize("form,rows,N,K,lda,ldw", [(1, 1, 1001, 512, 1001, 512), (2, 1, 1000, 1000, 1001, 1003)])
def test_the_query_takes_a_single_rows_stride_as_the_call_does(form, rows, N, K, lda, ldw):
    """As it is given: the C calls round no stride."""
    assert name(form, rows, N, K, 1, lda, ldw) == "staged_128x128"
    assert name(form, rows, N, K, 1, lda + -lda % 8, ldw + -ldw % 8) == "tile_128x128"


@pytest.mark.parametrize("form", [0, 1])
def test_one_expert_has_no_stride(form):
    assert name(form, 300, 600, 72, 1, 600 if form else 72, 72, 12345) == name(form, 300, 600, 72, 1, 600 if form else 72, 72) == "tile_128x128"
    assert name(form, 300, 600, 72, 2, 600 if form else 72, 72, 12345) != "tile_128x128"


def test_sums_over_nothing_have_a_kernel_and_no_results_have_none():
    assert name(0, 5, 20, 0, 3, 8, 8) == name(1, 5, 0, 20, 3, 8, 24) == "staged_128x128" and name(2, 0, 64, 64, 3, 64, 64) is not None
    for form, rows, N, K in ((0, 0, 20, 30), (0, 5, 0, 30), (1, 0, 20, 30), (1, 5, 20, 0), (2, 5, 0, 30), (2, 5, 20, 0)):
        assert name(form, rows, N, K, 3, 32, 32, 960) is None
