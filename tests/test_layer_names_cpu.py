"""The kernel that a product with an epilogue runs, by name: that of the product without one (no GPU needed)."""
from __future__ import annotations

import os

import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from dense_fp32_matrix_02_amd import _fp8, _layer
from tests.test_wrappers_cpu import E4M3, _Stream, gpu


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(sg.LIB_PATH):
        from dense_fp32_matrix_02_amd import build
        build.build()
    return sg.load()


@pytest.mark.parametrize("M,N,want", [(1, 6487, "rows"), (40, 1, "rows"), (1, 1, "rows"), (2, 6487, "staged"), (2, 1, "staged")])
def test_single_rows_are_loaded_directly_whatever_their_stride(monkeypatch, M, N, want):
    calls = []
    for module in (_fp8, _layer):
        monkeypatch.setattr(module, "_empty", lambda shape, dtype, device, stream, strides=None: gpu(shape, dtype, strides))
    monkeypatch.setattr(_layer, "_launch", lambda call, on, *args: calls.append(args) or 0)
    K, padded = 1559, 1568
    A = gpu((M, K), E4M3, (padded if M == 40 else K, 1))
    B = gpu((N, K), E4M3, (padded if N == 6487 else K, 1))
    sg.gemm_fp8_epilogue(A, gpu((M, 13)), B, gpu((N, 13)), dtype=torch.bfloat16, stream=_Stream())
    kind, m, n, k, a, lda, _, _, _, b, ldb = calls[0][:11]
    assert (m, n, k) == (M, N, K) and lda >= K <= ldb
    assert sg.sgemm_mi355_fp8_kernel_name(sg.FP8_DENSE, kind, m, n, k, 0, a, lda, b, ldb).startswith(want)
