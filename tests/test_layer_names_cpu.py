"""The kernel that a product with an epilogue runs, by name (no GPU needed)."""
from __future__ import annotations

import os

import pytest

import dense_fp32_matrix_02_amd as sg
from tests.test_fp8_kernels_cpu import GOOD, X


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(sg.LIB_PATH):
        from dense_fp32_matrix_02_amd import build
        build.build()
    return sg.load()


def name(M, N, K, lda, ldb, kind=1, form=sg.FP8_EPILOGUE):
    return sg.sgemm_mi355_fp8_kernel_name(form, kind, M, N, K, 0, X, lda, X, ldb)


@pytest.mark.parametrize("M,N,lda,ldb,want", [(1, 6487, 1559, 1568, "rows"), (40, 1, 1568, 1559, "rows"), (1, 1, 1559, 1559, "rows"),
                                              (2, 6487, 1559, 1568, "staged"), (40, 2, 1568, 1559, "staged")])
def test_single_rows_are_loaded_directly_whatever_their_stride(M, N, lda, ldb, want):
    assert name(M, N, 1559, lda, ldb).startswith(want)
    assert name(M, N, 1559, lda, ldb, form=sg.FP8_DENSE) == "staged_128x128_bf16"  # the product without one: as it is given


@pytest.mark.parametrize("change", [{}, dict(M=8), dict(type=0), dict(type=0, M=1500, K=2048), dict(A=X + 1), dict(ldb=4097), dict(K=15),
                                    dict(type=1 | sg.FP32_SUMS), dict(M=512, N=512)])
def test_otherwise_it_is_the_dense_products(change):
    args = dict(GOOD, **change)
    assert sg.sgemm_mi355_fp8_kernel_name(**dict(args, form=sg.FP8_EPILOGUE)) == sg.sgemm_mi355_fp8_kernel_name(**args)


@pytest.mark.parametrize("bad", [dict(type=3), dict(M=0), dict(N=0), dict(K=-1), dict(lda=0), dict(ldb=0), dict(form=3), dict(form=5)])
def test_no_name_where_nothing_runs(bad):
    assert sg.sgemm_mi355_fp8_kernel_name(**dict(GOOD, **dict(dict(form=sg.FP8_EPILOGUE), **bad))) is None
