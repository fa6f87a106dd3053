"""The choice of the FP8 products' kernels, asked on the host (no GPU needed)."""
from __future__ import annotations

import os

import numpy as np
import pytest

import dense_fp32_matrix_02_amd as sg
from tests import _fp8 as R

X = 0x10_0000_0000  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(sg.LIB_PATH):
        from dense_fp32_matrix_02_amd import build
        build.build()
    return sg.load()


GOOD = dict(form=0, type=1, M=4096, N=4096, K=4096, experts=0, A=X, lda=4096, B=X, ldb=4096, strideB=0)


@pytest.mark.parametrize("bad", [dict(form=3), dict(form=-1), dict(type=3), dict(type=3 | sg.FP32_SUMS), dict(M=0), dict(N=0), dict(K=-1), dict(form=1),
                                 dict(form=2, experts=0), dict(lda=0), dict(ldb=0), dict(form=1, experts=4, strideB=-16)])
def test_no_name_where_nothing_runs(bad):
    assert sg.sgemm_mi355_fp8_kernel_name(**GOOD) == "tile_256x256_fp8"
    assert sg.sgemm_mi355_fp8_kernel_name(**dict(GOOD, **bad)) is None


@pytest.mark.parametrize("change,name", [
    (dict(M=8), "rows_16_bf16"), (dict(M=8, type=0), "rows_16_bf16"), (dict(type=0), "tile_128x128_bf16"),
    (dict(A=X + 1), "staged_128x128_bf16"), (dict(ldb=4097), "staged_128x128_bf16"), (dict(K=15), "staged_128x128_bf16"),
    (dict(form=1, experts=4, strideB=8), "staged_128x128_bf16"), (dict(strideB=8), "tile_256x256_fp8"),
    (dict(type=1 | sg.FP32_SUMS), "tile_128x128_bf16"), (dict(type=0 | sg.FP32_SUMS), "tile_128x128_bf16")])
def test_names(change, name):
    assert sg.sgemm_mi355_fp8_kernel_name(**dict(GOOD, **change)) == name


def test_a_wrong_choice_of_ties_is_seen():
    """An oracle that takes the higher index of equal values (planted) differs from the one that the tests use."""
    logits = np.array([[0.0, 2.0, 2.0, 1.0, 2.0]], np.float32)
    right = R.route(logits, 2)[1]
    planted = logits.shape[1] - 1 - R.route(logits[:, ::-1], 2)[1]
    assert right.tolist() == [[1, 2]] and planted.tolist() == [[4, 2]]
    assert (right != planted).any()


def test_workspace_of_the_largest_plans():
    runs = -(-268435315 * 8 // 2048)  # in 512 groups, and a row for all
    assert sg.sgemm_mi355_route_plan_workspace_size(268435315, 8, 3) == (runs + 512 + 1) * 16
    assert sg.sgemm_mi355_route_plan_workspace_size(2 ** 31 - 1, 32, 3) == 0  # more than the call takes
