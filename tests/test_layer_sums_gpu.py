"""Sums over millions of rows, the norm's weight gradient and the bias' one, to within their additions' roundings: a group of
rows that went missing would be seen."""
from __future__ import annotations

import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _gpu as G
from tests.test_layer_large_gpu import pattern

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
RUN = 1 << 16


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()
    yield
    torch.cuda.empty_cache()


def holds(got, want, size, each, teams, groups):
    """Sums of `each` rows by a thread, of the workgroup's teams, then of the groups: every 64th by a thread, these by
    four, and four shuffles; each term comes with three roundings."""
    bound = (each + teams + groups / 64 + 3 + 4 + 3) * U * size
    assert bool(((got.double() - want).abs() <= bound).all())
    assert bool((want.abs() / groups > 2 * bound).all())  # one group's share


@pytest.mark.parametrize("rows,cols,teams,groups", [(560000, 4096, 1, 1024), (1100000, 2001, 1, 1024), (4300000, 520, 4, 512)])
def test_weight_gradient_of_the_norm(rows, cols, teams, groups):
    print(f"[gpu] rms_norm_backward {rows}x{cols}", flush=True)
    assert sg.sgemm_mi355_rms_norm_backward_workspace_size(rows, cols) == groups * cols * 4
    x, w = pattern(rows, cols, 1), torch.linspace(0.5, 1.5, cols, device="cuda")
    _, H, a = sg.rms_norm(x, w)
    _, dw = sg.rms_norm_backward(x, H, a, w)
    want = torch.zeros(cols, dtype=torch.float64, device="cuda")  # every term is a square
    for r in range(0, rows, RUN):
        want += (x[r:r + RUN].double() * H[r:r + RUN].double() * a[r:r + RUN, None].double()).sum(0)
    holds(dw, want, want, -(-rows // (teams * groups)), teams, groups)


@pytest.mark.parametrize("rows,cols,teams,groups", [(560000, 4096, 4, 256), (4300000, 100, 16, 2048), (1100000, 2001, 4, 512)])
def test_bias_gradient(rows, cols, teams, groups):
    print(f"[gpu] epilogue_backward {rows}x{cols}", flush=True)
    assert sg.sgemm_mi355_epilogue_backward_workspace_size(rows, cols) == groups * cols * 4
    d = pattern(rows, cols, 2).abs_()
    dP, db = sg.epilogue_backward(d, d, activation="relu")  # positive: the slope is 1
    assert torch.equal(dP[-300:], d[-300:])
    want = sum(d[r:r + RUN].double().sum(0) for r in range(0, rows, RUN))
    holds(db, want, want, -(-rows // (teams * groups)), teams, groups)
