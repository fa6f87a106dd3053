"""Single rows of the 16-bit experts' products: of any stride, NaN behind them, through the wrappers and the C calls."""
from __future__ import annotations

import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _gpu as G
from tests import test_experts16_gpu as E

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("N,K", [(1001, 512), (1000, 1000), (1, 1001), (999, 1), (1, 8), (300, 1000), (72, 65), (8, 7)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (3, 8), (8, 1)])
def test_single_rows(form, N, K, pad, offset):
    counts = [0, 1, 0] if (N + K) % 3 else [1]
    off = E.counts_to(counts)
    x, w = E.matrix((1, K if form != "dgrad" else N), 1, "bf16", pad, offset), E.matrix((len(counts), N, K), 2, "bf16", pad, offset)
    a, b = (x, w) if form != "wgrad" else (E.matrix((1, N), 2, "bf16", pad, offset), x)
    print(f"[gpu] {form} {counts} {N}x{K} pad {pad} offset {offset}", flush=True)
    want, size = E.expected(form, a, b, off.tolist())
    inner = {"forward": K, "dgrad": N, "wgrad": 1}[form]
    C = E.run(form, a, b, off, dtype=torch.float32)
    E.check(C, want, size, inner, "fp32")
    # the C call takes the stride as it is given
    D = torch.full_like(C, float("nan"))
    ints = (1, 0, 1, N, K, len(counts), a.data_ptr(), N + pad if form != "forward" else K + pad, b.data_ptr(), K + pad)
    stream = torch.cuda.current_stream().cuda_stream
    if form == "wgrad":
        code = sg.sgemm_mi355_experts_gemm_wgrad(*ints, off.data_ptr(), 0.0, D.data_ptr(), K, N * K, stream)
    else:
        call = sg.sgemm_mi355_experts_gemm if form == "forward" else sg.sgemm_mi355_experts_gemm_dgrad
        code = call(*ints, N * (K + pad), off.data_ptr(), D.data_ptr(), D.shape[1], stream)
    torch.cuda.synchronize()
    assert code == sg.OK
    E.check(D, want, size, inner, "fp32")
