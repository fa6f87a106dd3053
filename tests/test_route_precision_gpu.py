"""The routing gradient where scores are nearly 1: 64-bit definitions without cancellation."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _gpu as G

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24  # half a step of FP32, relative


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()


def weights_gradient(s, dw, renorm, scale):
    """(gradient, sum of the magnitudes) of the chosen scores s: dw_j - sum_m dw_m s_m / S = sum_m s_m (dw_j - dw_m) / S."""
    if not renorm:
        return scale * dw, scale * np.abs(dw)
    apart, total = dw[:, None] - dw[None], s.sum()
    return scale * (apart * s[None]).sum(1) / total ** 2, scale * (np.abs(apart) * s[None]).sum(1) / total ** 2


def sigmoid_row(l, ids, dw, renorm, scale):
    t = np.exp(-np.abs(l))
    s = np.where(l < 0, t, 1.0) / (1 + t)
    d, size = weights_gradient(s[ids], dw, renorm, scale)
    slope = (t / (1 + t) ** 2)[ids]  # s (1 - s)
    out, mag = np.zeros_like(l), np.zeros_like(l)
    out[ids], mag[ids] = d * slope, size * slope
    return out, mag


def softmax_row(l, ids, dw, renorm, scale):
    s = np.exp(l - l.max())
    s = s / s.sum()
    d, size = weights_gradient(s[ids], dw, renorm, scale)
    ds, mag = np.zeros_like(l), np.zeros_like(l)
    ds[ids], mag[ids] = d, size
    other = 1.0 - np.eye(len(l))  # s_i (ds_i - sum_m ds_m s_m) = s_i sum_m s_m (ds_i - ds_m)
    return s * ((ds[:, None] - ds[None]) * s[None]).sum(1), s * ((mag[:, None] + mag[None]) * s[None] * other).sum(1)


@pytest.mark.parametrize("experts", [7, 100, 256, 600])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_gradient_of_far_logits(score, renorm, experts, kind):
    T, k = 40, 5
    print(f"[gpu] {score} gradient, {experts} experts, renorm {renorm} {kind}", flush=True)
    g = torch.Generator().manual_seed(experts)
    L = torch.randn(T, experts, generator=g)
    if score == "sigmoid":
        L += torch.linspace(-60, 60, T)[:, None]
    else:  # one expert ahead of the others by up to 60
        L[torch.arange(T), torch.randint(0, experts, (T,), generator=g)] += torch.linspace(0, 60, T)
    L = L.to(kind)
    dw = torch.randn(T, k, generator=g)
    _, ids = sg.route(L.to("cuda"), k, score=score)
    got = sg.route_backward(L.to("cuda"), ids, dw.to("cuda"), score=score, renorm=renorm, scale=1.5).double().cpu().numpy()
    row = sigmoid_row if score == "sigmoid" else softmax_row
    for t in range(T):
        want, size = row(L[t].double().numpy(), ids[t].cpu().numpy(), dw[t].double().numpy(), renorm, 1.5)
        # one rounding to FP32, and 64-bit sums of at most 600 terms
        assert (np.abs(got[t] - want) <= 1.01 * STEP * np.abs(want) + 1e-12 * size).all(), t


def test_gradient_of_one_choice_is_zero_with_renorm():
    """The weight of a token's only expert is the scale, whatever its score."""
    L = torch.randn(30, 64, generator=torch.Generator().manual_seed(1)) * 20
    for score in ("sigmoid", "softmax"):
        _, ids = sg.route(L.to("cuda"), 1, score=score)
        got = sg.route_backward(L.to("cuda"), ids, torch.full((30, 1), 0.3, device="cuda"), score=score)
        assert bool((got == 0).all())
