"""FP32 results of 16-bit matrices: the bias' gradient and activations to which something is added before the rounding."""
from __future__ import annotations

import numpy as np
import pytest
import torch
from scipy import special

import dense_fp32_matrix_02_amd as sg
from tests import _fp8 as R
from tests import _gpu as G
from tests import _layer as L

pytestmark = pytest.mark.gpu

KINDS = ["fp32", "bf16", "fp16"]


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()


def arguments(kind):
    """Every magnitude that an activation tells apart, both signs, as the type holds them."""
    mags = np.concatenate([2.0 ** np.arange(-24, 8), np.linspace(0.001, 12, 4000), np.linspace(12, 200, 500), [0.0]])
    return torch.from_numpy(np.concatenate([mags, -mags])).to(R.TYPES[kind])


@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("kind", KINDS)
def test_bias_gradient_is_an_fp32_value(act, kind):
    """Of a single row the sum is the FP32 value of dP itself: off by the long slope's error, and SiLU's by what an
    exponent without correction (off by two roundings) changes s and 1 - s by."""
    p = arguments(kind).to("cuda")[None]
    _, db = sg.epilogue_backward(torch.ones_like(p), p, activation=act)
    q = L.plain(p)[0]
    _, slope, _, error = L.activation(q, act)
    if act == "silu":
        error = error + 2 * np.abs(q) * special.expit(q) * special.expit(-q) * (1 + np.abs(q))
    off = np.abs(L.plain(db) - slope) / (L.U * (error + np.abs(slope)) + 1e-300)
    assert (off <= 1.0).all(), (off.max(), q[off.argmax()])


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("kind", KINDS)
def test_bias_gradient_of_like_rows(act, kind):
    """Rows of one value each: an error of the slope enters every term alike. 40 rows are added by 64 additions at most."""
    p = arguments(kind)[:4500:9].to("cuda").expand(40, -1).contiguous()
    _, db = sg.epilogue_backward(torch.ones_like(p), p, activation=act)
    q = L.plain(p[0])
    _, slope, _, error = L.activation(q, act)
    assert (np.abs(L.plain(db) - 40 * slope) <= 40 * L.U * (error + 2 * np.abs(q) + 65 * np.abs(slope))).all()


def biases(M, N, K):
    """Operands of zeros, so that p is the bias; M and K choose the kernel."""
    A, B = (torch.zeros(n, K + K % 2, device="cuda").to(torch.float8_e4m3fn)[:, :K] for n in (M, N))
    return A, torch.ones(M, -(-K // 128), device="cuda"), B, torch.ones(N, -(-K // 128), device="cuda")


def forward_error(p, act, kind):
    """(value, its FP32 error in U): SiLU's exponent goes uncorrected in 16-bit results, off by two roundings."""
    value, _, error, _ = L.activation(p, act)
    if act == "silu" and kind != "fp32":
        error = error + 2 * np.abs(p) * special.expit(-p) * np.abs(value)
    return value, error


KERNELS = [(3, 0), (3, 128), (2000, 128), (2000, 127), (300, 4096)]


@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,K", KERNELS)
def test_residual_that_cancels_the_activation(act, kind, M, K):
    """A residual of -act(p) rounded to its type leaves what that rounding lost: act(p) has to be an FP32 value."""
    bias = arguments(kind)[:4100:3].float().to("cuda")
    value, error = forward_error(L.plain(bias)[None], act, kind)
    residual = torch.from_numpy(-value).to(R.TYPES[kind]).to("cuda").expand(M, -1).contiguous()
    for sums in (False, True):
        C = sg.gemm_fp8_epilogue(*biases(M, bias.numel(), K), bias=bias, activation=act, residual=residual, fp32_sums=sums)
        want = value + L.plain(residual[:1])
        assert bool((C == C[:1]).all())
        # the value's error, and the addition's
        L.near(C[:1], want, L.U * (error + np.abs(want)) + 1e-300, kind)


@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,K", KERNELS)
def test_activations_with_fp32_sums(act, kind, M, K):
    """fp32_sums without a residual: the FP32 value, rounded once."""
    bias = arguments(kind).float().to("cuda")
    value, error = forward_error(L.plain(bias)[None], act, kind)
    C = sg.gemm_fp8_epilogue(*biases(M, bias.numel(), K), bias=bias, activation=act, dtype=R.TYPES[kind], fp32_sums=True)
    L.near(C[:1], value, L.U * error + 1e-300, kind)
    assert bool((C == C[:1]).all())


def test_silu_near_the_least_exponential():
    """Down to p = -87.3 a relative error; below, where exp(p) < 2^-126 counts as zero, 1.1e-36 at most."""
    g = torch.linspace(-110, -80, 3001)
    z = L.plain(sg.gated(torch.stack([g, torch.ones_like(g)], 1).to("cuda")))[:, 0]
    p = g.double().numpy()
    value, _, error, _ = L.activation(p, "silu")
    above = p > -87.3
    assert (np.abs(z - value)[above] <= (L.U * 12 * np.abs(value))[above]).all()  # tests/_layer.py: 10, and gated's product
    assert (np.abs(z - value) <= 1.1e-36 + L.U * 12 * np.abs(value)).all() and (z[p < -87.4] == 0).all()
