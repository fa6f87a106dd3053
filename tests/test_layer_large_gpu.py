"""Matrices of more than 2^31 elements and more rows than a grid has workgroups: the last rows, experts and sums, against
the same calls on the small matrices that hold them."""
from __future__ import annotations

import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _gpu as G

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
PICK = 300  # rows at the end that are compared


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()
    yield
    torch.cuda.empty_cache()


def pattern(rows, cols, seed):
    """rows x cols bf16 that differ from row to row, made on the GPU."""
    base = torch.randn(1031, cols, generator=torch.Generator().manual_seed(seed)).to(BF).to("cuda")
    return base[torch.arange(rows, device="cuda") % 1031]


def bits(x):
    return x.contiguous().view(torch.uint8)


@pytest.mark.parametrize("rows,cols", [(560000, 4096), (1100000, 2001), (4300000, 520)])
def test_norm(rows, cols):
    print(f"[gpu] rms_norm {rows}x{cols}", flush=True)
    x, w = pattern(rows, cols, 1), torch.linspace(0.5, 1.5, cols, device="cuda")
    Q, S, H, a = sg.rms_norm_fp8(x, w, residual=x)
    q, s, h, b = sg.rms_norm_fp8(x[-PICK:].contiguous(), w, residual=x[-PICK:].contiguous())
    assert torch.equal(bits(Q[-PICK:]), bits(q)) and torch.equal(S[-PICK:], s) and torch.equal(H[-PICK:], h) and torch.equal(a[-PICK:], b)
    del Q, S
    dX, dw = sg.rms_norm_backward(x, H, a, w, dH=x)
    dx, _ = sg.rms_norm_backward(x[-PICK:].contiguous(), h, b, w, dH=x[-PICK:].contiguous())
    assert torch.equal(dX[-PICK:], dx)
    want = torch.zeros(cols, dtype=torch.float64, device="cuda")
    for r in range(0, rows, 1 << 16):
        want += (x[r:r + (1 << 16)].double() * H[r:r + (1 << 16)].double() * a[r:r + (1 << 16), None].double()).sum(0)
    # every term is positive or all of a column's are of either sign at random; each is off by 3 half steps, and a sum of
    # up to rows / 512 / 4 + 40 additions in a row by as many
    size = want.abs() + rows ** 0.5
    assert bool(((dw.double() - want).abs() <= (rows / 512 + 50) * 2.0 ** -24 * (size + 3 * rows)).all())


def test_activations():
    rows, cols = 560000, 2048
    H = pattern(rows, 2 * cols, 2)
    Q, S, Z = sg.gated_fp8(H, wide=True)
    last = H[-PICK:].contiguous()
    q, s, z = sg.gated_fp8(last, wide=True)
    assert torch.equal(bits(Q[-PICK:]), bits(q)) and torch.equal(S[-PICK:], s) and torch.equal(Z[-PICK:], z)
    del Q, S
    dH = sg.gated_backward(Z, H)
    assert torch.equal(dH[-PICK:], sg.gated_backward(z, last))
    dP, db = sg.epilogue_backward(dH, H, activation="silu")
    dp, _ = sg.epilogue_backward(dH[-PICK:].contiguous(), last, activation="silu")
    assert torch.equal(dP[-PICK:], dp)
    want = sum(dP[r:r + (1 << 16)].double().sum(0) for r in range(0, rows, 1 << 16))
    size = sum(dP[r:r + (1 << 16)].double().abs().sum(0) for r in range(0, rows, 1 << 16))
    # dP is rounded to bf16, its sum is not; and the additions
    assert bool(((db.double() - want).abs() <= (2.0 ** -8 + 400 * 2.0 ** -24) * size).all())


@pytest.mark.parametrize("pad", [0, 1])
def test_experts(pad):
    """Weights and their gradients of 40 x 8192 x 8192 elements, aligned and not: the last expert's."""
    E, N, K, rows = 40, 8192, 8192, 700
    W = pattern(E * N, K + pad, 3).view(E, N, K + pad)[:, :, pad:]
    x, dy = pattern(rows, K, 4), pattern(rows, N, 5)
    for first in (0, 400, 690):  # tiles, few rows
        off = torch.full((E + 1,), first, dtype=torch.int32, device="cuda")
        off[0], off[-1] = 0, rows
        one = torch.tensor([0, rows - first], dtype=torch.int32, device="cuda")
        tail, dtail = x[first:].contiguous(), dy[first:].contiguous()
        want = sg.gemm_experts(tail, W[-1:].contiguous(), one).double()
        got = sg.gemm_experts(x, W, off)[first:].double()
        # the same products in another order: K additions, then the rounding to bf16
        size = tail.abs().double() @ W[-1].abs().double().t().contiguous()
        assert bool(((got - want).abs() <= 2 * K * 2.0 ** -23 * size + 2 * 2.0 ** -8 * want.abs()).all())
        got = sg.gemm_experts_dgrad(dy, W, off)[first:].double()
        want = sg.gemm_experts_dgrad(dtail, W[-1:].contiguous(), one).double()
        size = dtail.abs().double() @ W[-1].abs().double()
        assert bool(((got - want).abs() <= 2 * N * 2.0 ** -23 * size + 2 * 2.0 ** -8 * want.abs()).all())
        if first == 400:
            C = sg.gemm_experts_wgrad(dy, x, off)
            want = sg.gemm_experts_wgrad(dtail, tail, one)[0].double()
            size = dtail.abs().double().t().contiguous() @ tail.abs().double()
            assert bool(((C[-1].double() - want).abs() <= 2 * rows * 2.0 ** -23 * size).all()) and bool((C[1:-1:13] == 0).all())
            del C
