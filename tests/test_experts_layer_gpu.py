"""The example of a layer of experts: each stage against 64 bits on the values it was given, and a falling loss."""
from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _fp8 as R
from tests import _gpu as G

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SPEC = importlib.util.spec_from_file_location("experts_layer", os.path.join(HERE, "examples", "experts_layer.py"))


@pytest.fixture(scope="module")
def example():
    G.require_gpu()
    module = importlib.util.module_from_spec(SPEC)
    SPEC.loader.exec_module(module)
    return module


def by_expert(x, weights, offsets):
    """(products, products of magnitudes) of rows by expert in 64 bits, for a quantised matrix's (Q, S) pairs."""
    a = R.values(R.bytes_of(x[0]), x[1].cpu().numpy())
    out, size = [], []
    for e in range(len(offsets) - 1):
        b = R.values(R.bytes_of(weights[0][e]), weights[1][e].cpu().numpy(), 128)
        rows = a[offsets[e]:offsets[e + 1]]
        out.append(rows @ b.T), size.append(np.abs(rows) @ np.abs(b).T)
    return np.concatenate(out), np.concatenate(size)


def near(got, want, size, K, kind):
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= R.product_bound(want, size, K, kind)).all()


def test_stages(example):
    T, D, F, E, k = 300, 256, 128, 6, 2
    layer = example.ExpertsLayer(D, F, E, k, seed=3)
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(4)).bfloat16().to("cuda")
    out, s = layer.forward(x)
    w, ids, S = R.route(s["logits"].cpu().numpy(), k)
    np.testing.assert_array_equal(s["experts"].cpu().numpy(), ids)
    for got, want in zip((s["offsets"], s["tokens"], s["place"]), R.plan(ids, E)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    off = s["offsets"].tolist()
    near(s["h"], *by_expert(sg.quantize_fp8(x, index=s["tokens"]), layer.q1, off), D, "bf16")
    near(s["y"], *by_expert(sg.quantize_fp8(s["z"]), layer.q2, off), F, "bf16")
    y, p = s["y"].double().cpu().numpy()[s["place"].cpu().numpy()], s["weights"].double().cpu().numpy()[..., None]
    want, size = (p * y).sum(1), np.abs(p * y).sum(1)
    assert (np.abs(out.double().cpu().numpy() - want) <= k * 2.0 ** -24 * size + 1.01 * 2.0 ** -8 * np.abs(want)
            + 1.01 * 2.0 ** -8 * k * 2.0 ** -24 * size).all()

    dout = (torch.randn(T, D, generator=torch.Generator().manual_seed(5)) * 0.01).bfloat16().to("cuda")
    g = layer.backward(dout, s)
    near(g["dz"], *by_expert(sg.quantize_fp8(g["dy"]), layer.q2t, off), D, "bf16")
    grad = R.route_grad(S, ids, g["dweights"].double().cpu().numpy(), "softmax", True, 1.0)
    np.testing.assert_allclose(g["dlogits"].double().cpu().numpy(), grad, rtol=1.01 * 2.0 ** -24, atol=1e-12)
    for name, left, right in (("w2", (g["dy"], None), (s["z"], None)), ("w1", (g["dh"], None), (x, s["tokens"]))):
        a, b = (sg.quantize_fp8_cols(m, index=i, offsets=s["offsets"]) for m, i in (left, right))
        a, b = R.values(R.bytes_of(a[0]), a[1].cpu().numpy()), R.values(R.bytes_of(b[0]), b[1].cpu().numpy())
        for e in range(E):
            at = 128 * (off[e] // 128 + e)
            to = at + off[e + 1] - off[e]
            near(g[name][e], a[:, at:to] @ b[:, at:to].T, np.abs(a[:, at:to]) @ np.abs(b[:, at:to]).T, max(to - at, 1), "fp32")


def test_loss_falls(example):
    losses = example.main(["--tokens", "512", "--width", "256", "--hidden", "128", "--experts", "8", "--choices", "2", "--steps", "4"])
    assert all(b < a for a, b in zip(losses, losses[1:]))
