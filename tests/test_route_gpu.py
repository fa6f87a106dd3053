"""Routing, the sorted rows and their weighted return on the GPU against plain 64-bit definitions."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _fp8 as R
from tests import _gpu as G

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24  # half a step of FP32, relative


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()


def logits_of(T, E, seed, kind="fp32", spread=1.5, pad=0):
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * spread
    room = torch.full((T, E + pad), float("nan"), dtype=R.TYPES[kind])
    room[:, :E] = x.to(R.TYPES[kind])
    return room.to("cuda")[:, :E]


CASES = [  # tokens, experts, k, score, bias, groups, top_groups, renorm, scale, kind, pad
    (1, 1, 1, "softmax", False, 1, 1, True, 1.0, "fp32", 0),
    (1, 8, 2, "softmax", False, 1, 1, False, 1.0, "bf16", 0),
    (3, 64, 6, "softmax", False, 1, 1, True, 1.0, "fp32", 1),
    (5, 60, 4, "sigmoid", True, 1, 1, True, 2.5, "fp16", 3),
    (65, 128, 8, "softmax", True, 4, 2, False, 1.0, "bf16", 0),
    (33, 160, 6, "sigmoid", True, 8, 3, True, 2.5, "fp32", 0),
    (130, 256, 8, "sigmoid", True, 8, 4, True, 2.5, "fp32", 0),
    (70, 256, 8, "sigmoid", False, 8, 4, True, 1.0, "bf16", 0),
    (9, 100, 32, "softmax", False, 1, 1, True, 1.0, "fp32", 5),
    (7, 500, 10, "sigmoid", True, 10, 2, True, 1.0, "fp32", 0),
    (4, 1024, 16, "softmax", False, 512, 8, True, 1.0, "fp32", 0),
    (6, 96, 5, "softmax", False, 96, 5, True, 1.0, "fp32", 0),  # groups of one expert
    (4, 300, 3, "softmax", True, 100, 70, False, 1.0, "fp16", 0),
]


@pytest.mark.parametrize("case", CASES)
def test_route_and_gradient(case):
    T, E, k, score, has_bias, groups, top, renorm, scale, kind, pad = case
    print(f"[gpu] route {case}", flush=True)
    L = logits_of(T, E, T + E, kind, pad=pad)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(2)).to("cuda") * 0.05 if has_bias else None
    w, ids = sg.route(L, k, bias=bias, score=score, groups=groups, top_groups=top, renorm=renorm, scale=scale)
    l = L.float().cpu().numpy()
    want, at, S = R.route(l, k, None if bias is None else bias.cpu().numpy(), score, groups, top, renorm, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), at)
    # 64-bit inside (its error is far below), one rounding to FP32
    assert (np.abs(w.double().cpu().numpy() - want) <= 1.01 * STEP * np.abs(want)).all()
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(3)).to("cuda")
    dl = sg.route_backward(L, ids, dw, score=score, renorm=renorm, scale=scale).double().cpu().numpy()
    grad = R.route_grad(S, at, dw.double().cpu().numpy(), score, renorm, scale)
    # one rounding, and 64-bit sums of terms that may cancel
    size = np.abs(dw.double().cpu().numpy()).sum(1, keepdims=True) * scale * (1 / np.take_along_axis(S, at, 1).sum(1, keepdims=True) if renorm else 1.0)
    assert (np.abs(dl - grad) <= 1.01 * STEP * np.abs(grad) + 1e-13 * size).all()


@pytest.mark.parametrize("experts,groups", [
    (2, 2), (6, 3), (48, 3), (64, 2), (64, 8), (64, 16), (128, 64), (120, 15), (128, 4), (256, 4), (256, 16), (256, 64), (240, 60),
    (512, 4), (512, 2), (1024, 8), (1024, 64), (960, 15)])
def test_groups_of_many_sizes(experts, groups):
    for score in ("softmax", "sigmoid"):
        for top in {1, (groups + 1) // 2, groups}:
            test_route_and_gradient((11, experts, min(8, experts // groups * top), score, True, groups, top, True, 1.0, "fp32", 0))
    # equal values, within a group and between groups
    L = torch.randint(0, 3, (20, experts), generator=torch.Generator().manual_seed(1)).float()
    top = (groups + 1) // 2
    for score in ("softmax", "sigmoid"):
        k = min(32, experts // groups * top)
        _, ids = sg.route(L.to("cuda"), k, score=score, groups=groups, top_groups=top)
        np.testing.assert_array_equal(ids.cpu().numpy(), R.route(L.numpy(), k, None, score, groups, top)[1])


@pytest.mark.parametrize("experts", [5, 64, 100, 256, 700])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_of_repeated_ids(score, experts):
    """Ids that are not route's own may name an expert twice: both parts count."""
    L = logits_of(9, experts, 4)
    ids = torch.randint(0, experts, (9, 6), generator=torch.Generator().manual_seed(2))
    ids[0] = torch.tensor([3, 1, 3, 3, 4, 1])
    ids[1] = 2
    dw = torch.randn(9, 6, generator=torch.Generator().manual_seed(3))
    got = sg.route_backward(L, ids.int().to("cuda"), dw.to("cuda"), score=score, renorm=False, scale=1.5).double().cpu().numpy()
    S = R.route(L.cpu().numpy(), 1, None, score)[2]
    want = np.zeros((9, experts))
    for k in range(6):
        want += R.route_grad(S, ids[:, k:k + 1].numpy(), dw[:, k:k + 1].double().numpy(), score, False, 1.5)
    size = 1.5 * np.abs(dw.double().numpy()).sum(1, keepdims=True)
    assert (np.abs(got - want) <= 1.01 * STEP * np.abs(want) + 1e-13 * size).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    """Central differences of the weights as the 64-bit definition computes them, the choice held fixed."""
    T, E, k = 3, 40, 5
    L = logits_of(T, E, 9)
    w, ids = sg.route(L, k, score=score, renorm=renorm, scale=1.5)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(3))
    dl = sg.route_backward(L, ids, dw.to("cuda"), score=score, renorm=renorm, scale=1.5).cpu().numpy()
    l, at, d = L.double().cpu().numpy(), ids.cpu().numpy(), dw.double().numpy()

    def loss(x):
        s = np.exp(x - x.max(1, keepdims=True)) if score == "softmax" else 1 / (1 + np.exp(-x))
        s = s / s.sum(1, keepdims=True) if score == "softmax" else s
        c = np.take_along_axis(s, at, 1)
        return (d * 1.5 * (c / c.sum(1, keepdims=True) if renorm else c)).sum(1)

    step = 1e-5
    for e in range(E):
        bump = np.zeros((1, E))
        bump[0, e] = step
        slope = (loss(l + bump) - loss(l - bump)) / (2 * step)
        # the difference's own error: step^2 of a third derivative of order 1, and 2^-53 / step
        np.testing.assert_allclose(dl[:, e], slope, rtol=2 * STEP, atol=1e-9)


def test_ties_take_the_lowest_index():
    T, E = 4, 256
    L = torch.zeros(T, E, device="cuda")
    L[1, 100:] = 1.0
    L[2, ::3] = 2.0
    L[3, 255] = 1.0
    for score in ("softmax", "sigmoid"):
        for groups, top in ((1, 1), (8, 3)):
            _, ids = sg.route(L, 8, score=score, groups=groups, top_groups=top)
            _, want, _ = R.route(L.cpu().numpy(), 8, None, score, groups, top)
            np.testing.assert_array_equal(ids.cpu().numpy(), want)
    # neighbours that FP32 scores would not tell apart
    L = (20.0 + torch.arange(64).flip(0) * 2.0 ** -19).repeat(2, 1).to("cuda")
    _, ids = sg.route(L, 6, score="sigmoid")
    np.testing.assert_array_equal(ids.cpu().numpy(), R.route(L.cpu().numpy(), 6, None, "sigmoid")[1])


def test_special_logits():
    inf, nan = float("inf"), float("nan")
    L = torch.randn(6, 70, generator=torch.Generator().manual_seed(1))
    L[0, 10:] = -inf           # fewer experts with a score than are chosen
    L[1, :] = -inf             # none
    L[2, 5] = nan
    L[3, 5] = inf
    L[4, :] = torch.finfo(torch.float32).min
    L[5, :69] = torch.finfo(torch.float32).min
    for score in ("softmax", "sigmoid"):
        w, ids = sg.route(L.to("cuda"), 16, score=score)
        w, ids = w.cpu(), ids.cpu()
        assert all(len(set(r.tolist())) == 16 and 0 <= min(r) and max(r) < 70 for r in ids)
        want, at, _ = R.route(L.numpy(), 16, None, score)
        rows = [0, 4, 5] if score == "softmax" else [0, 1, 2, 3, 4, 5]
        np.testing.assert_array_equal(ids.numpy()[rows], at[rows])
        np.testing.assert_allclose(w.numpy()[rows], want[rows], rtol=1.01 * STEP)
        if score == "softmax":
            assert bool(w[1:4].isnan().all())
        else:
            assert 5 not in ids[2].tolist()
        g = sg.route_backward(L.to("cuda"), ids.to("cuda"), torch.ones(6, 16, device="cuda"), score=score)
        assert bool(g[[0, 4, 5]].isfinite().all())
    # a token whose chosen scores are all zero gets zero weights and zero gradients
    L = torch.full((1, 70), -1e4, device="cuda")
    w, ids = sg.route(L, 4, score="sigmoid")
    assert bool((w == 0).all())
    assert bool((sg.route_backward(L, ids, torch.ones(1, 4, device="cuda"), score="sigmoid") == 0).all())


def test_backward_skips_ids_outside():
    L = logits_of(2, 10, 1)
    ids = torch.tensor([[1, -1, 10], [3, 4, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    dw = torch.tensor([[1.0, 5.0, 7.0], [1.0, 2.0, 9.0]], device="cuda")
    got = sg.route_backward(L, ids, dw, renorm=False).double().cpu().numpy()
    S = R.route(L.cpu().numpy(), 1)[2]
    for t, some in enumerate(([1], [3, 4])):
        want = R.route_grad(S[t:t + 1], np.array([some]), dw[t:t + 1, :len(some)].double().cpu().numpy(), "softmax", False, 1.0)
        np.testing.assert_allclose(got[t], want[0], rtol=2 * STEP, atol=1e-15)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (3, 2, 5), (64, 1, 64), (65, 4, 7), (200, 6, 64), (1000, 8, 256), (2000, 3, 1024),
                                   (4097, 1, 100), (700, 32, 33)])
def test_plan(T, k, E):
    print(f"[gpu] plan {T} {k} {E}", flush=True)
    g = torch.Generator().manual_seed(T)
    for ids in (torch.randint(0, E, (T, k), generator=g), torch.randint(-2, E + 3, (T, k), generator=g), torch.full((T, k), E - 1),
                torch.full((T, k), -1)):
        got = [x.cpu().numpy() for x in sg.route_plan(ids.int().to("cuda"), E)]
        for x, want in zip(got, R.plan(ids.numpy(), E)):
            np.testing.assert_array_equal(x, want)


def test_plan_of_no_tokens():
    offsets, tokens, place = sg.route_plan(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 10)
    torch.cuda.synchronize()
    assert offsets.tolist() == [0] * 11 and tokens.numel() == 0 and place.shape == (0, 4)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,k,N,pad", [(1, 1, 1, 0), (3, 2, 7, 1), (5, 4, 512, 0), (17, 8, 1000, 3), (130, 3, 260, 4), (2, 32, 4096, 0)])
def test_combine_and_gradient(kind, T, k, N, pad):
    print(f"[gpu] combine {kind} {T} {k} {N}", flush=True)
    g = torch.Generator().manual_seed(T * k)
    Z = torch.full((T * k, N + pad), float("nan"), dtype=R.TYPES[kind])
    Z[:, :N] = torch.randn(T * k, N, generator=g).to(Z.dtype)
    dY = torch.randn(T, N, generator=g).to(Z.dtype)
    place = torch.randperm(T * k, generator=g).int().view(T, k)
    w = torch.randn(T, k, generator=g)
    Zd, wd, pd = Z.to("cuda")[:, :N], w.to("cuda"), place.to("cuda")
    Y = sg.route_combine(Zd, pd, wd).double().cpu().numpy()
    z, d, ww = Z[:, :N].double().numpy()[place.numpy()], dY.double().numpy(), w.double().numpy()
    want, size = (ww[..., None] * z).sum(1), (np.abs(ww)[..., None] * np.abs(z)).sum(1)
    half, least = R.half_step(kind)
    inside = k * STEP * size
    assert (np.abs(Y - want) <= inside + half * (np.abs(want) + inside) + least).all()
    dZ, dw = sg.route_combine_backward(dY.to("cuda"), Zd, pd, wd)
    grad = np.empty((T * k, N))
    grad[place.numpy()] = ww[..., None] * d[:, None]
    # a product rounded to FP32, then to the type
    assert (np.abs(dZ.double().cpu().numpy() - grad) <= (half + STEP * (1 + half)) * np.abs(grad) + least).all()
    slope, size = (z * d[:, None]).sum(-1), np.abs(z * d[:, None]).sum(-1)
    assert (np.abs(dw.double().cpu().numpy() - slope) <= (N + 6) * STEP * size).all()


def test_combine_skips_places_outside():
    Z = torch.ones(4, 16, device="cuda")
    place = torch.tensor([[0, -1], [4, 2 ** 31 - 1], [2, 3]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[2.0, 3.0], [5.0, 7.0], [1.0, 0.5]], device="cuda")
    Y = sg.route_combine(Z, place, w)
    assert Y[:, 0].tolist() == [2.0, 0.0, 1.5]
    dZ, dw = sg.route_combine_backward(torch.ones(3, 16, device="cuda"), Z, place, w)
    assert dw.tolist() == [[16.0, 0.0], [0.0, 0.0], [16.0, 16.0]]
    assert dZ[[0, 2, 3], 0].tolist() == [2.0, 1.0, 0.5]


def test_captured_calls_replay_on_another_stream():
    L = logits_of(300, 64, 1)
    Z = torch.randn(1200, 100, device="cuda")
    dY = torch.randn(300, 100, device="cuda")

    def work(stream=None):
        w, ids = sg.route(L, 4, stream=stream)
        off, tok, place = sg.route_plan(ids, 64, stream=stream)
        return [w, ids, off, tok, place, sg.route_backward(L, ids, w, stream=stream), sg.route_combine(Z, place, w, stream=stream),
                *sg.route_combine_backward(dY, Z, place, w, stream=stream)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for a, b in zip(work(side), work()):
        torch.cuda.synchronize()
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for i in range(4):
        L.copy_(logits_of(300, 64, 20 + i))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, work()):
            assert torch.equal(a, b)
