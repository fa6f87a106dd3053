"""The gradient of the experts' rows where places leave rows without a name: zeros, in memory that held NaN."""
from __future__ import annotations

import ctypes

import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _fp8 as R
from tests import _gpu as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()


def backward(dY, Z, place, w, dZ, dw):
    """The C call, into memory of the test's own."""
    code = {torch.float32: sg.F32, torch.bfloat16: sg.BF16, torch.float16: sg.F16}[Z.dtype]
    rc = sg.sgemm_mi355_route_combine_backward(
        code, *place.shape, *Z.shape, dY.data_ptr(), dY.stride(0), Z.data_ptr(), Z.stride(0), place.data_ptr(), w.data_ptr(),
        dZ.data_ptr(), dZ.stride(0), dw.data_ptr(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == sg.OK, sg.strerror(rc)


def case(tokens, k, rows, cols, kind, named, seed, pad=0):
    """Inputs with small whole numbers (gradients are exact) and `named` of the places inside the rows."""
    g = torch.Generator().manual_seed(seed)
    place = torch.full((tokens * k,), -1, dtype=torch.int64)
    at = torch.randperm(tokens * k, generator=g)[:named]
    place[at] = torch.randperm(rows, generator=g)[:named]
    place[torch.randperm(tokens * k, generator=g)[:3]] = torch.tensor([rows, 2 ** 31 - 1, -2 ** 31])[:min(3, tokens * k)]
    w = torch.randint(1, 5, (tokens, k), generator=g).float()
    dY = torch.randint(1, 4, (tokens, cols), generator=g).to(R.TYPES[kind])
    Z = torch.randint(-3, 4, (rows, cols), generator=g).to(R.TYPES[kind])
    room = torch.full((rows, cols + pad), float("nan"), dtype=R.TYPES[kind], device="cuda")
    return place.int().view(tokens, k).to("cuda"), w.to("cuda"), dY.to("cuda"), Z.to("cuda"), room


def expected(place, w, dY, Z):
    rows, tokens, k = Z.shape[0], *place.shape
    there = (place >= 0) & (place < rows)
    at = place.long()[there]
    token = torch.arange(tokens, device="cuda").unsqueeze(1).expand(tokens, k)[there]
    dZ = torch.zeros(Z.shape, dtype=torch.float64, device="cuda")
    dZ[at] = w.double()[there].unsqueeze(1) * dY.double()[token]
    dw = torch.zeros(tokens, k, dtype=torch.float64, device="cuda")
    dw[there] = (dY.double()[token] * Z.double()[at]).sum(1)
    return dZ, dw


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("tokens,k,rows,cols,named,pad", [
    (1, 1, 1, 1, 0, 0), (1, 1, 1, 9, 1, 0), (3, 2, 4, 100, 3, 3), (3, 2, 100, 100, 6, 0), (8, 2, 16, 1000, 12, 5),
    (100, 8, 800, 260, 700, 0), (100, 8, 5000, 64, 800, 4), (300, 4, 1200, 33, 0, 0), (2100, 4, 8400, 40, 8390, 0),
    (4097, 2, 4100, 16, 4000, 0), (9000, 1, 9000, 24, 9000, 0)])
def test_rows_without_a_name_get_zeros(tokens, k, rows, cols, named, pad, kind):
    print(f"[gpu] combine backward {kind} {tokens}x{k} into {rows}x{cols}, {named} named", flush=True)
    place, w, dY, Z, room = case(tokens, k, rows, cols, kind, named, tokens + rows, pad)
    dw = torch.full((tokens, k), float("nan"), device="cuda")
    backward(dY, Z, place, w, room[:, :cols], dw)
    want, slope = expected(place, w, dY, Z)
    assert torch.equal(room[:, :cols].double(), want)
    assert torch.equal(dw.double(), slope)  # whole numbers below 2^24
    assert bool(room[:, cols:].isnan().all())
    got = sg.route_combine_backward(dY, Z, place, w)
    assert torch.equal(got[0].double(), want) and torch.equal(got[1].double(), slope)


def test_more_rows_than_the_gradients_own_workgroups_have_bits_for():
    rows, cols = 128 * 131072 + 5, 3
    print(f"[gpu] combine backward into {rows} rows", flush=True)
    Z = torch.ones(rows, cols, device="cuda")
    place = torch.tensor([[rows - 1, 0], [-1, 1 << 23]], dtype=torch.int32, device="cuda")
    w, dY = torch.tensor([[2.0, 3.0], [4.0, 5.0]], device="cuda"), torch.ones(2, cols, device="cuda")
    dZ = torch.full((rows, cols), float("nan"), device="cuda")
    dw = torch.empty(2, 2, device="cuda")
    backward(dY, Z, place, w, dZ, dw)
    assert dZ[[rows - 1, 0, 1 << 23], 0].tolist() == [2.0, 3.0, 5.0] and float(dZ.double().sum()) == 10.0 * cols
    assert dw.tolist() == [[3.0, 3.0], [0.0, 3.0]]


def test_as_many_rows_as_one_of_those_workgroups_can_have():
    rows, tokens, k = 128 * 131072, 1 << 20, 8
    print(f"[gpu] combine backward, {tokens} tokens into {rows} rows", flush=True)
    place = (torch.arange(tokens * k, device="cuda", dtype=torch.int64) * 2 + 1).int().view(tokens, k).flip(0).contiguous()
    dY, w = torch.ones(tokens, 1, device="cuda"), torch.full((tokens, k), 2.0, device="cuda")
    dZ = torch.full((rows, 1), float("nan"), device="cuda")
    backward(dY, dZ.new_ones(rows, 1), place, w, dZ, torch.empty(tokens, k, device="cuda"))
    assert bool((dZ[1::2] == 2).all()) and bool((dZ[::2] == 0).all())


def test_nothing_named_at_all():
    Z = torch.ones(5, 7, device="cuda")
    for tokens, k in ((0, 2), (3, 0)):
        dZ, dw = sg.route_combine_backward(torch.ones(tokens, 7, device="cuda"), Z,
                                           torch.empty(tokens, k, dtype=torch.int32, device="cuda"),
                                           torch.empty(tokens, k, device="cuda"))
        assert bool((dZ == 0).all()) and dw.shape == (tokens, k)


def test_captured_and_replayed():
    place, w, dY, Z, _ = case(500, 4, 2500, 130, "bf16", 1500, 1)
    sg.route_combine_backward(dY, Z, place, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sg.route_combine_backward(dY, Z, place, w)
    for i in range(4):
        place.copy_(case(500, 4, 2500, 130, "bf16", 1500, 2 + i)[0])
        got[0].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, expected(place, w, dY, Z)):
            assert torch.equal(a.double(), b)
