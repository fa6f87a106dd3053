"""The order of the experts' rows at the largest sizes."""
from __future__ import annotations

import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _gpu as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()


def test_plan_of_nearly_2_to_the_31_entries():
    """The last thousand entry counts that the call takes: their number of runs is rounded up past 32 bits."""
    tokens, k = 268435315, 8
    n = tokens * k
    assert 2 ** 31 - 2048 < n <= 2 ** 31 - 1025
    print(f"[gpu] plan of {n} entries", flush=True)
    ids = torch.ones(tokens, k, dtype=torch.int32, device="cuda")
    flat = ids.view(-1)
    flat[5], flat[n - 2], flat[n - 1] = 0, 0, 2
    offsets, rows, place = sg.route_plan(ids, 3)
    torch.cuda.synchronize()
    assert offsets.tolist() == [0, 2, n - 1, n]
    place = place.view(-1)
    step = 1 << 27
    for at in range(0, n, step):  # the first five move up by two places, entry 5 is first, the others move up by one
        entry = torch.arange(at, min(at + step, n), dtype=torch.int32, device="cuda")
        want = entry + 1
        if at == 0:
            want[:5] += 1
            want[5] = 0
        if at + step >= n:
            want[-2], want[-1] = 1, n - 1
        assert torch.equal(place[at:at + step], want)
        token = torch.div(torch.where(entry < 2, 0, entry - 1), k, rounding_mode="floor")
        if at == 0:
            token[0], token[1] = 5 // k, (n - 2) // k
            token[2:7] = torch.arange(5, device="cuda") // k
        if at + step >= n:
            token[-1] = (n - 1) // k
        assert torch.equal(rows[at:at + step], token)
        del entry, want, token
