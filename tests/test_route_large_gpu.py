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


@pytest.mark.parametrize("tokens,k,experts", [
    (16384, 8, 1024), (17001, 8, 1023), (65536, 8, 256), (70001, 8, 255), (262144, 8, 64), (600011, 8, 7), (200003, 1, 1000),
    (1 << 20, 8, 256)])
def test_plan_of_many_runs(tokens, k, experts):
    """Runs in groups, of one run and of more, the last run and the last group shorter; some ids outside the experts."""
    n = tokens * k
    print(f"[gpu] plan {tokens} {k} {experts}", flush=True)
    size = sg.sgemm_mi355_route_plan_workspace_size(tokens, k, experts)
    assert size > 4 * -(-n // 2048) * (experts + 1)  # room for groups: they are taken
    g = torch.Generator(device="cuda").manual_seed(n)
    for ids in (torch.randint(0, experts, (tokens, k), generator=g, device="cuda", dtype=torch.int32),
                torch.randint(-3, experts + 5, (tokens, k), generator=g, device="cuda", dtype=torch.int32),
                torch.full((tokens, k), experts - 1, dtype=torch.int32, device="cuda")):
        offsets, rows, place = sg.route_plan(ids, experts)
        flat = torch.where((ids < 0) | (ids >= experts), experts, ids).flatten().long()
        counts = torch.zeros(experts + 1, dtype=torch.long, device="cuda").index_add_(0, flat, torch.ones_like(flat))
        assert torch.equal(offsets.long(), torch.cat([counts.new_zeros(1), counts.cumsum(0)[:-1]]))
        order = (flat * n + torch.arange(n, device="cuda")).sort().indices  # by expert, then by place in ids
        assert torch.equal(rows.long(), order // k)
        assert torch.equal(place.flatten()[order].long(), torch.arange(n, device="cuda"))


def test_plan_of_many_runs_captured_and_replayed():
    ids = torch.zeros(70001, 8, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sg.route_plan(ids, 256)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sg.route_plan(ids, 256)
    for i in range(4):
        ids.copy_(torch.randint(0, 256, (70001, 8), generator=torch.Generator().manual_seed(i), dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, sg.route_plan(ids, 256)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("tokens,experts", [(262144, 64), (70001, 256)])
def test_plan_of_one_experts_many_runs_repeats(tokens, experts):
    """All additions to one counter, which take longest: every run sees those of the runs before it, each time."""
    ids = torch.full((tokens, 8), experts - 1, dtype=torch.int32, device="cuda")
    want = torch.arange(tokens * 8, dtype=torch.int32, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        _, rows, place = sg.route_plan(ids, experts)
        wrong += (place.flatten() != want).sum() + (rows != want // 8).sum()
    assert int(wrong) == 0
