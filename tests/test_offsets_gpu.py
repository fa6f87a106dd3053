"""Offsets of experts that fall or lie outside the rows: what each row's expert is then, and that nothing around C is touched."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _fp8 as R
from tests import _gpu as G
from tests import test_experts16_gpu as E

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()


def taken(off, rows):
    """The ascending offsets that these count as, of the rows of C."""
    return np.maximum.accumulate(np.concatenate([[0], np.clip(off[1:], 0, rows)])).astype(int).tolist()


def alone(off, rows):
    """[begin, end) of each expert by itself, as its rows are summed."""
    off = [0, *np.clip(off[1:], 0, rows).tolist()]
    return [(b, max(b, e)) for b, e in zip(off, off[1:])]


def many(experts, rows, seed):
    """Offsets that mostly ascend, some of which fall below many others or leave the rows."""
    r = np.random.default_rng(seed)
    off = np.sort(r.integers(0, rows + 1, experts + 1))
    at = r.choice(experts + 1, experts // 4, replace=False)
    off[at] = r.integers(-rows, 2 * rows, at.size)
    return off.tolist()


BAD = [[5, -3, 500, 100, 90], [0, 2 ** 31 - 1, -2 ** 31, 7, 200], [0, 199, 0, 199, 0], [300, 200, 100, 50, 0], [0, 0, 0, 0, -1], [7, 10, 20, 30, 40],
       many(63, 200, 1), many(64, 200, 2), many(65, 200, 3), many(150, 200, 4), list(range(0, 200, 3))[::-1]]


def inside(shape, kind, pad=5):
    """A view that a buffer of NaN surrounds, and what checks that it still does."""
    room = torch.full((*shape[:-2], shape[-2] + 4, shape[-1] + pad), float("nan"), dtype=kind, device="cuda")
    C = room[..., 2:-2, :shape[-1]]

    def check():
        torch.cuda.synchronize()
        assert bool(room[..., :2, :].isnan().all()) and bool(room[..., -2:, :].isnan().all()) and bool(room[..., shape[-1]:].isnan().all())
        assert not bool(C.isnan().any())  # every element was written

    return C, check


@pytest.mark.parametrize("form", ["forward", "dgrad"])
@pytest.mark.parametrize("N,K", [(72, 64), (71, 65), (304, 328), (33, 7)])
@pytest.mark.parametrize("which", range(len(BAD)))
def test_rows_of_16_bit_products(form, N, K, which):
    off, rows = BAD[which], 200
    n = len(off) - 1
    x, w = E.matrix((rows, K if form == "forward" else N), 1, "bf16"), E.matrix((n, N, K), 2, "bf16")
    print(f"[gpu] {form} {N}x{K} offsets {which}: {E.name_of(form, rows, N, K, n, x, w)}", flush=True)
    want, size = E.expected(form, x, w, taken(off, rows))
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    for kind in (torch.float32, torch.bfloat16):
        C, check = inside(want.shape, kind)
        E.run(form, x, w, offsets, C=C)
        check()
        E.check(C, want, size, K if form == "forward" else N, "fp32" if kind == torch.float32 else "bf16")


@pytest.mark.parametrize("form", ["forward", "dgrad"])
@pytest.mark.parametrize("off", [[0, 3000, 100, 7900, 5000, 7900], [0, 9000, 0, 9000, 0, 8000], [50, -7, 6144, 6144, 3, 3]])
def test_rows_of_large_tiles(form, off):
    """Whole numbers, every element: tiles of 256 and 192 rows and their pieces."""
    rows, wide, inner, n = 8000, 2000, 72, len(off) - 1
    N, K = (wide, inner) if form == "forward" else (inner, wide)
    x, w = E.matrix((rows, inner), 1, "bf16", 8, whole=True), E.matrix((n, N, K), 2, "bf16", 8, whole=True)
    assert E.name_of(form, rows, N, K, n, x, w) == "tile_256x256"
    want, _ = E.expected(form, x, w, taken(off, rows))
    C, check = inside(want.shape, torch.float32)
    E.run(form, x, w, torch.tensor(off, dtype=torch.int32, device="cuda"), C=C)
    check()
    np.testing.assert_array_equal(E.plain(C), want)


@pytest.mark.parametrize("N,K", [(72, 64), (71, 65)])
@pytest.mark.parametrize("which", range(len(BAD)))
def test_sums_of_16_bit_products(N, K, which):
    off, rows = BAD[which], 200
    dy, x = E.matrix((rows, N), 1, "bf16"), E.matrix((rows, K), 2, "bf16")
    print(f"[gpu] wgrad {N}x{K} offsets {which}", flush=True)
    C, check = inside((len(off) - 1, N, K), torch.float32)
    sg.gemm_experts_wgrad(dy, x, torch.tensor(off, dtype=torch.int32, device="cuda"), C)
    check()
    for e, (s, t) in enumerate(alone(off, rows)):
        p, q = E.plain(dy)[s:t], E.plain(x)[s:t]
        E.check(C[e], p.T @ q, np.abs(p).T @ np.abs(q), t - s, "fp32")


@pytest.mark.parametrize("K,pad", [(256, 0), (300, 4), (256, 3)])
@pytest.mark.parametrize("which", range(len(BAD)))
def test_rows_of_8_bit_products(K, pad, which):
    off, rows, N = BAD[which], 200, 72
    n = len(off) - 1
    A, B = R.random_bytes(rows, K, 1, pad), R.random_bytes(n * N, K, 2, pad).unflatten(0, (n, N))
    sa, sb = R.random_scales(rows, -(-K // 128), 3), R.random_scales(n, -(-K // 128), 4, False).unsqueeze(1)
    print(f"[gpu] fp8 experts K {K} pad {pad} offsets {which}", flush=True)
    C, check = inside((rows, N), torch.float32)
    sg.gemm_fp8_experts(A, sa, B, sb, torch.tensor(off, dtype=torch.int32, device="cuda"), C)
    check()
    a, off = R.values(R.bytes_of(A), sa.cpu().numpy()), taken(off, rows)
    for e in range(n):
        b = R.values(R.bytes_of(B[e]), sb[e].cpu().numpy(), 128)
        s, t = off[e], off[e + 1]
        want, size = a[s:t] @ b.T, np.abs(a[s:t]) @ np.abs(b).T
        assert (np.abs(E.plain(C[s:t]) - want) <= R.product_bound(want, size, K, "fp32")).all()
    assert bool((C[off[-1]:] == 0).all())
