"""Products by expert of 16-bit operands on the GPU against plain 64-bit products."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _fp8 as R
from tests import _gpu as G

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()


def matrix(shape, seed, kind, pad=0, offset=0, whole=False, spread=1.0):
    """A GPU tensor whose rows are padded with NaN, its first element `offset` past the buffer's; after it more NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-3, 4, shape, generator=g).float() if whole else torch.randn(shape, generator=g) * spread
    rows, cols = int(np.prod(shape[:-1])), shape[-1]
    room = torch.full((offset + rows * (cols + pad) + 64,), float("nan"), dtype=TYPES[kind])
    room[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = x.to(TYPES[kind]).view(rows, cols)
    room = room.to("cuda")[offset:offset + rows * (cols + pad)]
    return room.view(*shape[:-1], cols + pad)[..., :cols]


def plain(x):
    return x.double().cpu().numpy()


def counts_to(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def bound(want, size, K, kind):
    """Exact products, K additions each off by a whole FP32 step at most (the matrix unit may cut), and the rounding to C."""
    rel, least = R.half_step(kind)
    inside = (K + 2) * 2.0 ** -23 * size
    return inside + rel * (np.abs(want) + inside) + least


def check(C, want, size, K, kind):
    off = np.abs(plain(C) - want)
    worst = off / bound(want, size, K, kind)
    assert not np.isnan(off).any() and (worst <= 1.0).all(), worst.max()


def expected(form, x, w, off):
    """(product, product of magnitudes) in 64 bits."""
    a, b = plain(x), plain(w)
    if form == "wgrad":
        parts = [(a[s:t], b[s:t]) for s, t in zip(off, off[1:])]
        return np.stack([p.T @ q for p, q in parts]), np.stack([np.abs(p).T @ np.abs(q) for p, q in parts])
    cols = b.shape[1] if form == "forward" else b.shape[2]
    out, size = np.zeros((a.shape[0], cols)), np.zeros((a.shape[0], cols))
    for e, (s, t) in enumerate(zip(off, off[1:])):
        m = b[e].T if form == "forward" else b[e]
        out[s:t], size[s:t] = a[s:t] @ m, np.abs(a[s:t]) @ np.abs(m)
    return out, size


def run(form, x, w, off, **how):
    call = {"forward": sg.gemm_experts, "dgrad": sg.gemm_experts_dgrad, "wgrad": sg.gemm_experts_wgrad}[form]
    C = call(x, w, off, **how)
    torch.cuda.synchronize()
    return C


def name_of(form, rows, N, K, E, x, w):
    number = {"forward": 0, "dgrad": 1, "wgrad": 2}[form]
    return sg.sgemm_mi355_experts_kernel_name(number, rows, N, K, E, x.data_ptr(), x.stride(0), w.data_ptr(), w.stride(-2),
                                              w.stride(0) if form != "wgrad" else 0)


COUNTS = [[1], [0, 3, 0], [5, 0, 0, 17, 1], [64, 65, 63], [130, 0, 127, 128, 300], [260, 255, 513], [1] * 70]
SIZES = [(1, 1), (8, 8), (16, 64), (40, 72), (33, 100), (130, 200), (256, 128), (264, 136), (300, 1000), (520, 264), (128, 1100)]


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("counts", COUNTS, ids=range(len(COUNTS)))
@pytest.mark.parametrize("N,K", SIZES)
def test_products(form, counts, N, K):
    kind = "bf16" if (N + K + len(counts)) % 2 else "fp16"
    E, spare = len(counts), 3 if N % 3 else 0
    off, rows = counts_to(counts), sum(counts) + spare
    for pad, offset in ((0, 0), (8, 8), (3, 1)):
        x = matrix((rows, K if form != "dgrad" else N), 1, kind, pad, offset)
        w = matrix((E, N, K), 2, kind, pad, offset, spread=K ** -0.5) if form != "wgrad" else matrix((rows, N), 2, kind, pad, offset)
        a, b = (w, x) if form == "wgrad" else (x, w)
        name = name_of(form, rows, N, K, E, a, b)
        print(f"[gpu] {form} {kind} {counts} {N}x{K} pad {pad} offset {offset}: {name}", flush=True)
        aligned = offset % 8 == 0 and x.stride(0) % 8 == 0 and w.stride(-2) % 8 == 0
        whole = {"forward": K >= 8, "dgrad": K % 8 == 0 and N >= 8, "wgrad": N % 8 == 0 and K % 8 == 0}[form]
        if not aligned or not whole:
            assert name.startswith(("staged", "rows") if form == "forward" and K >= 8 else "staged")
        else:
            assert not name.startswith("staged")
        inner = {"forward": K, "dgrad": N, "wgrad": max(counts)}[form]
        want, size = expected(form, a, b, off.tolist())
        for c_type in (torch.float32, TYPES[kind]):
            C = run(form, a, b, off, dtype=c_type)
            assert C.dtype == c_type
            check(C, want, size, inner, "fp32" if c_type == torch.float32 else kind)
            if spare and form != "wgrad":
                assert bool((C[rows - spare:] == 0).all())


LARGE = [("forward", [300, 0, 517, 256, 1000, 3], 1030, 520), ("forward", [700, 900, 1], 2056, 72), ("dgrad", [300, 0, 517, 256, 1000], 520, 1032),
         ("dgrad", [700, 900, 1], 200, 2056), ("wgrad", [300, 0, 517, 256, 1000], 1032, 520), ("wgrad", [77, 1, 2000], 2048, 1024),
         ("forward", [20] * 9, 300, 456), ("forward", [40] * 9, 72, 200), ("forward", [9000], 264, 256), ("wgrad", [5000, 4000], 256, 264)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("form,counts,N,K", LARGE)
def test_larger_products_of_whole_numbers_are_exact(form, counts, N, K, kind):
    """Sums below 2^24 are exact in FP32 in any order: every element of every kernel's tile, bit for bit."""
    E, off, rows = len(counts), counts_to(counts), sum(counts)
    x = matrix((rows, K if form != "dgrad" else N), 1, kind, 8, 8, whole=True)
    w = matrix((E, N, K), 2, kind, 0, 0, whole=True) if form != "wgrad" else matrix((rows, N), 2, kind, 0, 0, whole=True)
    a, b = (w, x) if form == "wgrad" else (x, w)
    print(f"[gpu] {form} {kind} {counts} {N}x{K}: {name_of(form, rows, N, K, E, a, b)}", flush=True)
    want, _ = expected(form, a, b, off.tolist())
    np.testing.assert_array_equal(plain(run(form, a, b, off, dtype=torch.float32)), want)
    C = run(form, a, b, off, dtype=TYPES[kind])
    assert torch.equal(C, torch.from_numpy(want).float().to(TYPES[kind]).to("cuda"))


ODD_ROWS = [([3, 9, 0, 16], 100, 333), ([3, 9, 0, 16], 100, 128), ([2, 1], 33, 64), ([5, 0, 2], 64, 65), ([1], 20, 1025), ([100, 90, 128, 1, 140], 301, 327), ([30, 40, 64, 1, 61], 1001, 1031)]


@pytest.mark.parametrize("counts,N,K", ODD_ROWS)
def test_few_rows_of_any_alignment(counts, N, K):
    off, rows = counts_to(counts), sum(counts)
    for pad, offset in ((0, 0), (1, 1), (2, 3)):
        x, w = matrix((rows, K), 1, "bf16", pad, offset), matrix((len(counts), N, K), 2, "bf16", pad, offset)
        assert name_of("forward", rows, N, K, len(counts), x, w).startswith("rows" if offset or K > 64 else "tile")
        want, size = expected("forward", x, w, off.tolist())
        check(run("forward", x, w, off), want, size, K, "bf16")


KERNELS = {  # calls whose kernel is known
    ("forward", "rows_16"): ([3, 9, 0, 16], 100, 328), ("forward", "rows_32"): ([100, 90, 128, 1, 140], 300, 328),
    ("forward", "rows_64"): ([30, 40, 64, 1, 61], 1000, 1032), ("forward", "tile_128x128"): ([250, 300, 280, 1, 270], 600, 72),
    ("forward", "tile_256x256"): ([2000, 1000, 1999], 4000, 136), ("dgrad", "tile_128x128"): ([100, 90, 128, 1, 140], 328, 304),
    ("dgrad", "tile_256x256"): ([2000, 1000, 1999], 136, 4000), ("wgrad", "tile_128x128"): ([100, 90, 128, 1, 140], 328, 304),
    ("wgrad", "tile_256x256"): ([70, 1, 200, 64], 2000, 2008), ("forward", "staged_128x128"): ([250, 300, 280, 1, 270], 601, 73),
    ("dgrad", "staged_128x128"): ([100, 90, 128, 1, 140], 301, 333), ("wgrad", "staged_128x128"): ([100, 90, 128, 1, 140], 301, 333)}


@pytest.mark.parametrize("form,name", list(KERNELS), ids=lambda v: v)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_every_kernel_keeps_to_its_matrices(form, name, kind):
    """Each kernel by name: values, NaN around the operands and in rows of other experts, and what surrounds C."""
    counts, N, K = KERNELS[form, name]
    E, off, rows = len(counts), counts_to(counts), sum(counts)
    pad = (-K % 8 + 8) if "staged" not in name else 0
    x = matrix((rows + 4, K), 1, kind, pad if form != "dgrad" else 8)
    dy = matrix((rows + 4, N), 3, kind, -N % 8 + 8 if "staged" not in name else 0)
    w = matrix((E, N, K), 2, kind, pad)
    a, b = {"forward": (x, w), "dgrad": (dy, w), "wgrad": (dy, x)}[form]
    assert name_of(form, rows + 4, N, K, E, a, b) == name
    a[rows:] = float("nan")  # rows that no expert has
    if form == "wgrad":
        b[rows:] = float("nan")
    inner = {"forward": K, "dgrad": N, "wgrad": max(counts)}[form]
    want, size = expected(form, a, b, off.tolist())
    shape = {"forward": (rows + 4, N), "dgrad": (rows + 4, K), "wgrad": (E, N, K)}[form]
    for c_type in (torch.float32, TYPES[kind]):
        room = torch.full((*shape[:-1], shape[-1] + 5), float("nan"), dtype=c_type, device="cuda")
        C = room[..., :shape[-1]]
        assert run(form, a, b, off, C=C) is C
        check(C, want, size, inner, "fp32" if c_type == torch.float32 else kind)
        assert bool(room[..., shape[-1]:].isnan().all())
        again = run(form, a, b, off, dtype=c_type)
        assert torch.equal(again, C)
        if form == "wgrad":
            C.fill_(0.5)
            run(form, a, b, off, C=C, beta=-2.0)
            check(C, want - 1.0, size + 1.0, inner + 1, "fp32" if c_type == torch.float32 else kind)
    # a NaN and an infinity in one expert's operands stay with that expert
    bad = max(range(E), key=lambda e: counts[e])
    at = int(off[bad])
    if form == "wgrad":
        a[at, 1] = float("nan")
        C = run(form, a, b, off)
        assert bool(C[bad, 1].isnan().all()) and int(C.isnan().sum()) == K
    else:
        b[bad, 0] = float("inf")
        C = run(form, a, b, off).float()
        odd = ~C.isfinite()
        assert not bool(odd[:at].any()) and not bool(odd[int(off[bad + 1]):].any())
        assert bool(odd[at:int(off[bad + 1]), 0].any())
        if form == "forward":
            assert not bool(odd[:, 1:].any())


@pytest.mark.parametrize("form", ["forward", "dgrad", "wgrad"])
def test_bad_offsets_stay_inside(form):
    """Offsets that fall, or lie outside the rows: limited, so nothing outside the matrices is touched."""
    for off in ([5, -3, 500, 100, 90], [0, 2 ** 31 - 1, -2 ** 31, 7, 200], [0, 199, 0, 199, 0]):
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        for N, K in ((72, 64), (71, 65)):
            x, dy, w = matrix((200, K), 1, "bf16"), matrix((200, N), 2, "bf16"), matrix((4, N, K), 3, "bf16")
            a, b = {"forward": (x, w), "dgrad": (dy, w), "wgrad": (dy, x)}[form]
            assert bool(run(form, a, b, offsets).isfinite().all())


def test_empty_products():
    off = counts_to([0, 0])
    x, w = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), torch.ones(2, 32, 64, device="cuda", dtype=torch.bfloat16)
    assert sg.gemm_experts(x, w, off).shape == (0, 32) and sg.gemm_experts_dgrad(x[:, :32], w, off).shape == (0, 64)
    dw = sg.gemm_experts_wgrad(x[:, :32], x, off)
    assert dw.shape == (2, 32, 64) and bool((dw == 0).all())
    dw.fill_(3.0)
    assert bool((sg.gemm_experts_wgrad(x[:, :32], x, off, dw, beta=0.5) == 1.5).all())
    y = torch.ones(5, 64, device="cuda", dtype=torch.bfloat16)
    assert bool((sg.gemm_experts(y, w, off) == 0).all())  # no expert has these rows


def test_gradients_against_the_products():
    """The inner products <dy, y> = <dx, x> = <dW, W>: y is linear in either."""
    counts = [100, 0, 37, 290]
    off, rows = counts_to(counts), sum(counts)
    x, dy, w = matrix((rows, 136), 1, "bf16"), matrix((rows, 264), 2, "bf16"), matrix((4, 264, 136), 3, "bf16")
    y, dx, dw = sg.gemm_experts(x, w, off, dtype=torch.float32), sg.gemm_experts_dgrad(dy, w, off, dtype=torch.float32), \
        sg.gemm_experts_wgrad(dy, x, off)
    one, two, three = (float((plain(p) * plain(q)).sum()) for p, q in ((dy, y), (dx, x), (dw, w)))
    # each product is off by 300 steps of FP32 of the sum of magnitudes at most; that sum is over all products
    total = sum(float((np.abs(plain(dy[s:t])) @ np.abs(plain(w[e])) * np.abs(plain(x[s:t]))).sum())
                for e, (s, t) in enumerate(zip(off.tolist(), off.tolist()[1:])))
    assert abs(one - two) <= 600 * 2.0 ** -23 * total and abs(one - three) <= 600 * 2.0 ** -23 * total


def test_weights_that_experts_share():
    """A stride of 0 between experts: one matrix for all of them, read where it is."""
    counts = [70, 0, 200, 33]
    off, rows = counts_to(counts), sum(counts)
    for N, K in ((136, 264), (135, 263)):
        w = matrix((1, N, K), 1, "bf16")
        x, dy = matrix((rows, K), 2, "bf16"), matrix((rows, N), 3, "bf16")
        want, size = expected("forward", x, w.expand(4, N, K), off.tolist())
        check(run("forward", x, w.expand(4, N, K), off), want, size, K, "bf16")
        want, size = expected("dgrad", dy, w.expand(4, N, K), off.tolist())
        check(run("dgrad", dy, w.expand(4, N, K), off), want, size, N, "bf16")


@pytest.mark.parametrize("form", ["forward", "dgrad"])
@pytest.mark.parametrize("counts,left", [([3000, 100, 4900], 8), ([5, 3000, 0, 5200], 16), ([2048, 6144], 0), ([3000, 100, 7700], 96), ([2560, 2560, 7168], 128),
                                         ([300, 3000, 100, 14100], 56), ([3000, 100, 10000], 168)])
@pytest.mark.parametrize("wide", [2048, 2000, 1904])
def test_the_last_round_in_pieces(form, counts, left, wide):
    """Tiles of 256 x 256 past whole rounds of 256, in four pieces, in two or whole: every element, bit for bit."""
    rows, spare, off, inner = sum(counts), 300, counts_to(counts), 72
    assert sum(-(-c // 256) for c in counts) * 8 % 256 == left
    N, K = (wide, inner) if form == "forward" else (inner, wide)
    for extra in (0, spare):
        x, w = matrix((rows + extra, inner), 1, "bf16", 8, whole=True), matrix((len(counts), N, K), 2, "bf16", 8, whole=True)
        assert name_of(form, rows + extra, N, K, len(counts), x, w) == "tile_256x256"
        x[rows:] = float("nan")
        want = torch.zeros(rows + extra, wide, dtype=torch.float64, device="cuda")
        for e, (s, t) in enumerate(zip(off.tolist(), off.tolist()[1:])):
            want[s:t] = x[s:t].double() @ (w[e].double().t().contiguous() if form == "forward" else w[e].double())
        room = torch.full((rows + extra, wide + 8), float("nan"), device="cuda")
        run(form, x, w, off, C=room[:, :wide])
        assert torch.equal(room[:, :wide].double(), want) and bool(room[:, wide:].isnan().all())
        assert torch.equal(run(form, x, w, off), want.float().bfloat16())


@pytest.mark.parametrize("form", ["forward", "dgrad"])
@pytest.mark.parametrize("counts,wide", [([1100] * 8, 1024), ([300] * 24, 2048), ([300, 0, 301] * 12, 2000), ([1, 500] * 13 + [190] * 4, 1904), ([6144], 2048)])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_tiles_of_fewer_rows(form, counts, wide, kind):
    """Experts that fill rounds of 192-row tiles better, whole and in halves, and some that do not: every element, bit for bit."""
    rows, off, inner = sum(counts), counts_to(counts), 520
    N, K = (wide, inner) if form == "forward" else (inner, wide)
    for spare in (0, 200):
        x, w = matrix((rows + spare, inner), 1, kind, 8, whole=True), matrix((len(counts), N, K), 2, kind, 8, whole=True)
        assert name_of(form, rows + spare, N, K, len(counts), x, w) == "tile_256x256"
        x[rows:] = float("nan")
        want = torch.zeros(rows + spare, wide, dtype=torch.float64, device="cuda")
        for e, (s, t) in enumerate(zip(off.tolist(), off.tolist()[1:])):
            want[s:t] = x[s:t].double() @ (w[e].double().t().contiguous() if form == "forward" else w[e].double())
        room = torch.full((rows + spare, wide + 8), float("nan"), device="cuda")
        run(form, x, w, off, C=room[:, :wide])
        assert torch.equal(room[:, :wide].double(), want) and bool(room[:, wide:].isnan().all())
        assert torch.equal(run(form, x, w, off), want.float().to(TYPES[kind]))
