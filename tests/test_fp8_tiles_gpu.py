"""Every FP8 product kernel by name, in every form and type that can take it, against plain 64-bit definitions: partial
blocks, rows and columns, odd and even block counts, and C with guards beside its rows."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _fp8 as R
from tests import _gpu as G

pytestmark = pytest.mark.gpu

CODE = {"fp32": sg.F32, "bf16": sg.BF16, "fp16": sg.F16}


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()


def kernel_of(form, kind, M, N, K, experts, A, B):
    return sg.sgemm_mi355_fp8_kernel_name(form, CODE[kind], M, N, K, experts, A.data_ptr(), A.stride(0), B.data_ptr(),
                                          B.stride(-2), B.stride(0) if B.dim() == 3 else 0)


def room_for(shape, kind, seed=None, pad=5):
    """(C, the rest of its rows): C of `shape` with padded rows, all NaN or normal numbers; the rest is NaN."""
    room = torch.full((*shape[:-1], shape[-1] + pad), float("nan"), dtype=R.TYPES[kind], device="cuda")
    C, rest = room[..., :shape[-1]], room[..., shape[-1]:]
    if seed is not None:
        C.copy_(torch.randn(*shape, generator=torch.Generator().manual_seed(seed)))
    return C, rest


def near(C, a, b, K, kind, init=None):
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    if init is not None:
        want, size = want + init, size + np.abs(init)
    off = np.abs(C.double().cpu().numpy() - want)
    worst = (off / R.product_bound(want, size, K, kind)).max() if off.size else 0.0
    assert worst <= 1.0, f"{worst} times the bound"


def rounded(a, b, kind):
    """The product, exact in FP32, rounded once to the type."""
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    assert size.size == 0 or size.max() * 64 < 2 ** 24  # scales are multiples of 2^-6
    return torch.from_numpy(want).to(R.TYPES[kind])


DENSE = [  # kernel, kind, M, N, K
    ("tile_128x128_fp8", "bf16", 200, 8192, 512), ("tile_128x128_fp8", "fp16", 1100, 2050, 400),
    ("tile_128x128_fp8", "bf16", 1300, 2100, 260), ("tile_128x128_fp8", "fp16", 700, 3001, 640),
    ("tile_128x128_fp8", "bf16", 450, 1030, 2000), ("tile_128x128_fp8", "fp16", 1281, 2049, 100),
    ("tile_256x256_fp8", "bf16", 2100, 2200, 400), ("tile_256x256_fp8", "fp16", 3000, 4100, 400),
    ("tile_256x256_fp8", "bf16", 2305, 4097, 260), ("tile_256x256_fp8", "fp16", 2100, 2200, 100),
    ("tile_256x256_fp8", "bf16", 2304, 2560, 384), ("tile_256x256_fp8", "fp16", 2177, 2433, 129),
    ("tile_128x128_bf16", "fp32", 1300, 2100, 260), ("tile_128x128_bf16", "fp32", 700, 3001, 640),
    ("tile_128x128_bf16", "fp32", 257, 8200, 900), ("tile_192x128_bf16", "fp32", 2100, 2200, 400),
    ("rows_64_bf16", "fp32", 450, 500, 2000), ("rows_64_bf16", "fp32", 200, 1020, 1000),
    ("rows_64_bf16", "bf16", 505, 500, 3990), ("rows_32_bf16", "fp16", 300, 300, 8100),
    ("staged_128x128_bf16", "bf16", 300, 260, 10), ("staged_128x128_bf16", "fp16", 129, 257, 15)]


@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("kernel,kind,M,N,K", DENSE)
def test_dense(kernel, kind, M, N, K, tall):
    print(f"[gpu] {kernel} {kind} {M}x{N}x{K} tall {tall}", flush=True)
    blocks = -(-K // 128)
    for whole in (False, True):
        A, B = R.random_bytes(M, K, 1, -K % 16, whole=whole), R.random_bytes(N, K, 2, -K % 16, whole=whole)
        assert kernel_of(sg.FP8_DENSE, kind, M, N, K, 0, A, B) == kernel
        sa = R.random_scales(M, blocks, 3, powers=whole)
        sb = R.random_scales(-(-N // tall), blocks, 4, tall == 1, powers=whole)
        if kind == "fp16" and not whole:
            sa = sa * 1e-3
        a, b = R.values(R.bytes_of(A), sa.cpu().numpy()), R.values(R.bytes_of(B), sb.cpu().numpy(), tall)
        C, rest = room_for((M, N), kind)
        sg.gemm_fp8(A, sa, B, sb, C)
        if whole:
            if K <= 1024:
                assert torch.equal(C.cpu(), rounded(a, b, kind))
        else:
            near(C, a, b, K, kind)
            first = C.clone()
            sg.gemm_fp8(A, sa, B, sb, C)
            assert torch.equal(C, first)
            C.copy_(torch.randn(M, N, generator=torch.Generator().manual_seed(5)))
            init = -0.5 * C.double().cpu().numpy()
            sg.gemm_fp8(A, sa, B, sb, C, beta=-0.5)
            near(C, a, b, K, kind, init)
        assert bool(rest.isnan().all())


@pytest.mark.parametrize("kernel,kind,M,N,K", [DENSE[1], DENSE[6], DENSE[12], DENSE[15], DENSE[17], DENSE[18]])
def test_nan_stays_in_its_row_or_column(kernel, kind, M, N, K):
    print(f"[gpu] NaN in {kernel} {kind}", flush=True)
    A, B = R.random_bytes(M, K, 1, -K % 16), R.random_bytes(N, K, 2, -K % 16)
    assert kernel_of(sg.FP8_DENSE, kind, M, N, K, 0, A, B) == kernel
    sa, sb = R.random_scales(M, -(-K // 128), 3) * 1e-3, R.random_scales(N, -(-K // 128), 4)
    A.view(torch.uint8)[M - 1, K - 1] = 0x7F
    sb[9, 0] = float("nan")
    nan = sg.gemm_fp8(A, sa, B, sb, dtype=R.TYPES[kind]).isnan()
    assert bool(nan[M - 1].all()) and bool(nan[:, 9].all()) and int(nan.sum()) == M + N - 1


def offsets_of(rows, experts, left, seed):
    """Offsets with an expert of one row and an empty one where there is room, and `left` rows that no expert has."""
    cut = torch.randint(0, rows - left + 1, (experts - 1,), generator=torch.Generator().manual_seed(seed)).sort().values
    off = [0, *cut.tolist(), rows - left]
    if experts > 2:
        off[2] = off[1] + 1
        off[3] = max(off[3], off[2])
        off[-2] = off[-1]
    return sorted(off)


EXPERTS = [  # kernel, kind, rows, N, K, experts
    ("tile_256x256_fp8", "bf16", 5000, 2048, 400, 8), ("tile_256x256_fp8", "fp16", 5000, 1030, 400, 3),
    ("tile_256x256_fp8", "bf16", 5000, 2050, 1000, 4), ("tile_128x128_fp8", "fp16", 1500, 1000, 400, 4),
    ("tile_128x128_fp8", "bf16", 900, 2050, 260, 3), ("tile_128x128_fp8", "bf16", 2000, 500, 384, 5),
    ("tile_128x128_bf16", "fp32", 1500, 1000, 400, 4), ("tile_128x128_bf16", "fp32", 5000, 1030, 512, 3),
    ("rows_64_bf16", "fp16", 600, 1030, 600, 2), ("rows_64_bf16", "fp32", 600, 1030, 600, 2)]


@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("kernel,kind,rows,N,K,E", EXPERTS)
def test_experts(kernel, kind, rows, N, K, E, tall):
    print(f"[gpu] experts {kernel} {kind} {rows} rows, N {N} K {K} of {E}, tall {tall}", flush=True)
    off, blocks = offsets_of(rows, E, 37, rows + E), -(-K // 128)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    for whole in (False, True):
        A = R.random_bytes(rows, K, 1, -K % 16, whole=whole)
        B = R.random_bytes(E * N, K, 2, -K % 16, whole=whole).unflatten(0, (E, N))
        assert kernel_of(sg.FP8_EXPERTS, kind, rows, N, K, E, A, B) == kernel
        sa = R.random_scales(rows, blocks, 3, powers=whole)
        sb = R.random_scales(E * -(-N // tall), blocks, 4, False, powers=whole).unflatten(0, (E, -1))
        if kind == "fp16" and not whole:
            sa = sa * 1e-3
        C, rest = room_for((rows, N), kind)
        sg.gemm_fp8_experts(A, sa, B, sb, offsets, C)
        a = R.values(R.bytes_of(A), sa.cpu().numpy())
        for e in range(E):
            at, b = slice(off[e], off[e + 1]), R.values(R.bytes_of(B[e]), sb[e].cpu().numpy(), tall)
            if whole:
                assert torch.equal(C[at].cpu(), rounded(a[at], b, kind))
            else:
                near(C[at], a[at], b, K, kind)
        assert bool((C[off[-1]:] == 0).all()) and bool(rest.isnan().all())


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("off", [[0, 5, 5, 133, 300], [0, 0, 0, 0, 0], [0, 0, 257, 258, 290], [0, 300]])
@pytest.mark.parametrize("N,K,pad", [(100, 260, 12), (130, 512, 0), (100, 260, 3)])
def test_experts_of_few_rows_in_each_type(off, N, K, pad, kind):
    E, rows = len(off) - 1, 300
    print(f"[gpu] experts {off} {kind} N {N} K {K} pad {pad}", flush=True)
    A, B = R.random_bytes(rows, K, 1, pad), R.random_bytes(E * N, K, 2, pad).unflatten(0, (E, N))
    sa = R.random_scales(rows, -(-K // 128), 3) * (1e-3 if kind == "fp16" else 1.0)
    sb = R.random_scales(E * N, -(-K // 128), 4, False).unflatten(0, (E, N))
    C, rest = room_for((rows, N), kind)
    sg.gemm_fp8_experts(A, sa, B, sb, torch.tensor(off, dtype=torch.int32, device="cuda"), C)
    a = R.values(R.bytes_of(A), sa.cpu().numpy())
    for e in range(E):
        near(C[off[e]:off[e + 1]], a[off[e]:off[e + 1]], R.values(R.bytes_of(B[e]), sb[e].cpu().numpy()), K, kind)
    assert bool((C[off[-1]:] == 0).all()) and bool(rest.isnan().all())


WGRAD = [  # kernel, kind, M, N, rows, experts
    ("tile_256x256_fp8", "bf16", 1024, 1024, 4000, 32), ("tile_256x256_fp8", "fp16", 1100, 1030, 3000, 9),
    ("tile_256x256_fp8", "bf16", 257, 513, 1000, 70), ("tile_128x128_fp8", "bf16", 520, 260, 3000, 3),
    ("tile_128x128_fp8", "fp16", 300, 500, 900, 4), ("tile_128x128_bf16", "fp32", 520, 260, 3000, 3),
    ("tile_128x128_bf16", "fp32", 257, 513, 1000, 70)]


def small_numbers(Q):
    """Q with +-1 or +-2 for every number but zero."""
    q = Q.view(torch.uint8)
    return torch.where((q & 0x7F) == 0, q, (q & 0x80) | (0x38 + (q & 8))).view(Q.dtype)


@pytest.mark.parametrize("beta", [0.0, 0.5])
@pytest.mark.parametrize("kernel,kind,M,N,rows,E", WGRAD)
def test_weight_gradient(kernel, kind, M, N, rows, E, beta):
    print(f"[gpu] wgrad {kernel} {kind} {M}x{N} {rows} rows of {E}, beta {beta}", flush=True)
    off = offsets_of(rows, E, 11, rows + E)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    for whole in (False, True) if beta == 0.0 else (False,):
        g = torch.Generator().manual_seed(M)
        Y, X = (torch.randn(rows, n, generator=g) * 0.1 for n in (M, N))
        (A, sa), (B, sb) = (sg.quantize_fp8_cols(x.to("cuda"), offsets=offsets) for x in (Y, X))
        if whole:  # the same places hold -2, -1, 1 and 2, under scales that are powers of 2
            A, B = (small_numbers(q) for q in (A, B))
            sa, sb = R.random_scales(M, sa.shape[1], 3, powers=True), R.random_scales(N, sb.shape[1], 4, powers=True)
        assert A.stride(0) % 16 == 0
        assert kernel_of(sg.FP8_WGRAD, kind, M, N, rows, E, A, B) == kernel
        C, rest = room_for((E, M, N), kind, seed=5 if beta else None)
        init = beta * C.double().cpu().numpy() if beta else None
        sg.gemm_fp8_experts_wgrad(A, sa, B, sb, offsets, C, beta=beta)
        a, b = R.values(R.bytes_of(A), sa.cpu().numpy()), R.values(R.bytes_of(B), sb.cpu().numpy())
        for e in range(E):
            at = 128 * (off[e] // 128 + e)
            to = at + off[e + 1] - off[e]
            if whole:
                assert torch.equal(C[e].cpu(), rounded(a[:, at:to], b[:, at:to], kind))
            else:
                near(C[e], a[:, at:to], b[:, at:to], max(to - at, 1), kind, None if init is None else init[e])
        assert bool(rest.isnan().all())


def test_tiles_captured_and_replayed():
    """The tile kernels captured once and replayed on changed inputs, with eager work between, equal the eager calls."""
    offsets = torch.tensor([0, 1500, 1501, 2200, 2290], dtype=torch.int32, device="cuda")
    X = torch.randn(2300, 400, device="cuda")
    W, SW = sg.quantize_fp8(torch.randn(2304, 400, device="cuda"), blocks=True)

    def work():
        q, s = sg.quantize_fp8(X)
        t, u = sg.quantize_fp8_cols(X, offsets=offsets)
        return (sg.gemm_fp8(q, s, W, SW), sg.gemm_fp8(q, s, W, SW, dtype=torch.float32),
                sg.gemm_fp8_experts(q, s, W.expand(4, -1, -1), SW.expand(4, -1, -1), offsets),
                sg.gemm_fp8_experts_wgrad(t, u, t, u, offsets, dtype=torch.bfloat16))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for i in range(4):
        X.copy_(torch.randn(2300, 400, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(got, work()):
            assert torch.equal(g, w)


def cancelling(K, seed):
    """(a, b): whose products are 2^16, -2^16 and six of 4 in every eight, in random places; their sum is 3 K."""
    g = torch.Generator().manual_seed(seed)
    b = torch.full((K // 8, 8), 2.0)
    at = torch.rand(K // 8, 8, generator=g).argsort(-1)
    b.scatter_(1, at[:, :2], 256.0)
    a = b.clone().scatter_(1, at[:, :1], -256.0)
    return a.flatten(), b.flatten()


def stored(x):
    return x.to(torch.float8_e4m3fn).to("cuda")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K,asked", [
    (1, 100, 640, False), (8, 1000, 1040, False), (30, 700, 640, False), (64, 1100, 512, False), (450, 1030, 640, True),
    (1100, 2050, 400, True), (2304, 2560, 384, True)])
def test_sums_into_16_bits_are_fp32(kind, M, N, K, asked):
    """Products of 2^16 that cancel leave the small ones whole: partial sums are whole numbers below 2^24, which FP32
    holds in any order. Few rows keep them always, larger products where the caller asks."""
    print(f"[gpu] cancelling products {M}x{N}x{K} {kind}", flush=True)
    a, b = cancelling(K, 1)
    g = torch.Generator().manual_seed(2)
    sign = torch.randint(0, 2, (M, 1), generator=g) * 2.0 - 1.0
    A, B = stored(sign * a), stored(b.repeat(N, 1))
    sb = torch.exp2(torch.randint(-3, 4, (N, 1), generator=g).float())
    name = sg.sgemm_mi355_fp8_kernel_name(sg.FP8_DENSE, CODE[kind] | (sg.FP32_SUMS if asked else 0), M, N, K, 0,
                                          A.data_ptr(), K, B.data_ptr(), K)
    assert name.endswith("bf16")
    C = sg.gemm_fp8(A, torch.ones(M, -(-K // 128), device="cuda"), B, sb.to("cuda").expand(N, -(-K // 128)),
                    dtype=R.TYPES[kind], fp32_sums=asked)
    assert torch.equal(C.cpu(), (sign * sb.t() * 3 * K).to(R.TYPES[kind]))


def test_experts_sums_are_fp32_where_asked():
    rows, N, K, E = 3000, 1030, 640, 3
    offsets = torch.tensor([0, 1500, 1501, 2990], dtype=torch.int32, device="cuda")
    a, b = cancelling(K, 1)
    factor = torch.tensor([1.0, 0.25, 4.0])
    got = sg.gemm_fp8_experts(stored(a.repeat(rows, 1)), torch.ones(rows, 5, device="cuda"), stored(b.repeat(E, N, 1)),
                              factor.to("cuda").view(E, 1, 1).expand(E, N, 5), offsets, fp32_sums=True)
    want = torch.zeros(rows, N)
    for e, (at, to) in enumerate([(0, 1500), (1500, 1501), (1501, 2990)]):
        want[at:to] = 3 * K * factor[e]
    assert torch.equal(got.cpu(), want.bfloat16())
    # as the summed axis: 128 rows of one expert in the first block, 512 of the other in blocks 2 to 5
    offsets = torch.tensor([0, 128, 640], dtype=torch.int32, device="cuda")
    (a, b), used = cancelling(128 * 7, 3), torch.ones(7, 128)
    used[1], used[6] = 0.0, 0.0
    a, b = (x.view(7, 128) * used for x in (a, b))
    got = sg.gemm_fp8_experts_wgrad(stored(a.flatten().repeat(300, 1)), torch.ones(300, 7, device="cuda"),
                                    stored(b.flatten().repeat(500, 1)), torch.ones(500, 7, device="cuda"), offsets,
                                    dtype=torch.float16, fp32_sums=True)
    want = torch.stack([torch.full((300, 500), 3.0 * n) for n in (128, 512)]).to(torch.float16)
    assert torch.equal(got.cpu(), want)
