"""FP8 quantisers and products on the GPU against plain 64-bit definitions."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _fp8 as R
from tests import _gpu as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()


def wide(rows, cols, seed, kind, pad=0, offset=0):
    """A GPU matrix whose columns differ in size, in a buffer of NaN with padded rows."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(1, cols, generator=g))
    room = torch.full((offset + rows * (cols + pad),), float("nan"), dtype=R.TYPES[kind])
    room[offset:].view(rows, cols + pad)[:, :cols] = x.to(R.TYPES[kind])
    return room.to("cuda")[offset:].view(rows, cols + pad)[:, :cols]


def plain(x):
    return x.float().cpu().numpy()


def check_quantized(Q, S, want_q, want_s):
    torch.cuda.synchronize()
    np.testing.assert_array_equal(S.cpu().numpy(), want_s)
    np.testing.assert_array_equal(R.bytes_of(Q), want_q)


# ---- quantisers: every step is defined to the bit ------------------------------

@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,cols,pad,offset", [
    (1, 1, 0, 0), (1, 128, 0, 0), (3, 127, 0, 1), (5, 129, 3, 0), (17, 1000, 8, 3), (130, 260, 4, 0), (2, 4096, 0, 0)])
def test_quantize_rows_and_tiles(kind, rows, cols, pad, offset):
    print(f"[gpu] quantize {kind} {rows}x{cols} pad {pad} offset {offset}", flush=True)
    X = wide(rows, cols, rows + cols, kind, pad, offset)
    Q, S = sg.quantize_fp8(X)
    assert Q.stride(0) % 16 == 0 and S.shape == (rows, -(-cols // 128))
    check_quantized(Q, S, *R.quantize(plain(X)))
    check_quantized(*sg.quantize_fp8(X, blocks=True), *R.quantize(plain(X), 128))


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,cols,pad,offset", [
    (1, 1, 0, 0), (128, 128, 0, 0), (127, 3, 0, 1), (129, 5, 3, 0), (1000, 17, 8, 3), (260, 130, 4, 0), (700, 300, 0, 0)])
def test_quantize_cols(kind, rows, cols, pad, offset):
    print(f"[gpu] quantize cols {kind} {rows}x{cols} pad {pad} offset {offset}", flush=True)
    X = wide(rows, cols, rows + cols, kind, pad, offset)
    check_quantized(*sg.quantize_fp8_cols(X), *R.quantize(np.ascontiguousarray(plain(X).T)))


def test_quantize_gathered_rows_and_bad_indices():
    X = wide(40, 200, 1, "bf16")
    index = torch.tensor([3, 3, 39, -1, 40, 0, 2 ** 31 - 1, -2 ** 31, 7], dtype=torch.int32, device="cuda")
    inside = (index.cpu().numpy() >= 0) & (index.cpu().numpy() < 40)
    x = np.where(inside[:, None], plain(X)[np.where(inside, index.cpu().numpy(), 0)], np.float32(0))
    check_quantized(*sg.quantize_fp8(X, index=index), *R.quantize(x))
    check_quantized(*sg.quantize_fp8_cols(X, index=index), *R.quantize(np.ascontiguousarray(x.T)))
    Q, S = sg.quantize_fp8(X, index=index[:0])
    assert Q.shape == (0, 200) and S.shape == (0, 2)


def test_quantize_special_values():
    X = torch.zeros(9, 256)
    X[1, 5], X[2, 200] = float("nan"), float("inf")
    X[3, 3], X[3, 4] = 1e-30, -2e-30          # below the least magnitude a block is scaled by
    X[4, :128] = torch.linspace(-3e38, 3e38, 128)
    X[5, :128] = torch.arange(128) * 2.0 ** -149
    X[6, 0], X[6, 1:] = 448.0, torch.arange(255) / 16.0  # ties of e4m3 among them
    X[7] = -X[6]
    X[8, 0], X[8, 1] = 2.0 ** -64, 2.0 ** -74
    check_quantized(*sg.quantize_fp8(X.to("cuda")), *R.quantize(X.numpy()))
    check_quantized(*sg.quantize_fp8_cols(X.to("cuda")), *R.quantize(np.ascontiguousarray(X.numpy().T)))
    check_quantized(*sg.quantize_fp8(X.to("cuda"), blocks=True), *R.quantize(X.numpy(), 128))


def test_quotients_are_rounded_correctly():
    """Random quotients over many scales: a quotient an FP32 step off shows where it crosses a tie of e4m3."""
    g = torch.Generator().manual_seed(5)
    X = torch.randn(512, 1024, generator=g) * torch.exp2(torch.randint(-60, 60, (512, 1), generator=g).float())
    s = X.view(512, 8, 128).abs().amax(-1) / 448.0
    # half of the values next to a tie of their block
    tie = (torch.randint(16, 32, X.shape, generator=g) + 0.5) / 16.0 * torch.exp2(torch.randint(-6, 8, X.shape, generator=g).float())
    near = tie * s.repeat_interleave(128, 1) * (1 + torch.randint(-2, 3, X.shape, generator=g) * 2.0 ** -24)
    keep = (torch.rand(X.shape, generator=g) < 0.5) | (X.abs() == X.view(512, 8, 128).abs().amax(-1).repeat_interleave(128, 1))
    X = torch.where(keep, X, near.float())
    check_quantized(*sg.quantize_fp8(X.to("cuda")), *R.quantize(X.numpy()))


OFFSETS = [[0, 5, 5, 133, 300], [0, 0, 0, 0, 0], [0, 128, 256, 256, 299], [0, 300, 300, 300, 300], [0, 1, 2, 3, 4],
           [0, 0, 127, 128, 300]]


def slots_of(x, off, rows):
    """The transposed matrix of quantize_fp8_cols for these offsets, unquantised."""
    E = len(off) - 1
    out = np.zeros((128 * (rows // 128 + E), x.shape[1]), np.float32)
    for e in range(E):
        at = 128 * (off[e] // 128 + e)
        out[at:at + off[e + 1] - off[e]] = x[off[e]:off[e + 1]]
    return np.ascontiguousarray(out.T)


@pytest.mark.parametrize("off", OFFSETS)
def test_quantize_cols_by_expert(off):
    X = wide(50, 140, 3, "fp32")
    index = torch.randint(0, 50, (300,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).to("cuda")
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    x = plain(X)[index.cpu().numpy()]
    check_quantized(*sg.quantize_fp8_cols(X, index=index, offsets=offsets), *R.quantize(slots_of(x, off, 300)))


def test_quantize_cols_with_bad_offsets_stays_inside():
    """Offsets that fall, or lie outside the rows: limited, so nothing outside the matrices is touched."""
    X = wide(200, 64, 4, "fp32")
    for off in ([5, -3, 500, 100, 90], [0, 2 ** 31 - 1, -2 ** 31, 7, 200], [0, 199, 0, 199, 0]):
        Q, S = sg.quantize_fp8_cols(X, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert Q.shape == (64, 128 * (1 + 4)) and not np.isnan(R.bytes_of(Q)).any() and bool((S > 0).all())


# ---- products ---------------------------------------------------------------------

def check_product(C, a, b, K, kind, init=None):
    torch.cuda.synchronize()
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    if init is not None:
        want, size = want + init, size + np.abs(init)
    off = np.abs(C.double().cpu().numpy() - want)
    worst = (off / R.product_bound(want, size, K, kind)).max() if off.size else 0.0
    assert worst <= 1.0, f"{worst} times the bound"


SHAPES = [(1, 1, 1), (1, 128, 128), (2, 130, 129), (3, 33, 100), (16, 256, 512), (17, 100, 640), (31, 1, 300),
          (33, 64, 1000), (64, 512, 256), (65, 200, 384), (127, 129, 255), (128, 128, 128), (129, 257, 130),
          (200, 300, 1024), (256, 256, 2048), (257, 512, 260), (300, 1000, 144), (520, 640, 384)]


@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, tall):
    kind = ["fp32", "bf16", "fp16"][(M + N + K) % 3]
    print(f"[gpu] gemm_fp8 {M}x{N}x{K} {kind} tall {tall}", flush=True)
    for pad, offset in ((-K % 16, 0), (16 - K % 16, 16), (3, 0), (0, 5)):
        A, B = R.random_bytes(M, K, M, pad, offset), R.random_bytes(N, K, N + 1, pad, offset)
        sa, sb = R.random_scales(M, -(-K // 128), 1), R.random_scales(-(-N // tall), -(-K // 128), 2, tall == 1)
        if kind == "fp16":
            sa = sa * 1e-3
        C = sg.gemm_fp8(A, sa, B, sb, dtype=R.TYPES[kind])
        check_product(C, R.values(R.bytes_of(A), sa.cpu().numpy()), R.values(R.bytes_of(B), sb.cpu().numpy(), tall), K, kind)


@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("M,N,K,pad", [(1500, 4060, 300, 1), (3001, 2047, 400, 0), (1345, 3969, 128, 4), (2880, 2050, 16, 0)])
def test_product_of_many_rows_in_fp32(M, N, K, pad, tall):
    """More 128 x 128 tiles of C than the chip has CUs: some of two rounds, partial rows, columns and blocks."""
    A, B = R.random_bytes(M, K, 1, -K % 16), R.random_bytes(N, K, 2, -K % 16)
    sa, sb = R.random_scales(M, -(-K // 128), 3), R.random_scales(-(-N // tall), -(-K // 128), 4, tall == 1)
    room = torch.randn(M, N + pad, generator=torch.Generator().manual_seed(5)).to("cuda")
    before = room.clone()
    sg.gemm_fp8(A, sa, B, sb, room[:, :N], beta=0.5)
    a, b = R.values(R.bytes_of(A), sa.cpu().numpy()), R.values(R.bytes_of(B), sb.cpu().numpy(), tall)
    check_product(room[:, :N], a, b, K, "fp32", 0.5 * before[:, :N].double().cpu().numpy())
    assert torch.equal(room[:, N:], before[:, N:])


@pytest.mark.parametrize("M,N,K", [(5, 70, 200), (40, 256, 384), (130, 200, 700), (300, 520, 1300)])
def test_product_of_whole_numbers_is_exact(M, N, K):
    for tall in (1, 128):
        A, B = R.random_bytes(M, K, 1, -K % 16, whole=True), R.random_bytes(N, K, 2, -K % 16, whole=True)
        sa, sb = R.random_scales(M, -(-K // 128), 3, powers=True), R.random_scales(-(-N // tall), -(-K // 128), 4, powers=True)
        C = sg.gemm_fp8(A, sa, B, sb, dtype=torch.float32)
        want = R.values(R.bytes_of(A), sa.cpu().numpy()) @ R.values(R.bytes_of(B), sb.cpu().numpy(), tall).T
        np.testing.assert_array_equal(C.double().cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("M,N,K,pad", [(3, 100, 256, 0), (70, 130, 300, 5), (140, 384, 256, 8), (260, 300, 512, 1)])
def test_product_added_to_padded_c(kind, M, N, K, pad):
    A, B = R.random_bytes(M, K, 1, -K % 16), R.random_bytes(N, K, 2, -K % 16)
    sa, sb = R.random_scales(M, -(-K // 128), 3, by_block=False) * 1e-2, R.random_scales(N, -(-K // 128), 4, by_block=False)
    room = torch.randn(M, N + pad, generator=torch.Generator().manual_seed(5)).to(R.TYPES[kind]).to("cuda")
    before = room.clone()
    sg.gemm_fp8(A, sa, B, sb, room[:, :N], beta=-0.5)
    check_product(room[:, :N], R.values(R.bytes_of(A), sa.cpu().numpy()), R.values(R.bytes_of(B), sb.cpu().numpy()), K, kind,
                  -0.5 * before[:, :N].double().cpu().numpy())
    assert torch.equal(room[:, N:], before[:, N:])
    nan = torch.full((M, N + pad), float("nan"), dtype=R.TYPES[kind], device="cuda")
    sg.gemm_fp8(A, sa, B, sb, nan[:, :N])
    torch.cuda.synchronize()
    assert not bool(nan[:, :N].isnan().any()) and bool(nan[:, N:].isnan().all())


def test_product_of_strided_scales_and_nan():
    """Scales in other orders, one scale for a whole row (stride 0), and NaN that stays in its row or column."""
    M, N, K = 150, 140, 400
    A, B = R.random_bytes(M, K, 1), R.random_bytes(N, K, 2)
    sa = torch.rand(M * 4 * 3, generator=torch.Generator().manual_seed(1)).to("cuda").view(M, 4, 3)[:, :, 1]
    sb = torch.rand(N, 1, generator=torch.Generator().manual_seed(2)).to("cuda").expand(N, 4)
    a, b = R.values(R.bytes_of(A), sa.cpu().numpy()), R.values(R.bytes_of(B), sb.cpu().numpy())
    check_product(sg.gemm_fp8(A, sa, B, sb, dtype=torch.float32), a, b, K, "fp32")
    A = A.clone()
    A.view(torch.uint8)[7, 399] = 0x7F
    sb = sb.contiguous()
    sb[9, 2] = float("nan")
    C = sg.gemm_fp8(A, sa, B, sb, dtype=torch.float32).isnan()
    torch.cuda.synchronize()
    assert bool(C[7].all()) and bool(C[:, 9].all()) and int(C.sum()) == M + N - 1


def test_product_of_nothing():
    A, B = R.random_bytes(5, 0, 1), R.random_bytes(6, 0, 2)
    empty = torch.empty(5, 0, device="cuda"), torch.empty(6, 0, device="cuda")
    C = torch.ones(5, 6, device="cuda")
    sg.gemm_fp8(A, empty[0], B, empty[1], C, beta=2.0)
    assert sg.gemm_fp8(A[:0], empty[0][:0], B, empty[1]).shape == (0, 6)
    torch.cuda.synchronize()
    assert bool((C == 2).all())
    assert bool((sg.gemm_fp8(A, empty[0], B, empty[1]) == 0).all())


def test_product_repeats_its_bits_and_follows_its_stream():
    M, N, K = 300, 300, 1000
    A, B = R.random_bytes(M, K, 1, 8), R.random_bytes(N, K, 2, 8)
    sa, sb = R.random_scales(M, 8, 1), R.random_scales(3, 8, 2, False)
    first = sg.gemm_fp8(A, sa, B, sb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        assert torch.equal(sg.gemm_fp8(A, sa, B, sb), first)
        C = sg.gemm_fp8(A, sa, B, sb, stream=side)
        side.synchronize()
        assert torch.equal(C, first)


# ---- experts ------------------------------------------------------------------------

EXPERT_OFFSETS = [[0, 5, 5, 133, 300], [0, 0, 0, 0, 0], [0, 128, 256, 256, 299], [0, 300, 300, 300, 300], [0, 1, 2, 3, 4],
                  [0, 0, 257, 258, 290], [0, 300]]


@pytest.mark.parametrize("off", EXPERT_OFFSETS)
@pytest.mark.parametrize("N,K,tall", [(100, 260, 1), (256, 256, 128), (130, 512, 128)])
def test_experts(off, N, K, tall):
    E, rows, kind = len(off) - 1, 300, ["fp32", "bf16"][N % 3 % 2]
    print(f"[gpu] experts {off} N={N} K={K} {kind}", flush=True)
    for pad in (-K % 16, 3):
        A = R.random_bytes(rows, K, 1, pad)
        B = R.random_bytes(E * N, K, 2, pad).unflatten(0, (E, N))
        sa = R.random_scales(rows, -(-K // 128), 3)
        sb = R.random_scales(E * -(-N // tall), -(-K // 128), 4, False).unflatten(0, (E, -1))
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        C = torch.full((rows, N), float("nan"), dtype=R.TYPES[kind], device="cuda")
        sg.gemm_fp8_experts(A, sa, B, sb, offsets, C)
        a = R.values(R.bytes_of(A), sa.cpu().numpy())
        for e in range(E):
            b = R.values(R.bytes_of(B[e]), sb[e].cpu().numpy(), tall)
            check_product(C[off[e]:off[e + 1]], a[off[e]:off[e + 1]], b, K, kind)
        assert bool((C[off[-1]:] == 0).all())


def test_many_experts_of_few_rows():
    E, N, K = 150, 64, 384
    counts = torch.randint(0, 4, (E,), generator=torch.Generator().manual_seed(3))
    off = [0, *counts.cumsum(0).tolist()]
    rows = off[-1] + 2
    A, B = R.random_bytes(rows, K, 1), R.random_bytes(E * N, K, 2).unflatten(0, (E, N))
    sa, sb = R.random_scales(rows, 3, 3), R.random_scales(E, 3, 4, False).unsqueeze(1)
    C = sg.gemm_fp8_experts(A, sa, B, sb, torch.tensor(off, dtype=torch.int32, device="cuda"), dtype=torch.float32)
    a = R.values(R.bytes_of(A), sa.cpu().numpy())
    for e in range(E):
        b = R.values(R.bytes_of(B[e]), sb[e].cpu().numpy(), 128)
        check_product(C[off[e]:off[e + 1]], a[off[e]:off[e + 1]], b, K, "fp32")
    assert bool((C[off[-1]:] == 0).all())


@pytest.mark.parametrize("off", EXPERT_OFFSETS)
@pytest.mark.parametrize("M,N,beta", [(70, 130, 0.0), (256, 100, 0.5), (129, 257, 0.0)])
def test_experts_weight_gradient(off, M, N, beta):
    rows, E = 300, len(off) - 1
    print(f"[gpu] wgrad {off} M={M} N={N}", flush=True)
    Y, X = wide(rows, M, 1, "fp32"), wide(rows, N, 2, "bf16")
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    (A, sa), (B, sb) = sg.quantize_fp8_cols(Y, offsets=offsets), sg.quantize_fp8_cols(X, offsets=offsets)
    C = torch.randn(E, M, N, generator=torch.Generator().manual_seed(5)).to("cuda")
    init = beta * C.double().cpu().numpy()
    sg.gemm_fp8_experts_wgrad(A, sa, B, sb, offsets, C, beta=beta)
    a, b = R.values(R.bytes_of(A), sa.cpu().numpy()), R.values(R.bytes_of(B), sb.cpu().numpy())
    for e in range(E):
        at = 128 * (off[e] // 128 + e)
        to = at + off[e + 1] - off[e]
        check_product(C[e], a[:, at:to], b[:, at:to], max(to - at, 1), "fp32", init[e])


def test_experts_with_bad_offsets_stay_inside():
    A, B = R.random_bytes(200, 256, 1), R.random_bytes(4 * 64, 256, 2).unflatten(0, (4, 64))
    sa, sb = R.random_scales(200, 2, 1), R.random_scales(4, 2, 2, False).unsqueeze(1)
    W, sw = R.random_bytes(64, 128 * 5, 3), R.random_scales(64, 5, 3)
    for off in ([5, -3, 500, 100, 90], [0, 2 ** 31 - 1, -2 ** 31, 7, 200], [0, 199, 0, 199, 0]):
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        room = torch.zeros(202, 64, device="cuda")
        sg.gemm_fp8_experts(A, sa, B, sb, offsets, room[1:201])
        out = sg.gemm_fp8_experts_wgrad(W, sw, W, sw, offsets)
        torch.cuda.synchronize()
        assert bool((room[0] == 0).all()) and bool((room[201] == 0).all()) and bool(out.isfinite().all())


# ---- graphs and far offsets --------------------------------------------------------------

def test_captured_calls_replay():
    """Every call captured once and replayed on changed inputs, with eager work between, equals the eager call."""
    X, W = wide(200, 300, 1, "bf16"), wide(256, 300, 2, "fp32")
    offsets = torch.tensor([0, 50, 50, 190], dtype=torch.int32, device="cuda")

    def work():
        q, s = sg.quantize_fp8(X)
        w, t = sg.quantize_fp8(W, blocks=True)
        e = sg.gemm_fp8_experts(q, s, w.expand(3, -1, -1), t.expand(3, -1, -1), offsets)
        c, u = sg.quantize_fp8_cols(X, offsets=offsets)
        return sg.gemm_fp8(q, s, w, t), e, sg.gemm_fp8_experts_wgrad(c, u, c, u, offsets)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for i in range(4):
        X.copy_(wide(200, 300, 10 + i, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(got, work()):
            assert torch.equal(g, w)


def test_offsets_past_32_bits():
    """Operands over 2^31 bytes (rows, and experts), checked at their far end."""
    rows, K, N = 70000, 32768, 64
    A = torch.zeros(rows, K, dtype=torch.uint8, device="cuda")
    A[-3:] = 0x38  # 1.0
    sa = torch.ones(256, 1, device="cuda").t().expand(rows, 256)
    B = torch.full((N, K), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    C = sg.gemm_fp8(A.view(torch.float8_e4m3fn), sa, B, torch.ones(1, 256, device="cuda"), dtype=torch.float32)
    torch.cuda.synchronize()
    assert bool((C[-3:] == K).all()) and bool((C[:-3] == 0).all())
    E, N, K = 40, 8192, 8192
    W = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    W[-1, -1] = 0x38
    offsets = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    X = torch.full((E, K), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    C = sg.gemm_fp8_experts(X, torch.ones(E, 64, device="cuda"), W.view(torch.float8_e4m3fn),
                            torch.ones(E, 64, 64, device="cuda"), offsets, dtype=torch.float32)
    torch.cuda.synchronize()
    assert float(C[-1, -1]) == K and float(C.sum()) == K
