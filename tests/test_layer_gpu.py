"""The norm, gated activations and products with an epilogue on the GPU against plain 64-bit definitions."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _fp8 as R
from tests import _gpu as G
from tests import _layer as L

pytestmark = pytest.mark.gpu

KINDS = ["fp32", "bf16", "fp16"]
# An error of the FP32 value of y = h a w: the sum of squares has 16 + 6 + 16 additions in a row at most and its
# products' roundings, half of which the root passes on; quotient, eps, root, reciprocal and two products: 26.
NORM = 26 * L.U


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()


def matrix(rows, cols, seed, kind, pad=0, offset=0, spread=1.0):
    """A GPU matrix in a buffer of NaN: padded rows, its first element `offset` past the buffer's."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.5 * torch.randn(1, cols, generator=g)) * spread
    room = torch.full((offset + rows * (cols + pad) + 8,), float("nan"), dtype=R.TYPES[kind])
    room[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = x.to(R.TYPES[kind])
    return room.to("cuda")[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def added(x, r, kind):
    """x + r as the kernel forms it: added in FP32, rounded to the type."""
    return (x.float() + r.float()).to(R.TYPES[kind])


# ---- the norm --------------------------------------------------------------------

SHAPES = [(1, 1, 0, 0), (1, 128, 0, 0), (3, 127, 1, 1), (5, 129, 3, 0), (4, 512, 0, 0), (7, 513, 8, 3), (2, 1024, 0, 0),
          (9, 1025, 5, 1), (3, 2048, 0, 0), (130, 2047, 1, 1), (2, 4096, 0, 0), (5, 4097, 0, 2), (3, 8192, 8, 0),
          (2, 8200, 0, 0), (1, 16384, 0, 0), (2, 16383, 1, 1), (1100, 260, 0, 0), (2100, 100, 4, 0), (1500, 1500, 0, 0)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_norm(kind, rows, cols, pad, offset):
    print(f"[gpu] rms_norm {kind} {rows}x{cols} pad {pad} offset {offset}", flush=True)
    x, r = matrix(rows, cols, 1, kind, pad, offset), matrix(rows, cols, 2, kind, pad, offset, 2.0)
    for weight, residual in ((torch.float32, r), (R.TYPES[kind], None)):
        w = (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(3))).to(weight).to("cuda")
        Q, S, H, a, Y = sg.rms_norm_fp8(x, w, residual=residual, eps=1e-5, wide=True)
        torch.cuda.synchronize()
        if residual is None:
            assert H is x
        else:
            assert torch.equal(H, added(x, r, kind))
        rstd, y = L.norm(L.plain(H), L.plain(w), 1e-5)
        L.near(a, rstd, 24 * L.U * rstd, "fp32")
        L.quantised(Q, S, y, NORM * np.abs(y))
        L.near(Y, y, NORM * np.abs(y), kind)
        Y2, H2, a2 = sg.rms_norm(x, w, residual=residual, eps=1e-5)
        assert torch.equal(Y2, Y) and torch.equal(H2, H) and torch.equal(a2, a)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_norm_backward(kind, rows, cols, pad, offset):
    print(f"[gpu] rms_norm_backward {kind} {rows}x{cols} pad {pad} offset {offset}", flush=True)
    h, dy = matrix(rows, cols, 1, kind, pad, offset), matrix(rows, cols, 2, kind, pad, offset, 0.3)
    dh = matrix(rows, cols, 4, kind, pad, offset, 0.3)
    for weight, more in ((torch.float32, dh), (R.TYPES[kind], None)):
        w = (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(3))).to(weight).to("cuda")
        _, _, rstd = sg.rms_norm(h, w)
        dX, dw = sg.rms_norm_backward(dy, h, rstd, w, dH=more)
        torch.cuda.synchronize()
        other = np.zeros((rows, cols)) if more is None else L.plain(more)
        want, want_w, error, size = L.norm_backward(L.plain(dy), L.plain(h), L.plain(rstd), L.plain(w), other)
        L.near(dX, want, error, kind)
        # a team's rows (3 at most here) in turn, the four teams, the groups by 64 and these, and the two products
        assert (np.abs(L.plain(dw) - want_w) <= (3 + 4 + rows / 64 + 8 + 3) * L.U * size + 1e-40).all()
        again = sg.rms_norm_backward(dy, h, rstd, w, dH=more)
        assert torch.equal(again[0], dX) and torch.equal(again[1], dw)


def test_norm_backward_against_differences():
    rows, cols, eps = 6, 200, 1e-3
    x, w = L.plain(matrix(rows, cols, 1, "fp32")), 1 + 0.1 * np.random.default_rng(0).standard_normal(cols)
    dy = np.random.default_rng(1).standard_normal((rows, cols))
    f32 = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    _, H, rstd = sg.rms_norm(f32(x), f32(w), eps=eps)
    dX, dw = (L.plain(v) for v in sg.rms_norm_backward(f32(dy), H, rstd, f32(w)))
    loss = lambda x, w: (dy * L.norm(x, w, eps)[1]).sum()  # noqa: E731
    step = 1e-5
    for k in range(20):
        i, j = k % rows, 37 * k % cols
        e = np.zeros_like(x)
        e[i, j] = step
        # the difference is off by step^2 times a third derivative (under 1e3) and 1e-12 of rounding; the kernel by 1e-5
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * step) - dX[i, j]) < 1e-4
        v = np.zeros_like(w)
        v[j] = step
        assert abs((loss(x, w + v) - loss(x, w - v)) / (2 * step) - dw[j]) < 1e-4


def test_norm_in_place_and_padding_untouched():
    for kind in KINDS:
        x, r = matrix(33, 700, 1, kind), matrix(33, 700, 2, kind, 12, 0)
        w = torch.ones(700, device="cuda")
        want, before = added(x, r, kind), r.clone()
        Q, S, H, a = sg.rms_norm_fp8(x, w, residual=r, H=r)
        Q2, S2, H2, a2 = sg.rms_norm_fp8(x, w, residual=before)
        assert H is r and torch.equal(r, want) and torch.equal(H2, want) and torch.equal(a, a2) and torch.equal(S, S2)
        assert torch.equal(Q.view(torch.uint8), Q2.view(torch.uint8))
        assert bool(r.as_strided((32, 12), (712, 1), 700).isnan().all())


@pytest.mark.parametrize("cols", [300, 1000, 4096, 9000])
def test_norm_of_extreme_rows(cols):
    """Squares past FP32's range, tiny ones, a row of zeros, an infinity and a NaN, each in a row of its own."""
    x = matrix(9, cols, 1, "fp32")
    x[0] *= 1e25
    x[1] *= 1e-30
    x[2] = 0
    x[3, cols // 2] = float("inf")
    x[4, cols - 1] = float("nan")
    x[5] = 3e38
    w = torch.ones(cols, device="cuda")
    Q, S, H, a, Y = sg.rms_norm_fp8(x, w, eps=0.0, wide=True)
    torch.cuda.synchronize()
    h = L.plain(x)
    for row in (0, 1, 5, 6, 7, 8):
        rstd, y = L.norm(h[row:row + 1], np.ones(cols), 0.0)
        L.near(a[row:row + 1], rstd, 24 * L.U * rstd, "fp32")
        L.near(Y[row:row + 1], y, NORM * np.abs(y), "fp32")
        L.quantised(Q[row:row + 1], S[row:row + 1], y, NORM * np.abs(y))
    assert a[2] == float("inf") and bool(Y[2].isnan().all()) and bool(a[4].isnan()) and bool(Y[4].isnan().all())
    assert a[3] == 0 and bool(Y[3, cols // 2].isnan()) and int(Y[3].isnan().sum()) == 1
    assert bool(S[4].isnan().all()) and bool(S[3, cols // 2 // 128].isnan()) and int(S[3].isnan().sum()) == 1
    Y, _, a = sg.rms_norm(x[2:3], w, eps=1e-6)
    assert bool((Y == 0).all()) and abs(float(a) - 1e3) < 1e-3


def test_empty_norms():
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda")
    Q, S, H, a = sg.rms_norm_fp8(x, w)
    assert Q.shape == (0, 64) and S.shape == (0, 1) and H is x and a.shape == (0,)
    dX, dw = sg.rms_norm_backward(x, x, a, w)
    assert dX.shape == (0, 64) and bool((dw == 0).all()) and dw.shape == (64,)


# ---- gated activations -------------------------------------------------------------

GATED = [(1, 1, 0, 0), (1, 128, 0, 0), (3, 127, 1, 1), (5, 129, 2, 0), (17, 1000, 8, 3), (130, 260, 3, 0), (2, 4096, 0, 0),
         (1000, 64, 0, 0)]


@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("rows,cols,pad,offset", GATED)
def test_gated(act, rows, cols, pad, offset):
    kind = KINDS[(rows + cols + len(act)) % 3]
    print(f"[gpu] gated {act} {kind} {rows}x{cols} pad {pad} offset {offset}", flush=True)
    H, dZ = matrix(rows, 2 * cols, 1, kind, pad, offset, 2.0), matrix(rows, cols, 2, kind, pad, offset)
    Q, S, Z = sg.gated_fp8(H, activation=act, wide=True)
    dH = sg.gated_backward(dZ, H, activation=act)
    torch.cuda.synchronize()
    h, dz = L.plain(H), L.plain(dZ)
    g, u = h[:, :cols], h[:, cols:]
    value, slope, value_error, slope_error = L.activation(g, act)
    z, error = value * u, L.U * (np.abs(u) * value_error + 2 * np.abs(value * u))
    L.quantised(Q, S, z, error + 1e-38)
    L.near(Z, z, error, kind)
    assert torch.equal(sg.gated(H, activation=act), Z)
    L.near(dH[:, :cols], slope * u * dz, L.U * np.abs(u * dz) * (slope_error + 3 * np.abs(slope)) + 1e-37, kind)
    L.near(dH[:, cols:], value * dz, L.U * np.abs(dz) * (value_error + 2 * np.abs(value)) + 1e-37, kind)


@pytest.mark.parametrize("act", L.ACTS)
def test_activations_over_their_range(act):
    """Every magnitude, both signs, the infinities and NaN, in FP32, by way of u = dz = 1."""
    mags = np.concatenate([2.0 ** np.arange(-126, 128), np.linspace(0.001, 30, 3000), np.linspace(30, 200, 500), [0.0, 3.4e38]])
    p = np.concatenate([mags, -mags, [np.inf, -np.inf, np.nan]]).astype(np.float32)
    H = torch.stack([torch.from_numpy(p), torch.ones(p.size)], 1).to("cuda")
    z = L.plain(sg.gated(H, activation=act))[:, 0]
    d = L.plain(sg.gated_backward(torch.ones(p.size, 1, device="cuda"), H, activation=act))
    assert np.isnan(z[-1]) and (np.isnan(d[-1, 0]) if act != "none" else d[-1, 0] == 1.0)  # the identity's slope is 1 anywhere
    least = {"none": -np.inf}.get(act, 0.0)
    assert z[-3] == np.inf and d[-3, 0] == 1.0 and z[-2] == least and d[-2, 0] == (1.0 if act == "none" else 0.0)
    value, slope, value_error, slope_error = L.activation(p[:-3].astype(np.float64), act)
    # results under 2^-126 may be flushed
    assert (np.abs(z[:-3] - value) <= L.U * (value_error + np.abs(value)) + 2.0 ** -120).all()
    assert (np.abs(d[:-3, 0] - slope) <= L.U * (slope_error + np.abs(slope)) + 2.0 ** -120).all()
    np.testing.assert_array_equal(d[:, 1], z)


def test_gated_nan_stays_in_its_block():
    H = matrix(4, 600, 1, "bf16")
    H[1, 5] = float("nan")
    H[2, 300 + 290] = float("inf")
    Q, S = sg.gated_fp8(H)
    S, q = S.cpu().numpy(), R.bytes_of(Q)
    assert np.isnan(S).sum() == 2 and np.isnan(S[1, 0]) and np.isnan(S[2, 2])
    assert np.isnan(q[1, :128]).all() and np.isnan(q[2, 256:]).all() and np.isnan(q).sum() == 128 + 44


# ---- the epilogue ------------------------------------------------------------------

def operands(M, N, K, tall, seed=0, pad=None, offset=0):
    pad = -K % 16 if pad is None else pad
    A, B = R.random_bytes(M, K, seed + 1, pad, offset), R.random_bytes(N, K, seed + 2, pad, offset)
    sa = R.random_scales(M, -(-K // 128), seed + 3) * 1e-3
    sb = R.random_scales(-(-N // tall), -(-K // 128), seed + 4, tall == 1)
    a, b = R.values(R.bytes_of(A), sa.cpu().numpy()), R.values(R.bytes_of(B), sb.cpu().numpy(), tall)
    return (A, sa, B, sb), a @ b.T, np.abs(a) @ np.abs(b).T


def check_epilogue(C, P, product, size, K, kind, act, bias, residual):
    """p is off as a product of FP32 results is (16-bit results: by the FP8 unit's sums too) before its rounding."""
    torch.cuda.synchronize()
    p = product + (0.0 if bias is None else bias)
    inside = R.product_bound(product, size, K, kind) - R.product_bound(product, 0 * size, K, kind) + L.U * np.abs(p)
    inside /= 1 + R.half_step(kind)[0]
    value, _, value_error, _ = L.activation(p, act, kind != "fp32")
    if P is not None:
        L.near(P, p, inside, kind)
    want = value + (0.0 if residual is None else residual)
    # no activation's slope is over 1.13
    L.near(C, want, 1.13 * inside + L.U * (1.2 * value_error + np.abs(value) + np.abs(want)) + 1e-37, kind)


EPILOGUES = [(1, 1, 1, 1), (3, 33, 100, 1), (16, 256, 512, 128), (17, 100, 640, 1), (33, 64, 1000, 128), (40, 520, 384, 1),
             (64, 512, 256, 128), (70, 130, 300, 1), (129, 257, 130, 128), (200, 300, 1024, 1), (257, 512, 260, 128),
             (300, 1000, 144, 1), (520, 640, 384, 128), (1500, 4060, 300, 1), (2100, 2300, 256, 128), (2100, 2300, 200, 1)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K,tall", EPILOGUES)
def test_epilogue(kind, M, N, K, tall):
    act = L.ACTS[(M + N + K + len(kind)) % 5]
    print(f"[gpu] epilogue {kind} {act} {M}x{N}x{K} tall {tall}", flush=True)
    g = torch.Generator().manual_seed(5)
    bias, room = torch.randn(N, generator=g).to("cuda"), torch.randn(M, N + 3, generator=g).to(R.TYPES[kind]).to("cuda")
    residual = room[:, :N]
    (A, sa, B, sb), product, size = operands(M, N, K, tall)
    C, P = sg.gemm_fp8_epilogue(A, sa, B, sb, bias=bias, activation=act, residual=residual, pre=True)
    assert C.dtype == R.TYPES[kind]
    check_epilogue(C, P, product, size, K, kind, act, L.plain(bias), L.plain(residual))
    before = room.clone()
    assert sg.gemm_fp8_epilogue(A, sa, B, sb, residual, bias=bias, activation=act, residual=residual) is residual
    assert torch.equal(residual, C) and torch.equal(room[:, N:], before[:, N:])
    C = sg.gemm_fp8_epilogue(A, sa, B, sb, dtype=R.TYPES[kind])
    assert torch.equal(C, sg.gemm_fp8(A, sa, B, sb, dtype=R.TYPES[kind]))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", [(1, 500, 1559), (1, 70, 100), (60, 1, 333), (1, 1, 1001)])
def test_epilogue_of_single_rows(kind, M, N, K):
    """A row's stride is its length where there is one row: any number."""
    g = torch.Generator().manual_seed(6)
    bias, residual = torch.randn(N, generator=g).to("cuda"), torch.randn(M, N, generator=g).to(R.TYPES[kind]).to("cuda")
    (A, sa, B, sb), product, size = operands(M, N, K, 1)
    C, P = sg.gemm_fp8_epilogue(A, sa, B, sb, bias=bias, activation="gelu", residual=residual, pre=True)
    check_epilogue(C, P, product, size, K, kind, "gelu", L.plain(bias), L.plain(residual))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad,offset", [(4, 0), (3, 5)])
def test_epilogue_of_any_alignment(kind, pad, offset):
    M, N, K = 200, 270, 333
    for act, tall in (("silu", 1), ("gelu", 128)):
        (A, sa, B, sb), product, size = operands(M, N, K, tall, 7, pad, offset)
        assert sg.sgemm_mi355_fp8_kernel_name(0, R.TYPES[kind] == torch.bfloat16, M, N, K, 0, A.data_ptr(), A.stride(0),
                                              B.data_ptr(), B.stride(0)).startswith("staged")
        bias, residual = torch.randn(N, device="cuda"), torch.randn(M, N, device="cuda").to(R.TYPES[kind])
        C, P = sg.gemm_fp8_epilogue(A, sa, B, sb, bias=bias, activation=act, residual=residual, pre=True)
        check_epilogue(C, P, product, size, K, kind, act, L.plain(bias), L.plain(residual))


def test_epilogue_without_a_product():
    """K = 0: p is the bias; no bias: zero."""
    A, B = torch.empty(5, 0, device="cuda").to(torch.float8_e4m3fn), torch.empty(7, 0, device="cuda").to(torch.float8_e4m3fn)
    sa, sb = torch.empty(5, 0, device="cuda"), torch.empty(7, 0, device="cuda")
    bias, residual = torch.randn(7, device="cuda"), torch.randn(5, 7, device="cuda")
    C = sg.gemm_fp8_epilogue(A, sa, B, sb, bias=bias, activation="relu", residual=residual)
    assert torch.equal(C, residual + bias.clamp_min(0))
    assert bool((sg.gemm_fp8_epilogue(A, sa, B, sb, activation="gelu") == 0).all())


def test_epilogue_with_fp32_sums_and_nan():
    (A, sa, B, sb), product, size = operands(300, 400, 512, 1)
    C = sg.gemm_fp8_epilogue(A, sa, B, sb, activation="silu", fp32_sums=True)
    value, _, error, _ = L.activation(product, "silu", True)
    inside = R.product_bound(product, size, 512, "fp32")
    L.near(C, value, 1.13 * inside + L.U * error, "bf16")
    residual = torch.zeros(300, 400, device="cuda", dtype=torch.bfloat16)
    residual[9, 11] = float("nan")
    C = sg.gemm_fp8_epilogue(A, sa, B, sb, activation="relu", residual=residual)
    assert bool(C[9, 11].isnan()) and int(C.isnan().sum()) == 1
    A = A.clone()
    A.view(torch.uint8)[7, 3] = 0x7F
    for act in L.ACTS:
        C, P = sg.gemm_fp8_epilogue(A, sa, B, sb, activation=act, pre=True)
        assert bool(C[7].isnan().all()) and int(C.isnan().sum()) == 400 == int(P.isnan().sum())


@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("kind", KINDS)
def test_epilogue_backward_over_the_activations_range(act, kind):
    """Every magnitude that the type holds, both signs, the infinities and NaN."""
    mags = np.concatenate([2.0 ** np.arange(-24, 16), np.linspace(0.01, 30, 3000), np.linspace(30, 200, 500), [0.0, 6e4]])
    if kind != "fp16":
        mags = np.concatenate([mags, 2.0 ** np.arange(-126, 128), [3.3e38]])
    p = torch.from_numpy(np.concatenate([mags, -mags, [np.inf, -np.inf, np.nan]])).to(R.TYPES[kind]).to("cuda")[None]
    dP, _ = sg.epilogue_backward(torch.ones_like(p), p, activation=act)
    assert dP[0, -3] == 1.0 and dP[0, -2] == (1.0 if act == "none" else 0.0) and (act == "none" or bool(dP[0, -1].isnan()))
    _, slope, _, error = L.activation(L.plain(p)[:, :-3], act, kind != "fp32")
    L.near(dP[:, :-3], slope, L.U * (error + np.abs(slope)), kind)


@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("kind", KINDS)
def test_epilogue_over_the_activations_range(act, kind):
    """K = 0: p is the bias, every magnitude of it, the infinities and NaN, by each kernel's epilogue."""
    mags = np.concatenate([2.0 ** np.arange(-24, 16), np.linspace(0.01, 30, 400), np.linspace(30, 200, 50), [0.0, 6e4]])
    if kind != "fp16":
        mags = np.concatenate([mags, 2.0 ** np.arange(-126, 128), [3.3e38]])
    bias = torch.from_numpy(np.concatenate([mags, -mags, [np.inf, -np.inf, np.nan]])).float().to("cuda")
    N = bias.numel()
    want, _, error, _ = L.activation(L.plain(bias)[None, :-3], act, kind != "fp32")
    for M, K in ((3, 0), (3, 128), (2000, 128), (2000, 127)):
        A, B = torch.zeros(M, K + 1, device="cuda").to(torch.float8_e4m3fn)[:, :K], torch.zeros(N, K, device="cuda").to(torch.float8_e4m3fn)
        sa, sb = torch.ones(M, -(-K // 128), device="cuda"), torch.ones(N, -(-K // 128), device="cuda")
        C = sg.gemm_fp8_epilogue(A, sa, B, sb, bias=bias, activation=act, dtype=R.TYPES[kind])
        assert bool((C[:1] == C)[:, :-1].all()) and C[0, -3] == float("inf") and bool(C[:, -1].isnan().all())
        assert C[0, -2] == (-float("inf") if act == "none" else 0.0)
        L.near(C[:1, :-3], want, L.U * (error + np.abs(want)), kind)


@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("rows,cols,pad,offset", [(1, 1, 0, 0), (3, 127, 1, 1), (70, 128, 0, 0), (129, 129, 2, 0), (33, 512, 8, 3),
                                                  (700, 1030, 0, 0), (3000, 40, 0, 0), (5000, 600, 0, 0)])
def test_epilogue_backward(act, rows, cols, pad, offset):
    kind = KINDS[(rows + cols + len(act)) % 3]
    print(f"[gpu] epilogue_backward {act} {kind} {rows}x{cols}", flush=True)
    P, dC = matrix(rows, cols, 1, kind, pad, offset, 1.5), matrix(rows, cols, 2, kind, pad, offset)
    dP, db = sg.epilogue_backward(dC, P, activation=act)
    torch.cuda.synchronize()
    _, slope, _, slope_error = L.activation(L.plain(P), act, kind != "fp32")
    dc = L.plain(dC)
    want, error = slope * dc, L.U * np.abs(dc) * (slope_error + np.abs(slope)) + 1e-37
    L.near(dP, want, error, kind)
    # a thread's rows (8 here at most), a group's threads (16), every 64th group (3), and these by fours and pairs (8): under 64 additions
    assert (np.abs(L.plain(db) - want.sum(0)) <= error.sum(0) + 64 * L.U * np.abs(want).sum(0)).all()
    again, none = sg.epilogue_backward(dC, P, activation=act, bias=False)
    assert none is None and torch.equal(again, dP)
    assert torch.equal(sg.epilogue_backward(dC, P, activation=act)[1], db)


def test_empty_epilogues():
    x = torch.empty(0, 30, device="cuda")
    dP, db = sg.epilogue_backward(x, x, activation="silu")
    assert dP.shape == (0, 30) and bool((db == 0).all())
    Q, S = sg.gated_fp8(torch.empty(3, 0, device="cuda"))
    assert Q.shape == (3, 0) and sg.gated(x).shape == (0, 15) and sg.gated_backward(x[:, :15], x).shape == (0, 30)
