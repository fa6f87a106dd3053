"""Refusals of the FP8 and routing calls: codes come from the host before any HIP call (no GPU needed)."""
from __future__ import annotations

import os

import numpy as np
import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _fp8 as R

BIG = 2 ** 31 - 1
# Fake, never-dereferenced device addresses, far apart.
X, Q, S, T, I, O, C, D = (0x10_0000_0000 * (i + 1) for i in range(8))


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(sg.LIB_PATH):
        from dense_fp32_matrix_02_amd import build
        build.build()
    return sg.load()


def call(fn, good, **bad):
    args = dict(good, **bad)
    return fn(*args.values())


ROWS = dict(type=0, rows=10, cols=300, X=X, ldx=300, index=None, n=0, Q=Q, ldq=304, S=S, s_row=1, s_block=10, stream=0)
COLS = dict(type=1, rows=10, cols=300, X=X, ldx=300, index=I, n=20, offsets=O, experts=2, Q=Q, ldq=256, S=S, s_row=1,
            s_block=300, stream=0)
TILES = dict(type=2, rows=200, cols=300, X=X, ldx=300, Q=Q, ldq=304, S=S, s_row=3, s_block=1, stream=0)
GEMM = dict(type=0, M=10, N=20, K=300, A=X, lda=304, SA=S, sa_row=1, sa_block=10, B=Q, ldb=304, SB=T, sb_row=1, sb_block=20,
            sb_rows=1, beta=0.0, C=C, ldc=20, stream=0)
EXPERTS = dict(type=1, rows=10, N=20, K=300, experts=3, A=X, lda=304, SA=S, sa_row=1, sa_block=10, B=Q, ldb=304,
               strideB=6080, SB=T, sb_row=3, sb_block=1, stride_sb=3, sb_rows=128, offsets=O, C=C, ldc=20, stream=0)
WGRAD = dict(type=0, rows=300, M=10, N=20, experts=3, A=X, lda=640, SA=S, sa_row=1, sa_block=10, B=Q, ldb=640, SB=T, sb_row=1,
             sb_block=20, offsets=O, beta=0.0, C=C, ldc=20, strideC=200, stream=0)

E = sg
BAD = [
    (sg.sgemm_mi355_fp8_quantize_rows, ROWS, [
        (dict(type=3), E.ERR_TYPE), (dict(type=-1), E.ERR_TYPE), (dict(rows=-1), E.ERR_DIM), (dict(cols=-1), E.ERR_DIM),
        (dict(index=I, n=-1), E.ERR_DIM), (dict(ldx=299), E.ERR_LD), (dict(ldq=299), E.ERR_LD), (dict(X=None), E.ERR_NULL),
        (dict(Q=None), E.ERR_NULL), (dict(S=None), E.ERR_NULL), (dict(X=X + 2), E.ERR_ALIGN), (dict(S=S + 1), E.ERR_ALIGN),
        (dict(index=I + 2, n=3), E.ERR_ALIGN), (dict(s_row=-1), E.ERR_STRIDE), (dict(s_row=0), E.ERR_STRIDE),
        (dict(s_block=9), E.ERR_STRIDE), (dict(Q=X + 8), E.ERR_ALIAS), (dict(S=X), E.ERR_ALIAS), (dict(S=Q), E.ERR_ALIAS),
        (dict(index=Q, n=4), E.ERR_ALIAS), (dict(rows=BIG), E.ERR_EXTENT), (dict(cols=BIG, ldx=BIG, ldq=BIG), E.ERR_EXTENT),
        (dict(rows=BIG - 1024, s_block=BIG), E.ERR_ALIAS), (dict(rows=0), E.OK), (dict(cols=0), E.OK), (dict(index=I, n=0), E.OK)]),
    (sg.sgemm_mi355_fp8_quantize_cols, COLS, [
        (dict(type=5), E.ERR_TYPE), (dict(experts=0), E.ERR_DIM), (dict(experts=-2), E.ERR_DIM), (dict(n=-1), E.ERR_DIM),
        (dict(ldq=255), E.ERR_LD), (dict(ldx=1), E.ERR_LD), (dict(offsets=O + 1), E.ERR_ALIGN), (dict(X=None), E.ERR_NULL),
        (dict(s_block=299), E.ERR_STRIDE), (dict(offsets=S), E.ERR_ALIAS), (dict(Q=S), E.ERR_ALIAS),
        (dict(experts=BIG // 128), E.ERR_EXTENT), (dict(cols=0), E.OK), (dict(offsets=None, n=0), E.OK)]),
    (sg.sgemm_mi355_fp8_quantize_tiles, TILES, [
        (dict(type=3), E.ERR_TYPE), (dict(rows=-1), E.ERR_DIM), (dict(ldq=200), E.ERR_LD), (dict(X=X + 1), E.ERR_ALIGN),
        (dict(s_row=2), E.ERR_STRIDE), (dict(Q=None), E.ERR_NULL), (dict(S=X), E.ERR_ALIAS), (dict(rows=0), E.OK)]),
    (sg.sgemm_mi355_fp8_gemm, GEMM, [
        (dict(type=3), E.ERR_TYPE), (dict(sb_rows=64), E.ERR_OP), (dict(sb_rows=0), E.ERR_OP), (dict(M=-1), E.ERR_DIM),
        (dict(N=-1), E.ERR_DIM), (dict(K=-1), E.ERR_DIM), (dict(lda=299), E.ERR_LD), (dict(ldb=299), E.ERR_LD),
        (dict(ldc=19), E.ERR_LD), (dict(sa_row=-1), E.ERR_STRIDE), (dict(sb_block=-1), E.ERR_STRIDE), (dict(A=None), E.ERR_NULL),
        (dict(SB=None), E.ERR_NULL), (dict(C=None), E.ERR_NULL), (dict(C=C + 2), E.ERR_ALIGN), (dict(SA=S + 3), E.ERR_ALIGN),
        (dict(C=X), E.ERR_ALIAS), (dict(C=Q + 100), E.ERR_ALIAS), (dict(C=S), E.ERR_ALIAS), (dict(C=T), E.ERR_ALIAS),
        (dict(M=BIG), E.ERR_EXTENT), (dict(K=BIG, lda=BIG, ldb=BIG), E.ERR_EXTENT),
        (dict(M=BIG - 1024, N=BIG - 1024, ldc=BIG, K=0, lda=1, ldb=1, C=8), E.ERR_EXTENT), (dict(M=0), E.OK), (dict(N=0), E.OK),
        (dict(M=0, A=None, B=None, C=None), E.OK)]),
    (sg.sgemm_mi355_fp8_gemm_experts, EXPERTS, [
        (dict(type=3), E.ERR_TYPE), (dict(experts=0), E.ERR_DIM), (dict(rows=-1), E.ERR_DIM), (dict(strideB=-1), E.ERR_STRIDE),
        (dict(stride_sb=-1), E.ERR_STRIDE), (dict(offsets=None), E.ERR_NULL), (dict(offsets=O + 2), E.ERR_ALIGN),
        (dict(offsets=C), E.ERR_ALIAS), (dict(C=Q + 2 * 6080), E.ERR_ALIAS), (dict(C=C + 1), E.ERR_ALIGN), (dict(lda=1), E.ERR_LD),
        (dict(sb_rows=2), E.ERR_OP), (dict(experts=BIG, N=4000, ldc=4000, strideB=0, stride_sb=0), E.ERR_EXTENT), (dict(rows=0), E.OK), (dict(N=0), E.OK)]),
    (sg.sgemm_mi355_fp8_gemm_experts_wgrad, WGRAD, [
        (dict(type=3), E.ERR_TYPE), (dict(experts=0), E.ERR_DIM), (dict(rows=-1), E.ERR_DIM), (dict(lda=639), E.ERR_LD),
        (dict(ldb=639), E.ERR_LD), (dict(ldc=19), E.ERR_LD), (dict(strideC=199), E.ERR_STRIDE), (dict(strideC=-1), E.ERR_STRIDE),
        (dict(C=X), E.ERR_ALIAS), (dict(offsets=C + 400), E.ERR_ALIAS), (dict(A=None), E.ERR_NULL), (dict(M=0), E.OK),
        (dict(rows=BIG - 1024, experts=BIG // 128), E.ERR_EXTENT)]),
]


@pytest.mark.parametrize("fn,good,bad,code", [(f, g, b, c) for f, g, cases in BAD for b, c in cases],
                         ids=lambda v: getattr(v, "__name__", None) or (str(v) if isinstance(v, int) else None))
def test_fp8_refusals(fn, good, bad, code):
    assert call(fn, good, **bad) == code


ROUTE = dict(type=0, tokens=10, experts=64, logits=X, ld=64, bias=None, score=0, groups=8, top_groups=4, choices=8, renorm=1,
             scale=1.0, weights=S, ids=I, stream=0)
BACK = dict(type=0, tokens=10, experts=64, logits=X, ld=64, ids=I, dweights=S, score=1, choices=8, renorm=1, scale=1.0,
            dlogits=C, ldd=64, stream=0)
PLAN = dict(tokens=300, choices=8, experts=64, ids=I, offsets=O, row_token=X, place=S, workspace=T, bytes=520, stream=0)
COMBINE = dict(type=1, tokens=10, choices=8, rows=80, cols=100, Z=X, ldz=100, place=I, weights=S, Y=C, ldy=100, stream=0)
COMBACK = dict(type=1, tokens=10, choices=8, rows=80, cols=100, dY=X, lddy=100, Z=Q, ldz=100, place=I, weights=S, dZ=C, lddz=100,
               dweights=T, stream=0)
BAD_ROUTE = [
    (sg.sgemm_mi355_route, ROUTE, [
        (dict(type=3), E.ERR_TYPE), (dict(score=2), E.ERR_OP), (dict(tokens=-1), E.ERR_DIM), (dict(experts=0), E.ERR_DIM),
        (dict(choices=-1), E.ERR_DIM), (dict(experts=1025, ld=1025), E.ERR_ROUTE), (dict(choices=33), E.ERR_ROUTE),
        (dict(groups=0), E.ERR_ROUTE), (dict(groups=7), E.ERR_ROUTE), (dict(groups=128), E.ERR_ROUTE),
        (dict(top_groups=0), E.ERR_ROUTE), (dict(top_groups=9), E.ERR_ROUTE), (dict(top_groups=1, choices=9), E.ERR_ROUTE),
        (dict(ld=63), E.ERR_LD), (dict(logits=None), E.ERR_NULL), (dict(weights=None), E.ERR_NULL), (dict(ids=None), E.ERR_NULL),
        (dict(logits=X + 1), E.ERR_ALIGN), (dict(bias=T + 2), E.ERR_ALIGN), (dict(ids=S), E.ERR_ALIAS), (dict(weights=X), E.ERR_ALIAS),
        (dict(tokens=BIG), E.ERR_EXTENT), (dict(tokens=0), E.OK), (dict(choices=0), E.OK)]),
    (sg.sgemm_mi355_route_backward, BACK, [
        (dict(type=3), E.ERR_TYPE), (dict(score=-1), E.ERR_OP), (dict(experts=0), E.ERR_DIM), (dict(ldd=63), E.ERR_LD),
        (dict(ld=63), E.ERR_LD), (dict(dlogits=None), E.ERR_NULL), (dict(ids=None), E.ERR_NULL), (dict(dlogits=X), E.ERR_ALIAS),
        (dict(dweights=S + 2), E.ERR_ALIGN), (dict(tokens=0), E.OK)]),
    (sg.sgemm_mi355_route_plan, PLAN, [
        (dict(tokens=-1), E.ERR_DIM), (dict(experts=0), E.ERR_DIM), (dict(experts=1025), E.ERR_ROUTE), (dict(ids=None), E.ERR_NULL),
        (dict(offsets=None), E.ERR_NULL), (dict(place=None), E.ERR_NULL), (dict(workspace=None), E.ERR_NULL),
        (dict(bytes=519), E.ERR_WORKSPACE), (dict(workspace=None, bytes=0), E.ERR_WORKSPACE), (dict(workspace=O), E.ERR_ALIAS),
        (dict(place=I), E.ERR_ALIAS), (dict(offsets=O + 2), E.ERR_ALIGN), (dict(tokens=BIG // 8), E.ERR_EXTENT)]),
    (sg.sgemm_mi355_route_combine, COMBINE, [
        (dict(type=3), E.ERR_TYPE), (dict(choices=-1), E.ERR_DIM), (dict(rows=-1), E.ERR_DIM), (dict(ldz=99), E.ERR_LD),
        (dict(ldy=99), E.ERR_LD), (dict(Z=None), E.ERR_NULL), (dict(Y=None), E.ERR_NULL), (dict(Y=X), E.ERR_ALIAS),
        (dict(Z=X + 1), E.ERR_ALIGN), (dict(tokens=BIG), E.ERR_EXTENT), (dict(tokens=0), E.OK), (dict(cols=0), E.OK)]),
    (sg.sgemm_mi355_route_combine_backward, COMBACK, [
        (dict(type=3), E.ERR_TYPE), (dict(cols=-1), E.ERR_DIM), (dict(lddy=99), E.ERR_LD), (dict(lddz=99), E.ERR_LD),
        (dict(dZ=None), E.ERR_NULL), (dict(dweights=None), E.ERR_NULL), (dict(dZ=Q), E.ERR_ALIAS), (dict(dweights=S), E.ERR_ALIAS),
        (dict(dweights=T + 1), E.ERR_ALIGN), (dict(tokens=0), E.OK), (dict(choices=0), E.OK)]),
]


@pytest.mark.parametrize("fn,good,bad,code", [(f, g, b, c) for f, g, cases in BAD_ROUTE for b, c in cases],
                         ids=lambda v: getattr(v, "__name__", None) or (str(v) if isinstance(v, int) else None))
def test_route_refusals(fn, good, bad, code):
    assert call(fn, good, **bad) == code


def test_messages_and_workspace():
    for code in (sg.ERR_TYPE, sg.ERR_ROUTE):
        assert sg.strerror(code) != sg.strerror(12345)
    size = sg.sgemm_mi355_route_plan_workspace_size
    assert size(10, 8, 64) == 0 and size(2048, 1, 64) == 0 and size(2049, 1, 64) == 2 * 260 and size(0, 8, 64) == 0
    assert size(-1, 8, 64) == 0 and size(1, 8, 1025) == 0


def test_wrappers_refuse_tensors_of_the_host_and_of_other_types():
    x, q, s = torch.zeros(4, 256), torch.zeros(4, 256).to(torch.float8_e4m3fn), torch.ones(4, 2)
    off, ids = torch.zeros(2, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32)
    for bad in (lambda: sg.quantize_fp8(x), lambda: sg.quantize_fp8_cols(x), lambda: sg.gemm_fp8(q, s, q, s),
                lambda: sg.gemm_fp8_experts(q, s, q[None], s[None], off), lambda: sg.gemm_fp8_experts_wgrad(q, s, q, s, off),
                lambda: sg.route(x, 2), lambda: sg.route_backward(x, ids, s), lambda: sg.route_plan(ids, 4),
                lambda: sg.route_combine(x, ids, s), lambda: sg.route_combine_backward(x, x, ids, s)):
        with pytest.raises(TypeError):
            bad()


def test_wrappers_refuse_shapes():
    q, s, off = torch.zeros(4, 256).to(torch.float8_e4m3fn), torch.ones(4, 2), torch.zeros(2, dtype=torch.int32)
    for bad in (lambda: sg.gemm_fp8(q, s, q[:, :128], s), lambda: sg.gemm_fp8(q[0], s, q, s),
                lambda: sg.gemm_fp8_experts(q, s, q, s, off), lambda: sg.gemm_fp8_experts(q, s, q[None], s, off),
                lambda: sg.gemm_fp8_experts(q, s, q[None, :, :128], s[None], off),
                lambda: sg.route_plan(off, 4)):
        with pytest.raises(ValueError):
            bad()


def test_the_tables_of_these_tests():
    """The 64-bit helpers against torch's conversions on the CPU."""
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(50000, generator=g) * 100, torch.arange(7200) / 16.0, torch.arange(64) * 2.0 ** -11])
    np.testing.assert_array_equal(R.encode(x.numpy()), x.clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy())
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    np.testing.assert_array_equal(R.bytes_of(every), every.float().numpy())
    w, ids, s = R.route(np.array([[0.0, 2.0, 2.0, 1.0]], np.float32), 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, 0.5) and np.isclose(s.sum(), 1.0)
    # a planted mistake in the oracle's choice (the higher index on a tie) is seen
    assert ids.tolist() != [[2, 1]]
    off, tok, place = R.plan(np.array([[1, 0], [0, 5], [1, -1]]), 2)
    assert off.tolist() == [0, 2, 4] and tok.tolist() == [0, 1, 0, 2, 1, 2] and place.tolist() == [[2, 0], [1, 4], [3, 5]]
