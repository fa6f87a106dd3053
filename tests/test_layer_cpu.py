"""Refusals of the norm, activation and epilogue calls: codes come from the host before any HIP call, and what the
wrappers refuse, with tensors that say they are on a GPU (no GPU needed)."""
from __future__ import annotations

import contextlib
import os

import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from dense_fp32_matrix_02_amd import _fp8, _layer
from tests.test_wrappers_cpu import E4M3, FAR, _Stream, call_with, gpu

BIG = 2 ** 31 - 1
# Fake, never-dereferenced device addresses, far apart.
X, R, W, H, A, Y, Q, S, D, G, O, P, C = (0x10_0000_0000 * (i + 1) for i in range(13))


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(sg.LIB_PATH):
        from dense_fp32_matrix_02_amd import build
        build.build()
    return sg.load()


@pytest.fixture(autouse=True)
def no_allocation(monkeypatch):
    """Outputs without memory, on no stream."""
    for module in (_fp8, _layer):
        monkeypatch.setattr(module, "_empty", lambda shape, dtype, device, stream, strides=None: gpu(shape, dtype, strides))


NORM = dict(type=1, rows=10, cols=300, X=X, ldx=300, R=R, ldr=300, W=W, w_type=0, eps=1e-6, H=H, ldh=300, rstd=A, Y=Y, ldy=300,
            Q=Q, ldq=304, S=S, s_row=1, s_block=10, stream=0)
BACK = dict(type=1, rows=100, cols=300, dY=Y, lddy=300, H=H, ldh=300, rstd=A, W=W, w_type=1, dH=D, lddh=300, dX=X, lddx=300, dW=G,
            workspace=O, bytes=25 * 1200, stream=0)
GATED = dict(type=2, act=2, rows=10, cols=300, H=H, ldh=600, Z=Y, ldz=300, Q=Q, ldq=304, S=S, s_row=1, s_block=10, stream=0)
GBACK = dict(type=0, act=1, rows=10, cols=300, dZ=D, lddz=300, H=H, ldh=600, dH=G, lddh=600, stream=0)
EBACK = dict(type=0, act=3, rows=1000, cols=300, dC=C, lddc=300, P=P, ldp=300, dP=D, lddp=300, dbias=G, workspace=O, bytes=32 * 1200,
             stream=0)
EPILOGUE = dict(type=1, M=10, N=20, K=300, A=X, lda=304, SA=S, sa_row=1, sa_block=10, B=Q, ldb=304, SB=W, sb_row=1, sb_block=20,
                sb_rows=1, bias=G, act=2, residual=R, ldr=20, P=P, ldp=20, C=C, ldc=20, stream=0)

BAD = [
    (sg.sgemm_mi355_rms_norm, NORM, [
        (dict(type=3), sg.ERR_TYPE), (dict(w_type=2), sg.ERR_TYPE), (dict(rows=-1), sg.ERR_DIM), (dict(cols=0), sg.ERR_DIM),
        (dict(cols=-5), sg.ERR_DIM), (dict(cols=16385, ldx=BIG, ldr=BIG, ldh=BIG, ldy=BIG, ldq=BIG), sg.ERR_EXTENT),
        (dict(rows=BIG), sg.ERR_EXTENT), (dict(eps=-1e-6), sg.ERR_OP), (dict(eps=float("nan")), sg.ERR_OP),
        (dict(eps=float("inf")), sg.ERR_OP), (dict(ldx=299), sg.ERR_LD), (dict(ldr=299), sg.ERR_LD), (dict(ldh=299), sg.ERR_LD),
        (dict(ldy=299), sg.ERR_LD), (dict(ldq=299), sg.ERR_LD), (dict(Q=None), sg.ERR_NULL), (dict(S=None), sg.ERR_NULL),
        (dict(X=None), sg.ERR_NULL), (dict(W=None), sg.ERR_NULL), (dict(X=None, H=None), sg.ERR_NULL),
        (dict(s_row=-1), sg.ERR_STRIDE), (dict(s_row=0), sg.ERR_STRIDE), (dict(s_block=9), sg.ERR_STRIDE),
        (dict(X=X + 1), sg.ERR_ALIGN), (dict(W=W + 2), sg.ERR_ALIGN), (dict(rstd=A + 2), sg.ERR_ALIGN), (dict(H=X + 2), sg.ERR_ALIAS),
        (dict(H=X, ldh=301), sg.ERR_ALIAS), (dict(H=R, ldh=301), sg.ERR_ALIAS), (dict(Y=X), sg.ERR_ALIAS), (dict(Y=H), sg.ERR_ALIAS),
        (dict(Q=R), sg.ERR_ALIAS), (dict(S=W), sg.ERR_ALIAS), (dict(rstd=S), sg.ERR_ALIAS), (dict(rows=0), sg.OK),
        (dict(rows=0, Q=None), sg.ERR_NULL), (dict(H=None, rstd=None, Y=None, Q=None, S=None), sg.ERR_NULL)]),
    (sg.sgemm_mi355_rms_norm_backward, BACK, [
        (dict(type=-1), sg.ERR_TYPE), (dict(w_type=2), sg.ERR_TYPE), (dict(cols=0), sg.ERR_DIM), (dict(rows=-1), sg.ERR_DIM),
        (dict(cols=16385, lddy=BIG, ldh=BIG, lddh=BIG, lddx=BIG), sg.ERR_EXTENT), (dict(lddy=299), sg.ERR_LD),
        (dict(ldh=299), sg.ERR_LD), (dict(lddh=299), sg.ERR_LD), (dict(lddx=299), sg.ERR_LD), (dict(dY=None), sg.ERR_NULL),
        (dict(rstd=None), sg.ERR_NULL), (dict(dX=None), sg.ERR_NULL), (dict(workspace=None), sg.ERR_NULL),
        (dict(bytes=25 * 1200 - 1), sg.ERR_WORKSPACE), (dict(workspace=None, bytes=0), sg.ERR_WORKSPACE),
        (dict(workspace=O + 2), sg.ERR_ALIGN), (dict(workspace=D), sg.ERR_ALIAS), (dict(dX=H), sg.ERR_ALIAS),
        (dict(dX=Y, lddx=301), sg.ERR_ALIAS), (dict(dX=D, lddx=301), sg.ERR_ALIAS), (dict(dW=W), sg.ERR_ALIAS), (dict(rows=0), sg.OK)]),
    (sg.sgemm_mi355_gated, GATED, [
        (dict(type=3), sg.ERR_TYPE), (dict(act=5), sg.ERR_OP), (dict(act=-1), sg.ERR_OP), (dict(rows=-1), sg.ERR_DIM),
        (dict(cols=-1), sg.ERR_DIM), (dict(ldh=599), sg.ERR_LD), (dict(ldz=299), sg.ERR_LD), (dict(ldq=299), sg.ERR_LD),
        (dict(cols=1 << 30, ldh=BIG, ldz=BIG, ldq=BIG), sg.ERR_EXTENT), (dict(rows=BIG), sg.ERR_EXTENT),
        (dict(rows=1 << 28, s_block=1 << 28), sg.ERR_EXTENT), (dict(H=None), sg.ERR_NULL), (dict(Q=None), sg.ERR_NULL),
        (dict(S=None), sg.ERR_NULL), (dict(H=H + 1), sg.ERR_ALIGN), (dict(Z=H), sg.ERR_ALIAS), (dict(Q=H), sg.ERR_ALIAS),
        (dict(s_block=1), sg.ERR_STRIDE), (dict(rows=0), sg.OK), (dict(cols=0), sg.OK), (dict(Q=None, S=None, Z=None), sg.ERR_NULL)]),
    (sg.sgemm_mi355_gated_backward, GBACK, [
        (dict(type=4), sg.ERR_TYPE), (dict(act=9), sg.ERR_OP), (dict(rows=-1), sg.ERR_DIM), (dict(lddz=1), sg.ERR_LD),
        (dict(ldh=599), sg.ERR_LD), (dict(lddh=599), sg.ERR_LD), (dict(dZ=None), sg.ERR_NULL), (dict(dH=None), sg.ERR_NULL),
        (dict(dH=H), sg.ERR_ALIAS), (dict(dH=D), sg.ERR_ALIAS), (dict(dZ=D + 2), sg.ERR_ALIGN), (dict(rows=1 << 27, cols=300), sg.ERR_EXTENT),
        (dict(rows=0), sg.OK), (dict(cols=0), sg.OK)]),
    (sg.sgemm_mi355_epilogue_backward, EBACK, [
        (dict(type=3), sg.ERR_TYPE), (dict(act=5), sg.ERR_OP), (dict(cols=-1), sg.ERR_DIM), (dict(lddc=1), sg.ERR_LD),
        (dict(ldp=1), sg.ERR_LD), (dict(lddp=1), sg.ERR_LD), (dict(P=None), sg.ERR_NULL), (dict(dP=None), sg.ERR_NULL),
        (dict(dP=P), sg.ERR_ALIAS), (dict(dP=C), sg.ERR_ALIAS), (dict(dbias=P), sg.ERR_ALIAS), (dict(dbias=G + 1), sg.ERR_ALIGN),
        (dict(bytes=32 * 1200 - 1), sg.ERR_WORKSPACE), (dict(workspace=None), sg.ERR_NULL), (dict(workspace=D), sg.ERR_ALIAS),
        (dict(rows=BIG), sg.ERR_EXTENT), (dict(rows=1, cols=1 << 28, lddc=BIG, ldp=BIG, lddp=BIG), sg.ERR_EXTENT), (dict(rows=0), sg.OK),
        (dict(cols=0), sg.OK)]),
    (sg.sgemm_mi355_fp8_gemm_epilogue, EPILOGUE, [
        (dict(type=3), sg.ERR_TYPE), (dict(act=5), sg.ERR_OP), (dict(act=-1), sg.ERR_OP), (dict(sb_rows=2), sg.ERR_OP),
        (dict(M=-1), sg.ERR_DIM), (dict(K=-1), sg.ERR_DIM), (dict(lda=299), sg.ERR_LD), (dict(ldc=19), sg.ERR_LD), (dict(ldr=19), sg.ERR_LD),
        (dict(ldp=19), sg.ERR_LD), (dict(A=None), sg.ERR_NULL), (dict(C=None), sg.ERR_NULL), (dict(bias=G + 2), sg.ERR_ALIGN),
        (dict(residual=R + 1), sg.ERR_ALIGN), (dict(residual=C + 2), sg.ERR_ALIAS), (dict(residual=C, ldr=21), sg.ERR_ALIAS),
        (dict(P=C), sg.ERR_ALIAS), (dict(P=R), sg.ERR_ALIAS), (dict(C=G), sg.ERR_ALIAS), (dict(C=X), sg.ERR_ALIAS),
        (dict(sa_row=-1), sg.ERR_STRIDE), (dict(M=BIG), sg.ERR_EXTENT), (dict(M=0), sg.OK), (dict(N=0), sg.OK)]),
]


@pytest.mark.parametrize("fn,good,bad,code", [(f, g, b, c) for f, g, cases in BAD for b, c in cases],
                         ids=lambda v: getattr(v, "__name__", None) or (str(v) if isinstance(v, int) else None))
def test_refusals(fn, good, bad, code):
    assert fn(*dict(good, **bad).values()) == code


def test_workspaces():
    norm, epilogue = sg.sgemm_mi355_rms_norm_backward_workspace_size, sg.sgemm_mi355_epilogue_backward_workspace_size
    assert norm(4, 300) == 0 and norm(100, 300) == 25 * 300 * 4 and norm(2, 3000) == 2 * 3000 * 4 and norm(0, 300) == 0 and norm(10, 0) == 0 and norm(10, 16385) == 0
    assert norm(BIG - 2000, 16384) <= 2048 * 16384 * 4
    assert epilogue(32, 300) == 0 and epilogue(33, 300) == 2 * 300 * 4 and epilogue(0, 3) == 0 and epilogue(3, 0) == 0
    assert epilogue(64, 100) == 0 and epilogue(65, 100) == 2 * 100 * 4 and 0 < epilogue(BIG - 2000, 8192) <= 2048 * 8192 * 4


def bytes_(rows, cols):
    return gpu((rows, cols), E4M3)


TOGETHER = [  # the call and the number of its tensors
    (lambda t: sg.rms_norm_fp8(t((2, 8)), t((8,)), residual=t((2, 8)), H=t((2, 8)), stream=_Stream()), 4),
    (lambda t: sg.rms_norm(t((2, 8)), t((8,)), residual=t((2, 8)), stream=_Stream()), 3),
    (lambda t: sg.rms_norm_backward(t((2, 8)), t((2, 8)), t((2,)), t((8,)), dH=t((2, 8)), stream=_Stream()), 5),
    (lambda t: sg.gated_fp8(t((2, 8)), stream=_Stream()), 1),
    (lambda t: sg.gated(t((2, 8)), stream=_Stream()), 1),
    (lambda t: sg.gated_backward(t((2, 4)), t((2, 8)), stream=_Stream()), 2),
    (lambda t: sg.gemm_fp8_epilogue(t((2, 300), E4M3), t((2, 3)), t((4, 300), E4M3), t((4, 3)), t((2, 4)), bias=t((4,)),
                                    residual=t((2, 4)), stream=_Stream()), 7),
    (lambda t: sg.epilogue_backward(t((2, 8)), t((2, 8)), activation="silu", stream=_Stream()), 2),
]


@pytest.mark.parametrize("fn,far", [(fn, far) for fn, count in TOGETHER for far in range(count)],
                         ids=[f"{i}-{far}" for i, (fn, count) in enumerate(TOGETHER) for far in range(count)])
def test_tensors_and_stream_have_to_be_on_one_gpu(fn, far):
    with pytest.raises(ValueError, match="GPU 1"):
        call_with(fn, far)
    with pytest.raises(sg.SgemmError):  # all together: the C call is reached, and refuses tensors without memory
        call_with(fn, None)


def gemm(A=(2, 300), SA=(2, 3), B=(4, 300), SB=(4, 3), **more):
    return sg.gemm_fp8_epilogue(bytes_(*A), gpu(SA), bytes_(*B), gpu(SB), stream=_Stream(), **more)


REFUSED = [
    lambda: sg.rms_norm_fp8(gpu((2, 8)), gpu((9,))), lambda: sg.rms_norm_fp8(gpu((2, 8)), gpu((1, 8))),
    lambda: sg.rms_norm_fp8(gpu((2, 8)), gpu((8,), strides=(2,))), lambda: sg.rms_norm_fp8(gpu((2, 8)), gpu((8,)), residual=gpu((2, 9))),
    lambda: sg.rms_norm_fp8(gpu((2, 8)), gpu((8,)), H=gpu((2, 8))), lambda: sg.rms_norm_fp8(gpu((2, 8), strides=(8, 2)), gpu((8,))),
    lambda: sg.rms_norm_fp8(gpu((2, 8), strides=(FAR, 1)), gpu((8,))), lambda: sg.rms_norm(gpu((8,)), gpu((8,))),
    lambda: sg.rms_norm(gpu((2, 8)), gpu((8,)), residual=gpu((2, 8)), H=gpu((3, 8))), lambda: sg.rms_norm(gpu((FAR, 8)), gpu((8,))),
    lambda: sg.rms_norm_backward(gpu((2, 9)), gpu((2, 8)), gpu((2,)), gpu((8,))),
    lambda: sg.rms_norm_backward(gpu((2, 8)), gpu((2, 8)), gpu((3,)), gpu((8,))),
    lambda: sg.rms_norm_backward(gpu((2, 8)), gpu((2, 8)), gpu((2,)), gpu((7,))),
    lambda: sg.rms_norm_backward(gpu((2, 8)), gpu((2, 8)), gpu((2,)), gpu((8,)), dH=gpu((2, 7))),
    lambda: sg.gated_fp8(gpu((2, 7))), lambda: sg.gated_fp8(gpu((2, 8)), activation="tanh"), lambda: sg.gated(gpu((2, 8, 1))),
    lambda: sg.gated(gpu((2, 8), strides=(FAR, 1))), lambda: sg.gated_backward(gpu((2, 8)), gpu((2, 8))),
    lambda: sg.gated_backward(gpu((2, 4), strides=(1, 2)), gpu((2, 8))),
    lambda: sg.epilogue_backward(gpu((2, 8)), gpu((2, 9))), lambda: sg.epilogue_backward(gpu((2, 8)), gpu((2, 8)), activation="swish"),
    lambda: sg.epilogue_backward(gpu((2, 8), strides=(4, 1)), gpu((2, 8))),
    lambda: gemm(B=(4, 301)), lambda: gemm(SA=(2, 4)), lambda: gemm(bias=gpu((5,))), lambda: gemm(residual=gpu((2, 5), torch.bfloat16)),
    lambda: gemm(C=gpu((3, 4))), lambda: gemm(activation="swiglu"), lambda: gemm(SB=(5, 4, 3)),
]


@pytest.mark.parametrize("call", REFUSED, ids=range(len(REFUSED)))
def test_shapes_strides_and_names_are_refused(call):
    with pytest.raises(ValueError):
        call()


OTHER_TYPES = [
    lambda: sg.rms_norm_fp8(torch.zeros(2, 8), torch.ones(8)), lambda: sg.gated(torch.zeros(2, 8)),
    lambda: sg.gated_fp8(gpu((2, 8), torch.float64)), lambda: sg.rms_norm(gpu((2, 8)), gpu((8,)), residual=gpu((2, 8), torch.bfloat16)),
    lambda: sg.rms_norm(gpu((2, 8)), gpu((8,), torch.float64)), lambda: sg.rms_norm(gpu((2, 8)), torch.ones(8)),
    lambda: sg.rms_norm_backward(gpu((2, 8), torch.float16), gpu((2, 8)), gpu((2,)), gpu((8,))),
    lambda: sg.rms_norm_backward(gpu((2, 8)), gpu((2, 8)), gpu((2,), torch.float64), gpu((8,))),
    lambda: sg.epilogue_backward(gpu((2, 8), torch.float16), gpu((2, 8))), lambda: sg.gated_backward(torch.zeros(2, 4), gpu((2, 8))),
    lambda: gemm(bias=gpu((4,), torch.bfloat16)), lambda: gemm(residual=gpu((2, 4)), dtype=torch.bfloat16),
]


@pytest.mark.parametrize("call", OTHER_TYPES, ids=range(len(OTHER_TYPES)))
def test_other_types_are_refused(call):
    with pytest.raises(TypeError):
        call()


def test_weights_of_another_16_bit_type_are_refused():
    with pytest.raises(sg.SgemmError) as e:
        sg.rms_norm(gpu((2, 8), torch.bfloat16), gpu((8,), torch.float16), stream=_Stream())
    assert e.value.code == sg.ERR_TYPE


@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_with_their_tensors_gpu_as_the_current_one(monkeypatch, current):
    now = [current]

    @contextlib.contextmanager
    def device(i):
        was, now[0] = now[0], i
        yield
        now[0] = was

    monkeypatch.setattr(_layer, "_several", [True])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    assert _layer._launch(lambda *a: (now[0], a), 0, 5, 6) == (0, (5, 6)) and now == [current]
