"""Refusals of the 16-bit experts' products: codes come from the host before any HIP call, what the wrappers refuse, and the
choice of kernels (no GPU needed)."""
from __future__ import annotations

import os

import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from dense_fp32_matrix_02_amd import _experts, _fp8
from tests.test_wrappers_cpu import FAR, _Stream, call_with, gpu

BIG = 2 ** 31 - 1
# Fake, never-dereferenced device addresses, far apart.
A, W, O, C = (0x100_0000_0000 * (i + 1) for i in range(4))
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(sg.LIB_PATH):
        from dense_fp32_matrix_02_amd import build
        build.build()
    return sg.load()


@pytest.fixture(autouse=True)
def no_allocation(monkeypatch):
    """Outputs without memory, on no stream."""
    for module in (_fp8, _experts):
        monkeypatch.setattr(module, "_empty", lambda shape, dtype, device, stream, strides=None: gpu(shape, dtype, strides))


FORWARD = dict(type=1, c_type=1, rows=10, N=20, K=30, experts=3, A=A, lda=30, W=W, ldw=30, strideW=600, offsets=O, C=C, ldc=20, stream=0)
DGRAD = dict(FORWARD, lda=20, ldc=30)
WGRAD = dict(type=2, c_type=0, rows=10, N=20, K=30, experts=3, A=A, lda=20, B=W, ldb=30, offsets=O, beta=0.0, C=C, ldc=30, strideC=600,
             stream=0)
EVERY = [(dict(type=0), sg.ERR_TYPE), (dict(type=3), sg.ERR_TYPE), (dict(c_type=3), sg.ERR_TYPE), (dict(rows=-1), sg.ERR_DIM),
         (dict(N=-1), sg.ERR_DIM), (dict(K=-1), sg.ERR_DIM), (dict(experts=0), sg.ERR_DIM), (dict(rows=BIG), sg.ERR_EXTENT),
         (dict(N=1 << 30, lda=BIG, ldc=BIG), sg.ERR_EXTENT), (dict(K=1 << 30, lda=BIG, ldc=BIG), sg.ERR_EXTENT), (dict(lda=19), sg.ERR_LD),
         (dict(ldc=19), sg.ERR_LD), (dict(A=None), sg.ERR_NULL), (dict(C=None), sg.ERR_NULL), (dict(offsets=None), sg.ERR_NULL),
         (dict(A=A + 1), sg.ERR_ALIGN), (dict(offsets=O + 2), sg.ERR_ALIGN), (dict(C=C + 1), sg.ERR_ALIGN), (dict(C=A), sg.ERR_ALIAS),
         (dict(C=W), sg.ERR_ALIAS), (dict(C=O), sg.ERR_ALIAS)]
ROWS = [(dict(ldw=29), sg.ERR_LD), (dict(strideW=-8), sg.ERR_STRIDE), (dict(W=None), sg.ERR_NULL), (dict(W=W + 1), sg.ERR_ALIGN),
        (dict(c_type=2), sg.ERR_TYPE), (dict(rows=0), sg.OK)]


@pytest.mark.parametrize("fn,good,bad,code", [(f, g, b, c) for f, g, more in (
    (sg.sgemm_mi355_experts_gemm, FORWARD, ROWS + [(dict(N=0), sg.OK)]), (sg.sgemm_mi355_experts_gemm_dgrad, DGRAD, ROWS + [(dict(K=0), sg.OK)]),
    (sg.sgemm_mi355_experts_gemm_wgrad, WGRAD, [
        (dict(c_type=1), sg.ERR_TYPE), (dict(ldb=29), sg.ERR_LD), (dict(strideC=599), sg.ERR_STRIDE), (dict(strideC=-600), sg.ERR_STRIDE),
        (dict(B=None), sg.ERR_NULL), (dict(experts=70000, strideC=600), sg.ERR_EXTENT), (dict(N=0), sg.OK), (dict(K=0), sg.OK)]))
    for b, c in EVERY + more], ids=lambda v: getattr(v, "__name__", None) or (str(v) if isinstance(v, int) else None))
def test_refusals(fn, good, bad, code):
    args = dict(good, **bad)
    if "ldw" in args and "ldw" not in bad and ("N" in bad or "K" in bad):
        args["ldw"] = BIG
    if "ldb" in args and "ldb" not in bad and "K" in bad:
        args["ldb"] = BIG
    assert fn(*args.values()) == code


TOGETHER = [  # the call and the number of its tensors
    (lambda t: sg.gemm_experts(t((5, 8), BF), t((2, 4, 8), BF), t((3,), torch.int32), t((5, 4), BF), stream=_Stream()), 4),
    (lambda t: sg.gemm_experts_dgrad(t((5, 4), BF), t((2, 4, 8), BF), t((3,), torch.int32), t((5, 8), BF), stream=_Stream()), 4),
    (lambda t: sg.gemm_experts_wgrad(t((5, 4), BF), t((5, 8), BF), t((3,), torch.int32), t((2, 4, 8)), stream=_Stream()), 4),
]


@pytest.mark.parametrize("fn,far", [(fn, far) for fn, count in TOGETHER for far in range(count)],
                         ids=[f"{i}-{far}" for i, (fn, count) in enumerate(TOGETHER) for far in range(count)])
def test_tensors_and_stream_have_to_be_on_one_gpu(fn, far):
    with pytest.raises(ValueError, match="GPU 1"):
        call_with(fn, far)
    with pytest.raises(sg.SgemmError):  # all together: the C call is reached, and refuses tensors without memory
        call_with(fn, None)


def ints(n):
    return gpu((n,), torch.int32)


def forward(a=(5, 8), w=(2, 4, 8), o=3, kind=BF, w_kind=BF, C=None, **more):
    return sg.gemm_experts(gpu(a, kind), gpu(w, w_kind), ints(o), C, stream=_Stream(), **more)


REFUSED = [lambda: forward(a=(5, 9)), lambda: forward(w=(4, 8)), lambda: forward(w=(0, 4, 8), o=1), lambda: forward(o=4),
           lambda: forward(a=(5, 8, 1)), lambda: forward(C=gpu((5, 5), BF)), lambda: forward(a=(FAR, 8)),
           lambda: sg.gemm_experts(gpu((5, 8), BF, (FAR, 1)), gpu((2, 4, 8), BF), ints(3)),
           lambda: sg.gemm_experts(gpu((5, 8), BF), gpu((2, 4, 8), BF, (32, 1, 4)), ints(3)),
           lambda: sg.gemm_experts_dgrad(gpu((5, 8), BF), gpu((2, 4, 8), BF), ints(3)),
           lambda: sg.gemm_experts_wgrad(gpu((5, 4), BF), gpu((6, 8), BF), ints(3)),
           lambda: sg.gemm_experts_wgrad(gpu((5, 4), BF), gpu((5, 8), BF), ints(1)),
           lambda: sg.gemm_experts_wgrad(gpu((5, 4), BF), gpu((5, 8), BF), ints(3), beta=1.0),
           lambda: sg.gemm_experts_wgrad(gpu((5, 4), BF), gpu((5, 8), BF), ints(3), gpu((2, 8, 4)))]


@pytest.mark.parametrize("call", REFUSED, ids=range(len(REFUSED)))
def test_shapes_and_strides_are_refused(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call", [
    lambda: forward(kind=torch.float64, w_kind=torch.float64), lambda: forward(w_kind=torch.float16), lambda: forward(dtype=torch.float64),
    lambda: sg.gemm_experts(torch.zeros(5, 8), gpu((2, 4, 8)), ints(3)), lambda: sg.gemm_experts(gpu((5, 8), BF), gpu((2, 4, 8), BF), torch.zeros(3)),
    lambda: sg.gemm_experts_wgrad(gpu((5, 4), BF), gpu((5, 8), torch.float16), ints(3))], ids=range(6))
def test_other_types_are_refused(call):
    with pytest.raises(TypeError):
        call()


@pytest.mark.parametrize("call", [lambda: forward(kind=torch.float32, w_kind=torch.float32), lambda: forward(dtype=torch.float16)], ids=range(2))
def test_types_that_the_library_refuses(call):
    with pytest.raises(sg.SgemmError) as e:
        call()
    assert e.value.code == sg.ERR_TYPE


def name(form=0, rows=16384, N=2048, K=4096, experts=32, A=A, lda=None, W=W, ldw=4096, strideW=2048 * 4096):
    return sg.sgemm_mi355_experts_kernel_name(form, rows, N, K, experts, A, lda or (K if form == 0 else N), W, ldw, strideW)


@pytest.mark.parametrize("change,want", [
    (dict(), "tile_256x256"), (dict(rows=64), "rows_16"), (dict(rows=1, experts=1), "rows_16"), (dict(rows=2048), "tile_128x128"),
    (dict(form=1), "tile_256x256"), (dict(form=2), "tile_256x256"), (dict(form=1, rows=64), "tile_128x128"),
    (dict(form=2, N=512, K=512, ldw=512), "tile_128x128"), (dict(A=A + 2), "staged_128x128"), (dict(ldw=4097), "staged_128x128"),
    (dict(strideW=2048 * 4096 + 4), "staged_128x128"), (dict(form=2, strideW=4), "tile_256x256"), (dict(form=2, N=2044, lda=2048), "staged_128x128"),
    (dict(form=1, K=4092), "staged_128x128"), (dict(K=4, lda=8), "staged_128x128"), (dict(rows=64, A=A + 2), "rows_16"),
    (dict(rows=64, K=4, lda=8), "staged_128x128"), (dict(lda=1 << 22), "staged_128x128")])
def test_names(change, want):
    assert name(**change) == want


@pytest.mark.parametrize("bad", [dict(form=3), dict(form=-1), dict(rows=0), dict(rows=-1), dict(N=0), dict(K=0), dict(experts=0), dict(lda=-1),
                                 dict(ldw=0), dict(strideW=-8)])
def test_no_name_where_nothing_runs(bad):
    assert name(**bad) is None


def test_weights_gradients_without_rows_have_a_kernel():
    assert name(form=2, rows=0) == "tile_256x256"  # it sets them to zero


@pytest.mark.parametrize("form", [0, 1, 2])
def test_the_largest_sizes_have_a_name(form):
    assert name(form=form, rows=2**31 - 1, N=2**31 - 1, K=2**31 - 1, experts=2**31 - 1, lda=2**31 - 1, ldw=2**31 - 1) in ("staged_128x128", "rows_16", "rows_32", "rows_64")
