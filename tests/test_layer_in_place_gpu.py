"""Updates in place that the C calls allow, at rows of any length: H in the place of X or of R, dX in that of dY or of dH, or of
both, the same tensor given twice; against the same calls with matrices of their own."""
from __future__ import annotations

import pytest
import torch

import dense_fp32_matrix_02_amd as sg
from tests import _fp8 as R
from tests import _gpu as G
from tests.test_layer_gpu import matrix

pytestmark = pytest.mark.gpu

TYPE = {"fp32": 0, "bf16": 1, "fp16": 2}
SHAPES = [(70, 7, 2, 1), (33, 100, 0, 0), (5, 513, 3, 0), (9, 1025, 0, 3), (40, 2047, 1, 1), (3, 4097, 0, 0), (3, 8191, 5, 1), (2, 16381, 0, 0),
          (33, 4096, 8, 0), (8200, 4096, 0, 0)]


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    G.require_gpu()


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_norm(kind, rows, cols, pad, offset):
    print(f"[gpu] rms_norm in place {kind} {rows}x{cols}", flush=True)
    w = torch.linspace(0.5, 1.5, cols, device="cuda")
    x, r = matrix(rows, cols, 1, kind, pad, offset), matrix(rows, cols, 2, kind, pad, offset)

    def call(X, residual, H):
        Y, a = torch.empty(rows, cols, dtype=R.TYPES[kind], device="cuda"), torch.empty(rows, device="cuda")
        code = sg.sgemm_mi355_rms_norm(TYPE[kind], rows, cols, X.data_ptr(), cols + pad, None if residual is None else residual.data_ptr(),
                                       cols + pad, w.data_ptr(), 0, 1e-6, H.data_ptr(), cols + pad, a.data_ptr(), Y.data_ptr(), cols, None, 0,
                                       None, 0, 0, stream())
        torch.cuda.synchronize()
        assert code == sg.OK
        return Y, H.clone(), a

    own = matrix(rows, cols, 9, kind, pad, offset)
    for residual, places in ((r, "xr"), (x, "x"), (None, "x")):
        want = call(x, residual, own)
        for place in places:
            X = matrix(rows, cols, 1, kind, pad, offset)
            second = X if residual is x else None if residual is None else matrix(rows, cols, 2, kind, pad, offset)
            got = call(X, second, X if place == "x" else second)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            around = (X if place == "x" else second).as_strided((rows, pad), (cols + pad, 1), offset + cols)
            assert bool(around.isnan().all())


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_norm_backward(kind, rows, cols, pad, offset):
    print(f"[gpu] rms_norm_backward in place {kind} {rows}x{cols}", flush=True)
    w, h = torch.linspace(0.5, 1.5, cols, device="cuda"), matrix(rows, cols, 3, kind, pad, offset)
    a = sg.rms_norm(h, w)[2]
    need = sg.sgemm_mi355_rms_norm_backward_workspace_size(rows, cols)
    room = torch.empty(max(need // 4, 1), device="cuda")

    def call(dY, dH, dX):
        dw = torch.empty(cols, device="cuda")
        code = sg.sgemm_mi355_rms_norm_backward(TYPE[kind], rows, cols, dY.data_ptr(), cols + pad, h.data_ptr(), cols + pad, a.data_ptr(),
                                                w.data_ptr(), 0, None if dH is None else dH.data_ptr(), cols + pad, dX.data_ptr(), cols + pad,
                                                dw.data_ptr(), room.data_ptr(), need, stream())
        torch.cuda.synchronize()
        assert code == sg.OK
        return dX.clone(), dw

    def inputs():
        return matrix(rows, cols, 1, kind, pad, offset), matrix(rows, cols, 2, kind, pad, offset)

    own = matrix(rows, cols, 9, kind, pad, offset)
    dY, dH = inputs()
    want = call(dY, dH, own)
    for place in (0, 1):
        given = inputs()
        got = call(*given, given[place])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert bool(given[place].as_strided((rows, pad), (cols + pad, 1), offset + cols).isnan().all())
    want = call(dY, dY, own)  # one gradient given twice, and updated
    got = call(dY, dY, dY)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dY, _ = inputs()
    want = call(dY, None, own)
    got = call(dY, None, dY)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
