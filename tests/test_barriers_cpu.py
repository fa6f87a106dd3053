"""Every barrier of the built kernels is reached with the wave's own LDS operations done.

The compiler has left out the wait before a barrier at the head of a loop, where only the loop's end had LDS operations
on the way: the counts of many runs in route_plan were then read before the last of them had been added."""
from __future__ import annotations

import os
import shutil

import pytest

import dense_fp32_matrix_02_amd as sg
from tests import _isa

LOOP = """
\ts_mov_b32 s0, 0 // 000000000100: 00000000
\ts_barrier // 000000000104: 00000000
\tds_add_u32 v0, v1 // 000000000108: 00000000
\ts_cbranch_scc1 65532 // 000000000110: 00000000 <f+0x4>
\ts_waitcnt lgkmcnt(0) // 000000000114: 00000000
\ts_barrier // 000000000118: 00000000
\ts_endpgm // 00000000011C: 00000000
"""


def body_of(text):
    out = []
    for line in text.strip().splitlines():
        code, rest = line.strip().split(" // ")
        op, _, operands = code.partition(" ")
        out.append((int(rest.split(":")[0], 16), op, operands, 0x104 if "<f+0x4>" in rest else None))
    return out


def test_the_reader_sees_a_missing_wait():
    assert _isa.open_barriers(body_of(LOOP)) == (2, [0x104])
    mended = LOOP.replace("\ts_cbranch_scc1", "\ts_waitcnt lgkmcnt(0) // 00000000010C: 00000000\n\ts_cbranch_scc1")
    assert _isa.open_barriers(body_of(mended)) == (2, [])


def test_no_barrier_is_reached_with_lds_operations_on_the_way(tmp_path):
    if not os.path.exists(sg.LIB_PATH):
        from dense_fp32_matrix_02_amd import build
        build.build()
    if not shutil.which(_isa.OBJDUMP):
        pytest.skip("needs the ROCm llvm-objdump")
    functions, barriers, found = 0, 0, []
    for path in _isa.code_objects(sg.LIB_PATH, str(tmp_path)):
        for name, body in _isa.functions(path):
            if any(op == "s_barrier" for _, op, _, _ in body):
                n, open_ = _isa.open_barriers(body)
                functions, barriers = functions + 1, barriers + n
                found += [(name, hex(a)) for a in open_]
    assert functions > 300 and barriers > 1500  # the reader has seen the kernels
    assert not found, found
