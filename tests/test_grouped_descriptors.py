"""Wait states between a vector instruction that writes a scalar register and a memory instruction that reads it, checked on
the gfx950 assembly that hipcc generates for the grouped products.

  R4  no buffer or global memory instruction reads a scalar register (descriptor, base or offset) that a vector
      instruction (v_readfirstlane, v_readlane, a compare, a carry) wrote fewer than 5 wait states earlier, on any path

The compiler inserts these waits for its own instructions, but not for the direct loads to LDS that the tile kernels write
as inline assembly, and a descriptor word passes through a vector register wherever scalar ones are short.
"""
import concurrent.futures as cf
import os
import re
import shutil

import pytest

import waitstates
from test_grouped_waitstates import SOURCES, _assembly

_SREG = re.compile(r"\bs(\d+)\b|\bs\[(\d+):(\d+)\]")
R4_WAITS = 5


def sregs(text: str) -> set:
    out = set()
    for m in _SREG.finditer(text):
        if m.group(1):
            out.add(int(m.group(1)))
        else:
            out.update(range(int(m.group(2)), int(m.group(3)) + 1))
    if re.search(r"\bvcc\b", text):
        out.update(("vcc_lo", "vcc_hi"))
    return out


def valu_sgpr_writes(ins) -> set:
    """Scalar registers that a vector instruction writes: its first operand, or the carry that is its second."""
    if not ins.op.startswith("v_") or not ins.args:
        return set()
    out = sregs(ins.args[0])
    if ("_co_" in ins.op or ins.op.startswith(("v_mad_u64", "v_mad_i64", "v_div_scale"))) and len(ins.args) > 1:
        out |= sregs(ins.args[1])
    return out


def check_r4(items):
    insts, _, pred = waitstates._cfg(items)
    bad = []
    for i, ins in enumerate(insts):
        if not ins.op.startswith(("buffer_", "global_", "scratch_", "flat_")):
            continue
        reads = sregs(" ".join(ins.args))
        if not reads:
            continue
        stack, seen = [(p, 0) for p in pred[i]], set()
        while stack:  # back until the wait states have passed on every path
            j, w = stack.pop()
            if (j, w) in seen or w >= R4_WAITS:
                continue
            seen.add((j, w))
            if valu_sgpr_writes(insts[j]) & reads:
                bad.append((i, ins.text, insts[j].text, w))
                continue
            stack.extend((p, w + insts[j].waits) for p in pred[j])
    return bad


PLANTED = """
kern:
    v_readfirstlane_b32 s42, v117
    s_mov_b32 m0, s46
    v_mfma_i32_16x16x64_i8 a[0:3], v[8:11], v[4:7], a[0:3]
    %s
    buffer_load_dwordx4 v0, s[40:43], 0 offen lds
    s_endpgm
"""
LOOP = """
kern:
    s_nop 7
.LBB0_1:
    buffer_load_dwordx4 v0, s[40:43], 0 offen lds
    s_add_i32 s4, s4, 1
    v_readlane_b32 s40, v3, 7
    s_cbranch_scc1 .LBB0_1
    s_endpgm
"""


@pytest.mark.parametrize("between,bad", [("s_nop 0", 1), ("s_nop 1", 1), ("s_nop 2", 0)])
def test_r4_finds_a_planted_hazard(between, bad):
    assert len(check_r4(waitstates.functions(PLANTED % between)["kern"])) == bad


def test_r4_follows_back_edges_and_ignores_other_registers():
    assert len(check_r4(waitstates.functions(LOOP)["kern"])) == 1
    assert check_r4(waitstates.functions(LOOP.replace("s40, v3", "s44, v3"))["kern"]) == []


def test_generated_kernels_wait_for_descriptors(tmp_path):
    if shutil.which("hipcc") is None:
        pytest.skip("no hipcc")
    sources = SOURCES + ["grouped_decode.hip"]
    with cf.ThreadPoolExecutor(max_workers=len(sources)) as ex:
        texts = list(ex.map(lambda s: _assembly(str(tmp_path), s), sources))
    loads = 0
    for src, txt in zip(sources, texts):
        for name, items in waitstates.functions(txt).items():
            bad = check_r4(items)
            assert bad == [], (src, name, len(bad), bad[:3])
            loads += sum(not isinstance(i, str) and i.op.startswith("buffer_load") for i in items)
    assert loads > 1000
