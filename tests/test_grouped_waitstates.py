"""The wait states around the inline-assembly MFMAs of the grouped tile kernels, checked on the gfx950 assembly that hipcc
generates (rules R1 and R2 in waitstates.py; R3 here: no MFMA accumulates onto an AGPR written by a vector instruction
fewer than 2 wait states earlier)."""
import concurrent.futures as cf
import os
import shutil
import subprocess

import pytest

import waitstates

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_layer_token_amd", "csrc")
SOURCES = ["grouped_tile_%s.hip" % n for n in ("y_bf16", "y_i8", "dx_bf16", "dw_bf16", "dwg_bf16", "f32")]


def check_r3(items):
    """Straight-line scan (the accumulators are cleared outside the loops)."""
    bad, recent = [], []
    for it in items:
        if isinstance(it, str):
            continue
        if it.is_mfma:
            acc = waitstates._regs(it.args[3], "a")
            bad += [it.text for regs, age in recent if age < 2 and regs & acc]
        recent = [(regs, age + it.waits) for regs, age in recent if age < 2]
        if it.op.startswith(("v_accvgpr_write", "v_accvgpr_mov")):
            recent.append((waitstates._regs(it.args[0], "a"), 0))
    return bad


def test_r3_finds_a_planted_hazard():
    asm = """
kern:
    v_accvgpr_write_b32 a3, 0
    s_nop 0
    v_mfma_f32_16x16x32_bf16 a[0:3], v[8:11], v[4:7], a[0:3]
    v_accvgpr_write_b32 a4, 0
    s_nop 1
    v_mfma_f32_16x16x32_bf16 a[4:7], v[8:11], v[4:7], a[4:7]
    s_endpgm
"""
    assert len(check_r3(waitstates.functions(asm)["kern"])) == 1


def _assembly(tmp, src):
    from mixture_experts_layer_token_amd import build

    out = os.path.join(tmp, src + ".s")
    r = subprocess.run(["hipcc", "-x", "hip", *build.FLAGS, "-S", "--cuda-device-only", os.path.join(CSRC, src), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return open(out).read()


def test_generated_kernels_keep_the_wait_states(tmp_path):
    if shutil.which("hipcc") is None:
        pytest.skip("no hipcc")
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        texts = list(ex.map(lambda s: _assembly(str(tmp_path), s), SOURCES))
    kernels = 0
    for src, txt in zip(SOURCES, texts):
        for name, items in waitstates.functions(txt).items():
            if not any(not isinstance(i, str) and i.is_mfma for i in items):
                continue
            kernels += 1
            assert waitstates.check(items) == [], (src, name)
            assert check_r3(items) == [], (src, name)
    assert kernels >= 20
