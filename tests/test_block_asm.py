"""The wait states of the gated block's kernels in the gfx950 assembly that hipcc generates: around the inline-assembly MFMAs
(rules R1 to R3) and before memory instructions that read a scalar register which a vector instruction wrote (R4)."""
import concurrent.futures as cf
import shutil

import pytest

import waitstates
from test_grouped_descriptors import check_r4
from test_grouped_waitstates import _assembly, check_r3

SOURCES = ["grouped_tile_%s.hip" % n for n in ("glu_bf16", "gludx_bf16", "glu_f32")]


def test_generated_kernels_keep_the_wait_states(tmp_path):
    if shutil.which("hipcc") is None:
        pytest.skip("no hipcc")
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        texts = list(ex.map(lambda s: _assembly(str(tmp_path), s), SOURCES))
    kernels = loads = 0
    for src, txt in zip(SOURCES, texts):
        for name, items in waitstates.functions(txt).items():
            if not any(not isinstance(i, str) and i.is_mfma for i in items):
                continue
            kernels += 1
            assert waitstates.check(items) == [], (src, name)
            assert check_r3(items) == [], (src, name)
            bad = check_r4(items)
            assert bad == [], (src, name, len(bad), bad[:3])
            loads += sum(not isinstance(i, str) and i.op.startswith("buffer_load") for i in items)
    assert kernels >= 9 and loads > 300
