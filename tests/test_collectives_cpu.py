"""Collective instructions (.aligned forms of tensor memory, register splits and cluster barriers)
are for warps whose lanes have met; lanes part wherever one of them arrives at a barrier or
stores alone.  Read from the source: each stands right behind a __syncwarp()."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_attention_photon_gb300", "csrc")
COLLECTIVE = re.compile(r'"(tcgen05\.(?:alloc|dealloc|relinquish_alloc_permit|ld|st|wait::ld|wait::st|cp)'
                        r'|setmaxnreg|barrier\.cluster)\.[^"]*aligned')


def alone(text):
    """Collective instructions whose statement does not follow a __syncwarp()."""
    text = re.sub(r"//[^\n]*", "", text)
    found, missing = 0, []
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        end = text.index(");", m.end())
        hit = COLLECTIVE.search(text[m.start():end])
        if hit:
            found += 1
            if not text[:m.start()].rstrip().endswith("__syncwarp();"):
                missing.append(hit.group(1))
    return found, missing


@pytest.mark.parametrize("path", sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu*"))))
def test_lanes_meet_before_collective_instructions(path):
    with open(os.path.join(CSRC, path)) as f:
        assert alone(f.read())[1] == []


def test_the_reading_finds_them():
    with open(os.path.join(CSRC, "tc_common.cuh")) as f:
        assert alone(f.read())[0] >= 8
    assert alone('x(); asm volatile("tcgen05.ld.sync.aligned.32x32b" : "=r"(r));') == (1, ["tcgen05.ld"])
    assert alone('__syncwarp();   // met\n  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;");') == (1, [])
