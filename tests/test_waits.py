"""Waits that one lane takes for its warp (csrc): the others see what it waited for only
after a barrier of the warp, which a shuffle of its answer is not."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_gemm_tiled_gb300", "csrc")
FILES = sorted(p for p in glob.glob(os.path.join(CSRC, "*.cu*")) if "mbar_wait" in open(p).read())


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_one_lanes_answer_is_shared_behind_a_barrier(path):
    text = re.sub(r"//[^\n]*", "", open(path).read())
    # (no shuffle of a truth value but in that function)
    bare = re.findall(r"__shfl_sync\(0xffffffffu, \w+ \? 1 : 0, 0\)", text)
    assert len(bare) == (1 if path.endswith("common.cuh") else 0)
    # a wait of lane 0 alone is followed by that function
    for m in re.finditer(r"lane == 0[^\n;]*\)\s*\{?[^{};]*= mbar_wait\(", text):
        assert "warp_got(" in text[m.end(): m.end() + 700], text[m.start(): m.end() + 200]


def test_the_answer():
    text = open(os.path.join(CSRC, "common.cuh")).read()
    body = text[text.index("bool warp_got(bool got) {"):]
    body = body[: body.index("}")]
    assert body.index("__syncwarp();") < body.index("__shfl_sync(")


def test_every_box_is_a_group():
    """The 16-bit kernel's boxes take staging buffers in turn and wait until at most one
    group is still read: a box that is not stored (past M or N) counts as one too, and
    waits like the others before it writes its buffer."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "hgemm_tcgen05.cuh")).read())
    stores = list(re.finditer(r"tma_store_3d\([^;]*;", text))
    assert len(stores) == 2
    for m in stores:
        before, after = text[: m.start()], text[m.end():]
        assert re.search(r"if \(lane == 0\) \{\s*if \(here\) $", before), before[-120:]
        assert re.match(r"\s*bulk_commit\(\);\s*\}", after), after[:80]
        wait = before[before.rindex("const bool here"):]
        assert re.search(r"if \(CIN && here\) \{[^}]*c_wait[^}]*\}[^}]*\} else \{\s*wait_staging\(\);", wait)
