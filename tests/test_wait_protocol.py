"""A timed-out kernel ends (no GPU): what the sources must not do around a barrier of a group of warps.

bar.sync has no time limit.  A warp that leaves its group's loop on the CTA's abort flag, read after the
barrier, may see a flag that another role set after the group's other warps had read it: those go on to a
barrier that is never complete.  So the decision has to come out of the barrier itself (named_bar_any).
"""
import glob
import os
import re

import pytest

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "video_dit_full_b200", "csrc", "*.cu")))


def code(path):
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_warp_leaves_its_group_by_a_flag_of_its_own(path):
    after = re.findall(r"named_bar_sync\([^;]*;\s*if\s*\(\s*\*?\s*abort_flag[^;]*?\)\s*(break|return|continue|goto)", code(path))
    assert not after


def test_packed_forward_decides_in_the_barrier():
    text = code(os.path.join(ROOT, "video_dit_full_b200", "csrc", "attn_varlen_fwd.cu"))
    assert len(re.findall(r"if \(named_bar_any\(1 \+ t, BM, \*abort_flag != 0\)\) break;", text)) == 2
    # a vote of the whole warp stands behind no condition that its lanes read for themselves
    assert not re.search(r"!\s*\*abort_flag\s*&&\s*wait_(item|warp)", text)
