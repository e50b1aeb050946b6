"""A timed-out kernel ends (no GPU): what the sources must not do around a barrier of a group of warps.

bar.sync has no time limit.  A warp that leaves its group's loop on the CTA's abort flag, read after the
barrier, may see a flag that another role set after the group's other warps had read it: those go on to a
barrier that is never complete.  So the decision has to come out of the barrier itself (named_bar_any).
"""
import glob
import os
import re
import subprocess

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


def test_join_never_passes_its_workspace(tmp_path):
    """Whatever the count of parts in the workspace, the join walks between one part and as many as there is room for."""
    from video_dit_full_b200 import build
    text = code(os.path.join(ROOT, "video_dit_full_b200", "csrc", "attn_varlen_fwd.cu"))
    join = text[text.index("varlen_join_kernel(const VarlenFwdParams"):]
    assert "parts = parts_to_join(p.parts[token], p.most_parts);" in join and join[:join.index("\n}\n")].count("p.parts[") == 1
    src = tmp_path / "parts.cu"
    src.write_text("""#include <cstdio>
#include "varlen.cuh"
int main() {
    int stored, most;
    while (std::scanf("%d %d", &stored, &most) == 2) std::printf("%d\\n", wan::varlen::parts_to_join(stored, most));
}
""")
    exe = tmp_path / "parts"
    subprocess.check_call([build.nvcc(), "-std=c++17", *build.ARCH, "-I", build.CSRC, "-I", os.path.join(ROOT, "include"), "-o",
                           str(exe), str(src)])
    pairs = [(s, m) for s in (-2 ** 31, -1, 0, 1, 2, 63, 64, 65, 0x7f7f7f7f, 2 ** 31 - 1) for m in (1, 2, 7, 64)]
    out = subprocess.run([str(exe)], input="\n".join(f"{s} {m}" for s, m in pairs), capture_output=True, text=True, check=True)
    assert [int(a) for a in out.stdout.split()] == [max(1, min(s, m)) for s, m in pairs]
