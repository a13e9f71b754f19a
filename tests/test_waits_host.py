"""Checks (no GPU) that no role of a kernel can wait without a limit: after another role of its CTA
has given up, every wait has to end, so that the kernel returns its status."""
import glob
import os
import re

import pytest

from exact_attention_forward_fa_gb300 import _build


def code(path):
    """The file without its comments."""
    text = open(path).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


FILES = sorted(glob.glob(os.path.join(_build.CSRC, "*.cu*")))


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_no_barriers_by_name(path):
    """A named barrier has no limit: a warp that gives up ahead of one leaves its siblings there.  (The form that
    votes, `red`, lets all of them leave together: each brings to it whether it has given up.)"""
    assert not re.findall(r"(?<![a-z])(?:barrier|bar)(?:\.cta)?\.(?:sync|arrive)", code(path))


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_phases_are_polled_in_one_place(path):
    """mbarrier phases are awaited through the bounded waits alone."""
    if os.path.basename(path) != "fa_device.cuh":
        assert not re.findall(r"mbarrier\.(?:try|test)_wait", code(path))


@pytest.mark.parametrize("path", [p for p in FILES if "WaitCtx" in code(p) and os.path.basename(p) != "fa_device.cuh"],
                         ids=os.path.basename)
def test_roles_meet_outside_their_branches(path):
    """Kernels with roles meet as a whole block before and after the roles' branches alone: at the indentation of the
    kernel's own statements."""
    for line in code(path).splitlines():
        if "__syncthreads()" in line and "regs_" not in line:
            assert len(line) - len(line.lstrip()) <= 8, line


def test_statistics_are_read_as_written_data():
    """The masked dK/dV kernel may begin while the kernel that writes ws_l and ws_d runs: it reads them with plain loads
    behind its wait (the read-only path is for data that nobody writes meanwhile)."""
    text = code(os.path.join(_build.CSRC, "fa_bwd_kernel.cuh"))
    kernel = text[text.index("fa_bwd_dkdv_kernel("):]
    reads = re.findall(r"(\w+(?:<\w+>)?)\(\s*\(?(?:lse4|dd4|a\.ws_[ld]|lane < 8 \? a\.ws_l)", kernel)
    assert len(reads) >= 4 and set(reads) == {"ws_load<kMask>"}, reads
    body = text[text.index("T ws_load("):]
    assert re.match(r"T ws_load\(const T \*p\) \{\s*if constexpr \(kMask\) return \*p;", body)
