"""Registers that tcgen05.ld fills are pinned behind its wait: the wait names none of them, so without reg_fence the compiler may
use them before it. Every tmem_ld_wait() in the kernels' sources is followed by a reg_fence of each register array that the
loads before it fill."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_mixed_precision_saturating_gb300", "csrc")


def unpinned(text):
    """(line, arrays) of the waits whose loads' registers are not all fenced at once."""
    lines, filled, bad = text.split("\n"), set(), []
    for i, line in enumerate(lines):
        filled |= set(re.findall(r"\btmem_ld\d+\([^;]*,\s*(\w+)\)\s*;", line))
        if "tmem_ld_wait();" in line:
            j, fenced = i + 1, set()
            while (m := re.match(r"\s*reg_fence\((\w+)\);", lines[j])):
                fenced.add(m.group(1))
                j += 1
            if filled - fenced:
                bad.append((i + 1, sorted(filled - fenced)))
            filled = set()
    return bad


def test_every_wait_is_followed_by_its_fences():
    waits = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = open(path).read()
        waits += text.count("tmem_ld_wait();")
        assert not unpinned(text), (os.path.basename(path), unpinned(text))
    assert waits >= 8


def test_the_check_sees_a_missing_fence():
    good = "tmem_ld16(a, r);\ntmem_ld_wait();\nreg_fence(r);\nx"
    assert not unpinned(good) and unpinned(good.replace("reg_fence(r);\n", "")) == [(2, ["r"])]
