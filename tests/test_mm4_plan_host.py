"""How a product of 4-bit operands is run where the device holds few clusters: csrc/mm4_plan.h, compiled with g++. No GPU."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_mixed_precision_saturating_gb300", "csrc")
SIZES = [(65, 128, 64), (128, 4096, 4096), (1536, 1000, 16379), (16384, 14336, 4096), (300, 300, 256), (70, 16, 16384), (4096, 64, 8192)]
# resident pairs with K in 1 to 4 parts, and CTAs in clusters of 1 to 8, in the proportions of 152 SMs
GB300 = ([0, 76, 36, 23, 17], [0, 152, 76, 48, 36, 27, 23, 18, 17])


def plans(tmp_path, cases):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src = tmp_path / "plan.cpp"
    src.write_text("""
#include <cstdio>
#include "mm4_plan.h"
int main() {
  long long M, N, K, sms;
  fp8gb::Mm4Clusters f;
  while (std::scanf("%lld %lld %lld %lld", &M, &N, &K, &sms) == 4) {
    f.pair[0] = f.one[0] = 0;
    for (int i = 1; i < 5; ++i) std::scanf("%d", &f.pair[i]);
    for (int i = 1; i < 9; ++i) std::scanf("%d", &f.one[i]);
    const auto p = M <= 64 ? fp8gb::mm4_plan_few_rows(M, N, K, sms) : fp8gb::mm4_plan(M, N, K, sms, f);
    std::printf("%d %d\\n", p.bn, p.splits);
  }
}
""")
    exe = tmp_path / "plan"
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    text = "\n".join(" ".join(map(str, (*s, sms, *pair[1:], *one[1:]))) for s, sms, pair, one in cases)
    out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split()
    return [tuple(map(int, out[i:i + 2])) for i in range(0, len(out), 2)]


def test_only_clusters_that_are_held(tmp_path):
    """Clusters from some size on are not there: the plan does without them, and there is one."""
    cases = []
    for s in SIZES:
        for most in range(2, 9):  # CTAs of the largest cluster that fits
            pair = [0] + [GB300[0][i] if 2 * i <= most else 0 for i in range(1, 5)]
            one = [0] + [GB300[1][i] if i <= most else 0 for i in range(1, 9)]
            cases.append((s, 152, pair, one))
    for (s, _, pair, one), (bn, splits) in zip(cases, plans(tmp_path, cases)):
        assert splits >= 1 and splits <= -(-s[2] // 256), s
        assert (pair if bn == 0 else one)[splits] > 0, s


def test_without_any_cluster(tmp_path):
    """Single CTAs alone: what fits in one wave of them, else no plan (splits 0), and no division by zero."""
    none = [0] * 5
    assert plans(tmp_path, [((128, 1024, 512), 152, none, [0, 152] + [0] * 7), ((16384, 14336, 4096), 152, none, [0, 152] + [0] * 7)]) == [(128, 1), (0, 0)]


def test_plans_of_the_whole_device(tmp_path):
    """As they were timed: full size unsplit on pairs, few outputs with K in 2, one token on one CTA per SM."""
    got = plans(tmp_path, [(s, 152, *GB300) for s in ((16384, 14336, 4096), (1536, 1000, 16379), (1, 14336, 4096), (23, 6144, 1536))])
    assert got == [(0, 1), (0, 2), (16, 1), (32, 3)]
