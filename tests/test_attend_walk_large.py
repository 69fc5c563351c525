"""The shares of attention's work (csrc/attend_walk.cuh) where the items of a call pass 32 bits, compiled for the CPU and held against
whole numbers of any size: where each CTA's run begins, and which CTA takes an item."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cstdio>
#include "%s"
using namespace fp8gb::attend;
int main() {
  long long total, x;
  int c, ctas;
  while (scanf("%%lld %%lld %%d %%d", &total, &x, &c, &ctas) == 4) printf("%%lld %%d\n", (long long)begin_of(total, c, ctas), cta_of(total, x, ctas));
}
"""


def test_shares_of_more_than_32_bits_of_items(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "w.cpp").write_text(SOURCE % os.path.join(ROOT, "fp8_mixed_precision_saturating_gb300", "csrc", "attend_walk.cuh"))
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover", str(tmp_path / "w.cpp"), "-o", str(tmp_path / "w")], check=True)
    rng = random.Random(1)
    asked = []
    # 4295491584: one sequence of 2^20 new tokens over as many keys, 64 cache heads of 4 query heads each
    for total in [200, 65537, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1, 2 ** 32 + 5, 4295491584, 2 ** 33 + 7, 2 ** 40 - 1, 2 ** 54 - 1]:
        for ctas in (1, 2, 152, 160):
            edges = [total * c // ctas + d for c in range(ctas + 1) for d in (-1, 0, 1)] + [28254540, 2 ** 32 // ctas - 1, 2 ** 32 // ctas, total - 1]
            for x in [e for e in edges if 0 <= e < total] + [rng.randrange(total) for _ in range(20)]:
                asked.append((total, x, rng.randrange(ctas + 1), ctas))
    out = subprocess.run([str(tmp_path / "w")], input="\n".join(" ".join(map(str, a)) for a in asked), capture_output=True, text=True, check=True).stdout.split("\n")
    for (total, x, c, ctas), line in zip(asked, out):
        begin, cta = map(int, line.split())
        assert begin == total * c // ctas
        # the CTA whose run, from total c / ctas to total (c + 1) / ctas, holds item x
        assert total * cta // ctas <= x < total * (cta + 1) // ctas, (total, x, ctas, cta)
