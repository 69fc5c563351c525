"""The three-instruction quotient by six of the 4-bit group scale (fp4.cuh, `sixth`), compiled from its own source
with g++ and compared with the IEEE division: a stride through all positive finite fp32 values whose quotient is
normal. No GPU."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "fp8_mixed_precision_saturating_gb300", "csrc", "fp4.cuh")


def test_sixth_rounds_as_the_division(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    body = re.search(r"float sixth\(float a\) \{.*?\n\}", open(SRC).read(), re.S).group(0)
    prog = tmp_path / "sixth.cpp"
    prog.write_text("""
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
static float __fmul_rn(float a, float b) { return a * b; }
static float __fmaf_rn(float a, float b, float c) { return std::fmaf(a, b, c); }
static %s
int main() {
  long bad = 0, n = 0;
  for (uint64_t b = 0x00800000u * 4u; b < 0x7F800000u; b += 127) {
    uint32_t u = static_cast<uint32_t>(b);
    float a;
    std::memcpy(&a, &u, 4);
    volatile float want = a / 6.0f;
    if (want >= 1.17549435e-38f) {
      ++n;
      bad += sixth(a) != want;
    }
  }
  std::printf("%%ld %%ld", n, bad);
}
""" % body)
    exe = tmp_path / "sixth"
    subprocess.run([cxx, "-O2", "-ffp-contract=off", "-o", str(exe), str(prog)], check=True)
    n, bad = map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    assert n > 10 ** 7 and bad == 0
