"""The root of AdamW's 8-bit states (csrc/root.h) on the host: every significand of
either parity, from every approximation of the reciprocal root that is off by an
ulp at most, is rounded correctly, but for one (no GPU needed; what the hardware
gives for that one is tested on it)."""

import os
import shutil
import subprocess

import pytest

import moe_grouped_mlp_amd as m

CSRC = os.path.join(os.path.dirname(m.__file__), "csrc")
# The root is taken of v in [1, 4): in the range it is for, other exponents change
# no significand.  Correctly rounded roots in double and then in float are correctly
# rounded in float (53 >= 2 * 24 + 2 bits).
PROGRAM = r"""
#define __host__
#define __device__
#include "root.h"
#include <cmath>
#include <cstdio>
#include <cstring>
int main() {
  long tried = 0;
  for (float v = 1.0f; v < 4.0f; v = std::nextafterf(v, 8.0f)) {
    const double exact = 1.0 / std::sqrt(static_cast<double>(v));
    const float near = static_cast<float>(exact), want = static_cast<float>(std::sqrt(static_cast<double>(v)));
    const float ys[] = {std::nextafterf(near, 0.0f), near, std::nextafterf(near, 8.0f)};
    const double ulp = static_cast<double>(ys[2]) - near;
    for (float y : ys) {
      if (std::fabs(y - exact) > 1.001 * ulp) continue;
      ++tried;
      unsigned bits;
      std::memcpy(&bits, &v, 4);
      if (moe::root_from(v, y) != want) std::printf("%x %d ", bits, (y > near) - (y < near));
    }
  }
  std::printf("%ld\n", tried);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ missing")
def test_every_significand(tmp_path):
    src, exe = tmp_path / "root.cpp", tmp_path / "root"
    src.write_text(PROGRAM)
    fast = ["-mfma"] if " fma " in open("/proc/cpuinfo").read() else []   # (else fmaf is the library's)
    subprocess.run(["g++", "-O2", "-ffp-contract=off", *fast, f"-I{CSRC}", "-o", str(exe), str(src)], check=True)
    *wrong, tried = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert wrong == ["406e9372", "1"] and int(tried) > 2 * 2 ** 24
