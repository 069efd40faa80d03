"""Host check of the 64-bit RoPE angle routine (csrc/rope_angle.h:
rope_cos_sin_q62) against the exact cos and sin of its fixed-point phase,
worked out in rational arithmetic: within 2^-56, as the routine says (its series
is cut below 2^-58, and each of some ten products is rounded down by less than
2^-60). The kernels that select pages use it where fp32 cannot tell two scores
apart.
"""
import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from test_rope_angle_host import CSRC, phase_step

SHIM = r'''
#include <cstdio>
#include "rope_angle.h"
int main() {
  long long pos;
  unsigned long long step;
  while (std::scanf("%lld %llu", &pos, &step) == 2) {
    int64_t c, s;
    dattn::rope_cos_sin_q62(static_cast<int64_t>(pos), static_cast<uint64_t>(step), c, s);
    std::printf("%lld %lld\n", (long long)c, (long long)s);
  }
  return 0;
}
'''
# pi to 40 digits
PI = Fraction(31415926535897932384626433832795028841971, 10 ** 40)


def exact(pos, step):
    """cos and sin times 2^62 as fractions, off by less than 2^-30."""
    phase = (pos % (1 << 64)) * step % (1 << 64)
    quad, rem = divmod(phase + (1 << 61), 1 << 62)
    t = Fraction(rem - (1 << 61), 1 << 64) * 2 * PI
    t = Fraction(round(t * (1 << 100)), 1 << 100)
    c, s, term = Fraction(0), Fraction(0), Fraction(1)
    for n in range(26):
        if n % 2 == 0:
            c += term * (-1) ** (n // 2)
        else:
            s += term * (-1) ** (n // 2)
        term = Fraction(round(term * t / (n + 1) * (1 << 100)), 1 << 100)
    return [(c, s), (-s, c), (-c, -s), (s, -c)][quad % 4]


def test_against_rational_arithmetic(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    src = tmp_path / "shim.cpp"
    src.write_text(SHIM)
    exe = str(tmp_path / "shim")
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", CSRC, str(src), "-o", exe], check=True)
    rng = np.random.default_rng(7)
    cases = []
    for r, theta in ((64, 5e6), (128, 1e6), (256, 1e4)):
        for i in range(0, r // 2, 5):
            st = phase_step(theta, r, i)
            cases += [(int(p), st) for p in [0, 1, -1, 1 << 20, *rng.integers(-(1 << 31), 1 << 31, 6)]]
    for k in range(4):
        for d in (-3, -1, 0, 1, 3):
            cases += [(1, ((k << 62) + (1 << 61) + d) % (1 << 64)), (1, ((k << 62) + d) % (1 << 64))]
    out = subprocess.run([exe], input="\n".join(f"{p} {s}" for p, s in cases), capture_output=True, text=True, check=True)
    lines = out.stdout.split("\n")
    worst = 0
    for (p, st), line in zip(cases, lines):
        for got, want in zip(line.split(), exact(p, st)):
            worst = max(worst, abs(Fraction(int(got), 1 << 62) - want))
    assert worst <= Fraction(1, 1 << 56), float(worst) * 2.0 ** 56
