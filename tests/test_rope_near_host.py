"""Host check of the 4-bit cache's RoPE angle routine (csrc/rope_angle.h: rope_cos_sin_near)
against the exact cos and sin of its fixed-point phase, in rational arithmetic: the
larger of the two within 0.85 x 2^-24 of its size, the smaller within 1.4 x 2^-24 of its own -
what the bound of a key entry's error (int4.cuh) is made of.
"""
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from test_rope_angle_host import CSRC, phase_step
from test_rope_q62_host import exact

SHIM = r'''
#include <cstdio>
#include "rope_angle.h"
int main() {
  long long pos;
  unsigned long long step;
  while (std::scanf("%lld %llu", &pos, &step) == 2) {
    float c, s;
    dattn::rope_cos_sin_near(static_cast<int64_t>(pos), static_cast<uint64_t>(step), c, s);
    std::printf("%a %a\n", (double)c, (double)s);
  }
  return 0;
}
'''


def test_against_rational_arithmetic(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    src = tmp_path / "shim.cpp"
    src.write_text(SHIM)
    exe = str(tmp_path / "shim")
    subprocess.run([cxx, "-O2", "-std=c++17", "-ffp-contract=off", "-I", CSRC, str(src), "-o", exe], check=True)
    rng = np.random.default_rng(11)
    cases = [(int(p), phase_step(theta, r, int(rng.integers(0, r // 2)))) for theta in (1e4, 1e6, 5e6) for r in (64, 256)
             for p in rng.integers(0, 2 ** 21, 300)]
    # phases near the quarter turns and the octants' borders, and tiny remainders
    cases += [(1, (q * 2 ** 61 + d) % 2 ** 64) for q in range(8) for e in (0, 1, 5, 20, 31, 40, 55, 60) for d in (-(2 ** e), 2 ** e, 3 * 2 ** e // 2)]
    cases += [(1, int(x)) for x in rng.integers(0, 2 ** 63, 2000)] + [(0, 12345), (-77, phase_step(1e4, 64, 8))]
    text = "\n".join(f"{p} {s}" for p, s in cases)
    got = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
    worst = [Fraction(0), Fraction(0)]
    for (p, s), c, n in zip(cases, got[::2], got[1::2]):
        for g, w in sorted(zip((c, n), exact(p, s)), key=lambda x: abs(x[1]))[::-1][:1]:
            worst[0] = max(worst[0], abs(Fraction(float.fromhex(g)) - w) / abs(w))
        g, w = min(zip((c, n), exact(p, s)), key=lambda x: abs(x[1]))
        if abs(w) > Fraction(1, 2 ** 80):
            worst[1] = max(worst[1], abs(Fraction(float.fromhex(g)) - w) / abs(w))
        else:
            assert abs(float.fromhex(g)) < 2.0 ** -79
    print([float(x * 2 ** 24) for x in worst])
    assert worst[0] <= Fraction(85, 100) / 2 ** 24 and worst[1] <= Fraction(14, 10) / 2 ** 24
