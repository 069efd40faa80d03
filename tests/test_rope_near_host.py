"""Host check of the 4-bit cache's RoPE angle routine (csrc/rope_angle.h: rope_cos_sin_near)
against the exact cos and sin of its fixed-point phase, in rational arithmetic: the
larger of the two within 0.85 x 2^-24 of its size, the smaller within 1.4 x 2^-24 of its own,
both within 0.5 x 2^-24 with their second terms - what the bounds of a key entry's error
(int4.cuh) are made of.
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
    float c, s, cl, sl;
    dattn::rope_cos_sin_near(static_cast<int64_t>(pos), static_cast<uint64_t>(step), c, s, cl, sl);
    std::printf("%a %a %a %a\n", (double)c, (double)s, (double)c + (double)cl, (double)s + (double)sl);
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
    worst = [Fraction(0)] * 3
    for (p, step), *terms in zip(cases, *(got[i::4] for i in range(4))):
        c, n, c2, n2 = (Fraction(float.fromhex(x)) for x in terms)
        want = exact(p, step)
        big = int(abs(want[1]) > abs(want[0]))
        off = [abs(x - w) / max(abs(w), Fraction(1, 2 ** 80)) for x, w in ((c, want[0]), (n, want[1]), (c2, want[0]), (n2, want[1]))]
        worst = [max(worst[0], off[big]), max(worst[1], off[1 - big]), max(worst[2], off[2], off[3])]
    assert worst[0] <= Fraction(85, 100) / 2 ** 24 and worst[1] <= Fraction(14, 10) / 2 ** 24, [float(x * 2 ** 24) for x in worst]
    assert worst[2] <= Fraction(1, 2) / 2 ** 24, float(worst[2] * 2 ** 24)


def test_the_bound_of_a_turned_value_covers_its_errors(tmp_path):
    """kTurnError from the errors above: |computed - exact| <= kTurnError (|p| + |v|) as fp32 forms that, whatever the
    signs of the roundings, for every ratio of |v| to |p|."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "k.cpp", str(tmp_path / "k")
    src.write_text('#include <cstdio>\n#include "rope_angle.h"\nint main() { std::printf("%a\\n", (double)dattn::kTurnError); }\n')
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", CSRC, str(src), "-o", exe], check=True)
    bound = Fraction(float.fromhex(subprocess.run([exe], capture_output=True, text=True, check=True).stdout))
    u = Fraction(1, 2 ** 24)
    for ec, es in ((Fraction(85, 100) * u, Fraction(14, 10) * u), (Fraction(14, 10) * u, Fraction(85, 100) * u)):
        for v in (Fraction(0), Fraction(1, 2 ** 24), Fraction(1, 2 ** 12), Fraction(1, 16), Fraction(1), Fraction(3), Fraction(2 ** 20)):
            p = Fraction(1)
            xc = p / ((1 - ec) * (1 - u))                  # |x cos| is at most that
            off_p = xc * ((1 + ec) * (1 + u) - 1)          # p from x cos
            # v from p + y s: u |v|; y s from y sin: es |y sin|; |y sin| <= |v| + |x cos| + the error itself
            off = (off_p + u * v + es * (v + xc)) / (1 - es)
            formed = bound * (p + v) * (1 - u) ** 2        # two roundings down
            assert off <= formed, (float(v), float(off / u), float(formed / u))
