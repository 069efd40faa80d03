"""The 4-bit cache's rounding and layout (csrc/int4_format.h, built for the host)
against rational arithmetic and the layout that include/dattn.h describes. No GPU
needed."""
import ctypes
import os
import subprocess
import tempfile
from fractions import Fraction

import numpy as np
import pytest

import int4_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "decode_attention_kv_dattn_gb300", "csrc")

SHIM = r"""
#include "int4_format.h"
extern "C" void quantise(const float* x, unsigned* pair, unsigned char* code, long groups) {
  for (long i = 0; i < groups; ++i) {
    float lo = x[i * 64], hi = lo;
    for (int d = 1; d < 64; ++d) {
      const float v = x[i * 64 + d];
      lo = (v != v || lo != lo) ? v + lo : v < lo ? v : lo;
      hi = (v != v || hi != hi) ? v + hi : v > hi ? v : hi;
    }
    const dattn::Int4Grid q = dattn::int4_grid(lo, hi);
    pair[i] = q.pair;
    for (int d = 0; d < 64; ++d) code[i * 64 + d] = dattn::int4_code(x[i * 64 + d], q);
  }
}
extern "C" int key_word(int r, int w) { return dattn::int4_key_word(r, w); }
extern "C" int value_half(int r, int w) { return dattn::int4_value_half(r, w); }
extern "C" int pair_at(int D, int r, int G) { return dattn::int4_pair(D, r, G); }
"""


@pytest.fixture(scope="module")
def shim():
    d = tempfile.mkdtemp(prefix="dattn_int4_")
    src, lib = os.path.join(d, "shim.cpp"), os.path.join(d, "shim.so")
    open(src, "w").write(SHIM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
    return ctypes.CDLL(lib)


def quantise(shim, x):
    x = np.ascontiguousarray(x, np.float32)
    n = x.size // 64
    pair, code = np.empty(n, np.uint32), np.empty((n, 64), np.uint8)
    shim.quantise(x.ctypes.data_as(ctypes.c_void_p), pair.ctypes.data_as(ctypes.c_void_p),
                  code.ctypes.data_as(ctypes.c_void_p), ctypes.c_long(n))
    return code, (pair & 0xffff).astype(np.uint16), (pair >> 16).astype(np.uint16)


def bf16(x):
    return ref.f64(ref.bf16_bits(x)).astype(np.float32)


def groups(seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((3000, 64))
    x[500:1000] = x[500:1000] * 0.01 + 3.0                       # far from zero
    x[1000:1500] *= 2.0 ** rng.integers(-90, 90, (500, 1))       # every size
    x[1500:2000] *= 2.0 ** rng.integers(-12, 3, (500, 64))       # dims of unlike size
    x[2000:2500] = rng.integers(-30, 30, (500, 64)) / 2          # quotients that are ties
    x[2500:2600] = rng.integers(0, 2, (100, 64))                 # two values
    x[2600:2700] = rng.standard_normal((100, 1))                 # one value
    x[2700:2800, 1:] = 0                                         # one that is not zero
    x[2800] = 0
    return bf16(x.astype(np.float32))


def test_grid_and_codes_are_the_rounded_quotients(shim):
    x = groups(1)
    code, least, step = quantise(shim, x)
    for i in range(len(x)):
        v = [Fraction(float(y)) for y in x[i]]
        lo, width = min(v), (max(v) - min(v)) / 15
        assert Fraction(float(ref.f64(least[i]))) == lo
        s = Fraction(float(ref.f64(step[i])))
        # nearest bf16: no neighbour is nearer
        if width >= Fraction(2) ** -99:
            for other in (int(step[i]) - 1, int(step[i]) + 1):
                assert abs(s - width) <= abs(Fraction(float(ref.f64(other))) - width), i
        for d in range(64):
            want = 0 if s == 0 else min(15, round((v[d] - lo) / s))  # (Fraction rounds ties to even)
            assert code[i, d] == want, (i, d)
        assert code[i].min() == 0 and (s == 0 or code[i].max() == 15)


def test_reference_agrees(shim):
    x = groups(2)
    for got, want in zip(quantise(shim, x), ref.quantise(x.astype(np.float64).reshape(-1, 64))):
        assert np.array_equal(np.asarray(got).reshape(-1), np.asarray(want).reshape(-1))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_group_that_holds_no_number_is_nan(shim, bad):
    x = groups(3)[:64].copy()
    x[np.arange(64), np.arange(64)] = bad
    code, least, step = quantise(shim, x)
    assert (code == 0).all() and (least == 0x7fc0).all() and (step == 0).all()


def test_a_range_past_fp32_is_nan_and_a_tiny_one_is_flat(shim):
    x = np.zeros((3, 64), np.float32)
    x[0, 0], x[0, 1] = 3e38, -3e38
    x[1, 5] = 2.0 ** -98   # step 2^-98 / 15 < 2^-100
    x[2, 5] = 2.0 ** -95
    code, least, step = quantise(shim, bf16(x))
    assert least[0] == 0x7fc0 and step[0] == 0 and (code[0] == 0).all()
    assert least[1] == 0 and step[1] == 0 and (code[1] == 0).all()
    assert step[2] != 0 and code[2, 5] == 15


@pytest.mark.parametrize("D", [128, 256])
def test_layout(shim, D):
    """Every byte of a block holds one thing, and it is where the header says."""
    for side, unit, at in (("k", 8, shim.key_word), ("v", 4, shim.value_half)):
        used = np.zeros(9 * D, int)
        for r in range(16):
            for w in range(D // unit):
                base = at(r, w)
                for i in range(unit // 2):
                    assert base + i == ref.code_byte(side, D, r, w * unit + 2 * i)
                used[base:base + unit // 2] += 1
            for G in range(D // 64):
                p = shim.pair_at(D, r, G)
                assert p == ref.pair_byte(D, r, G)
                used[p:p + 4] += 1
        assert (used == 1).all()
