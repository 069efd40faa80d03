// RoPE angle: cos and sin of one rotary pair's angle at a position, from a
// 64-bit fixed-point phase and a short fp32 series.
//
// Plain C++ apart from the qualifiers, so that the host test suite can build
// the same function and check it against the exact values.
#pragma once

#include <stdint.h>

#include "bf16_exact.h"  // DATTN_HD, f32_mul, f32_fma

namespace dattn {

// int32 to fp32, rounded to nearest even.
DATTN_HD float f32_of_i32(int32_t x) {
#if defined(__CUDA_ARCH__)
  return __int2float_rn(x);
#else
  return static_cast<float>(x);  // the default rounding mode: to nearest, ties to even
#endif
}

// cos and sin of one RoPE pair's angle at position pos, as fp32 values.
// step = rint(2^64 * inv_freq / 2pi) is the pair's angle per position in
// 64-bit fixed-point turns, so pos * step mod 2^64 is the phase, exactly. Its
// top 32 bits split into a quadrant j (nearest quarter turn) and a remainder
// in [-1/8, 1/8) turn; cos and sin of the remainder t come from their Taylor
// series through t^10 and t^9 in fp32 (coefficients +-1/n!, first omitted
// terms below 2e-9 on [-pi/4, pi/4]) and are turned by j quarter turns. Every
// step is an integer or a correctly rounded fp32 operation (no contraction),
// so the result is the same on any IEEE machine: within 1.5e-7 of the exact
// values for |pos| <= 2^21, and no fp64 work.
DATTN_HD void rope_cos_sin(int64_t pos, uint64_t step, float& c, float& s) {
  const uint64_t phase = static_cast<uint64_t>(pos) * step;
  const uint32_t w = static_cast<uint32_t>(phase >> 32) + (1u << 29);
  const uint32_t quad = w >> 30;
  const int32_t rho = static_cast<int32_t>(w & 0x3fffffffu) - (1 << 29);
  const float t = f32_mul(f32_of_i32(rho), 1.46291807926715968e-09f);  // 2 pi / 2^32
  const float t2 = f32_mul(t, t);
  float sp = f32_fma(t2, 2.75573192e-06f, -1.98412698e-04f);
  sp = f32_fma(t2, sp, 8.33333333e-03f);
  sp = f32_fma(t2, sp, -1.66666667e-01f);
  const float sn = f32_fma(f32_mul(t, t2), sp, t);
  float cp = f32_fma(t2, -2.75573192e-07f, 2.48015873e-05f);
  cp = f32_fma(t2, cp, -1.38888889e-03f);
  cp = f32_fma(t2, cp, 4.16666667e-02f);
  cp = f32_fma(t2, cp, -5.0e-01f);
  const float cs = f32_fma(t2, cp, 1.0f);
  const float a = (quad & 1u) ? sn : cs;  // |cos| of the angle
  const float b = (quad & 1u) ? cs : sn;  // |sin| of the angle
  c = (quad == 1u || quad == 2u) ? -a : a;
  s = (quad >= 2u) ? -b : b;
}

// int64 to fp32, rounded to nearest even.
DATTN_HD float f32_of_i64(int64_t x) {
#if defined(__CUDA_ARCH__)
  return __ll2float_rn(x);
#else
  return static_cast<float>(x);
#endif
}

// cos and sin of the same angle as fp32 values near the nearest: within 0.85 x 2^-24 of
// the one above 0.7 in magnitude, relative, and 1.4 x 2^-24 of the other. The remainder keeps
// its 62 bits as a sum t + tl, the square of t its rounding error, and what is added
// last to t and to 1 - t^2 / 2 is small, so that one rounding remains. cl and sl are what
// that rounding took off: c + cl and s + sl are within 0.5 x 2^-24, relative.
DATTN_HD void rope_cos_sin_near(int64_t pos, uint64_t step, float& c, float& s, float& cl, float& sl) {
  const uint64_t w = static_cast<uint64_t>(pos) * step + (1ull << 61);
  const uint32_t quad = static_cast<uint32_t>(w >> 62);
  const int64_t rho = static_cast<int64_t>(w & 0x3fffffffffffffffull) - (1ll << 61);  // 2^-64 turns
  const float h = f32_of_i64(rho), l = f32_of_i64(rho - static_cast<int64_t>(h));
  const float kh = 6.28318548202514648f * 0x1p-64f, kl = -1.74845553e-07f * 0x1p-64f;  // 2 pi / 2^64
  const float t = f32_mul(h, kh), tl = f32_fma(l, kh, f32_fma(h, kl, f32_fma(h, kh, -t)));
  const float t2 = f32_mul(t, t), t2l = f32_fma(f32_mul(2.0f, t), tl, f32_fma(t, t, -t2));
  float sp = f32_fma(t2, 2.75573192e-06f, -1.98412698e-04f);
  sp = f32_fma(t2, sp, 8.33333333e-03f);
  sp = f32_fma(t2, sp, -1.66666667e-01f);
  const float half = f32_mul(0.5f, t2);
  const float r1 = f32_fma(f32_mul(t, t2), sp, f32_fma(-half, tl, tl));
  const float sn = f32_add(t, r1), snl = f32_add(r1, -f32_add(sn, -t));
  float cp = f32_fma(t2, -2.75573192e-07f, 2.48015873e-05f);
  cp = f32_fma(t2, cp, -1.38888889e-03f);
  cp = f32_fma(t2, cp, 4.16666667e-02f);
  const float a1 = f32_add(1.0f, -half);
  const float e1 = f32_add(f32_add(1.0f, -a1), -half);  // (exact)
  const float r2 = f32_fma(f32_mul(t2, t2), cp, f32_fma(-0.5f, t2l, e1));
  const float cs = f32_add(a1, r2), csl = f32_add(r2, -f32_add(cs, -a1));
  const float a = (quad & 1u) ? sn : cs, al = (quad & 1u) ? snl : csl;
  const float b = (quad & 1u) ? cs : sn, bl = (quad & 1u) ? csl : snl;
  const bool cneg = quad == 1u || quad == 2u, sneg = quad >= 2u;
  c = cneg ? -a : a;
  s = sneg ? -b : b;
  cl = cneg ? -al : al;
  sl = sneg ? -bl : bl;
}
DATTN_HD void rope_cos_sin_near(int64_t pos, uint64_t step, float& c, float& s) {
  float cl, sl;
  rope_cos_sin_near(pos, step, c, s, cl, sl);
}

// How far v = fma(y, s, p), p = x c rounded, with these c and s is from x cos + y sin, as a
// share of |p| + |v|. In units of 2^-24, p is off by 1 and by c's error, y s, which is at
// most |x cos| + |v|, by s's, v by its own rounding: (1 + 0.85 + 1.4) |p| + (1 + 1.4) |v|, and
// 3.25 are not enough where |v| is nothing beside |p|: terms of the second order and the
// roundings of the bound itself come on top.
constexpr float kTurnError = 0x1.a8p-23f;

// Signed product of two Q62 fixed-point numbers (value * 2^62), rounded down.
DATTN_HD int64_t mul_q62(int64_t a, int64_t b) {
#if defined(__CUDA_ARCH__)
  return __mul64hi(a, b) * 4;
#else
  return static_cast<int64_t>((static_cast<__int128>(a) * b) >> 64) * 4;
#endif
}

// cos and sin of the same angle to fp64 accuracy, as Q62 numbers, in integers:
// the remainder t of the phase in [-pi/4, pi/4) and its Taylor series through
// t^18 and t^17 (first omitted terms below 2^-61 and 2^-58). Each product is
// rounded down by less than 2^-60; the results are within 2^-56 of the exact
// values. Used where fp32 is not exact enough; 64-bit integer products cost a
// few instructions, fp64 arithmetic here tens of cycles a step.
DATTN_HD void rope_cos_sin_q62(int64_t pos, uint64_t step, int64_t& c, int64_t& s) {
  const uint64_t w = static_cast<uint64_t>(pos) * step + (1ull << 61);
  const uint32_t quad = static_cast<uint32_t>(w >> 62);
  const int64_t rho = static_cast<int64_t>(w & 0x3fffffffffffffffull) - (1ll << 61);  // 2^-64 turns
  // rho / 2^61 times pi / 4: Q63 x Q63 -> Q62
  const int64_t r63 = static_cast<int64_t>(static_cast<uint64_t>(rho) << 2);
  const int64_t pi4 = 0x6487ed5110b4611all;
#if defined(__CUDA_ARCH__)
  const int64_t t = __mul64hi(r63, pi4);
#else
  const int64_t t = static_cast<int64_t>((static_cast<__int128>(r63) * pi4) >> 64);
#endif
  const int64_t t2 = mul_q62(t, t);
  // 2^62 / n!, alternating in sign
  int64_t p = -720;                          // -1/18!
  p = 220414ll + mul_q62(t2, p);  // 1/16!
  p = -52899477ll + mul_q62(t2, p);  // -1/14!
  p = 9627704831ll + mul_q62(t2, p);  // 1/12!
  p = -1270857037706ll + mul_q62(t2, p);  // -1/10!
  p = 114377133393536ll + mul_q62(t2, p);  // 1/8!
  p = -6405119470038039ll + mul_q62(t2, p);  // -1/6!
  p = 192153584101141163ll + mul_q62(t2, p);  // 1/4!
  p = -2305843009213693952ll + mul_q62(t2, p);  // -1/2!
  const int64_t cs = 4611686018427387904ll + mul_q62(t2, p);
  int64_t q = 12966;                          // 1/17!
  q = -3526632ll + mul_q62(t2, q);  // -1/15!
  q = 740592679ll + mul_q62(t2, q);  // 1/13!
  q = -115532457973ll + mul_q62(t2, q);  // -1/11!
  q = 12708570377060ll + mul_q62(t2, q);  // 1/9!
  q = -915017067148291ll + mul_q62(t2, q);  // -1/7!
  q = 38430716820228233ll + mul_q62(t2, q);  // 1/5!
  q = -768614336404564651ll + mul_q62(t2, q);  // -1/3!
  const int64_t sn = t + mul_q62(t, mul_q62(t2, q));
  const int64_t a = (quad & 1u) ? sn : cs;
  const int64_t b = (quad & 1u) ? cs : sn;
  c = (quad == 1u || quad == 2u) ? -a : a;
  s = (quad >= 2u) ? -b : b;
}

}  // namespace dattn
