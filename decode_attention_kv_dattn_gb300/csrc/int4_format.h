// The 4-bit cache format (DATTN_KV_INT4): what a group of 64 dims of an entry is
// stored as, and where.
//
// A group keeps its least value and a step, both bf16, and a code 0..15 a dim:
//   step = bf16((most - least) / 15), code = rint((x - least) / step), ties to even,
// x - least being rounded to fp32 (which holds it unless the two are 2^15 apart in size:
// then a value that is nothing beside the least one may meet a tie that it misses by
// that nothing). A code stands for least + code * step. The entries are bf16, so the least value is
// exact, and an asymmetric grid spends no code outside the group's own range (a
// key's dims may lie far from zero all on one side). A step below 2^-100 is stored as
// 0 (its inverse stays a normal number; the codes are then 0, off by 15 steps at the
// most). A group with a NaN, an infinity or a range past fp32 is stored as NaN: it
// poisons what reads it, as the entry itself would have.
//
// Sixteen tokens of one (page, KV head) are a block of 9 D bytes, 4.5 bits a value:
// 8 D bytes of codes, then the tokens' D / 64 pairs (least, step) each. A block is one
// bulk copy, and its codes lie in the order of the MMA fragments they become, so a
// lane reads its share with 16-byte loads and no lane exchanges anything:
//   K (scores, A = K, 16 keys x 16 dims): sections of 128 dims x 16 tokens x 64 bytes;
//     16 bytes of a token hold dims 16 t .. 16 t + 15 (t = lane % 4) of the section's
//     first group, then of its second, the even dim in a byte's low half;
//   V (outputs, A = V^T, 16 dims x 16 keys): groups of 64 dims x 512 bytes, 16 bytes a
//     lane (g = lane / 4, t = lane % 4): dims 8 g .. 8 g + 7 of tokens 2 t, 2 t + 1, then of
//     2 t + 8, 2 t + 9; a 32-bit word holds 4 dims of the even token in its low half and
//     of the odd one in its high half (a key pair of a B16 fragment register is then a
//     mask away). Two bytes never hold two tokens, so a token is written without
//     reading its neighbours.
// Plain C++ apart from the qualifiers, so that the host test suite builds it too.
#pragma once

#include <stdint.h>

#include "bf16_exact.h"  // DATTN_HD, f32_mul, f32_fma

namespace dattn {

constexpr int kInt4Group = 64;  // dims that share a least value and a step
constexpr int kInt4Block = 16;  // tokens of a block

// Bytes of a block of one KV head.
DATTN_HD constexpr int int4_block_bytes(int D) { return 9 * D; }
// Byte offsets in a block: the 4 bytes of dims 8 w .. 8 w + 7 of token r's key, the 2 bytes of
// dims 4 w .. 4 w + 3 of its value, and its pair of group G.
DATTN_HD constexpr int int4_key_word(int r, int w) {
  return (w >> 4) * 1024 + r * 64 + ((w & 7) >> 1) * 16 + ((w >> 3) & 1) * 8 + (w & 1) * 4;
}
DATTN_HD constexpr int int4_value_half(int r, int w) {
  return (w >> 4) * 512 + (((w & 15) >> 1) * 4 + ((r & 7) >> 1)) * 16 + (r >> 3) * 8 + (w & 1) * 4 + (r & 1) * 2;
}
DATTN_HD constexpr int int4_pair(int D, int r, int G) { return 8 * D + (r * (D / kInt4Group) + G) * 4; }

struct Int4Grid {
  float least, step, inv;  // inv = about 1 / step, or 0 where the step is
  uint32_t pair;           // as stored: least in the low half, step in the high half
  uint32_t keep;           // ~0, or 0 for a group stored as NaN (its codes are 0)
};

DATTN_HD uint32_t int4_bf16_bits(float x) {  // nearest bf16 of a finite x, ties to even
#if defined(__CUDA_ARCH__)
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.f), "f"(x));
  return r;
#endif
  const uint32_t b = f32_bits(x);
  return (b + 0x7fffu + ((b >> 16) & 1u)) >> 16;
}

// The grid of a group with values between least and most (bf16 values; NaN in either
// for a group that holds one).
DATTN_HD Int4Grid int4_grid(float least, float most) {
  Int4Grid q;
  const float range = f32_add(most, -least);
  const bool ok = range <= 3.402823466e38f;  // false for NaN and infinity
  // range / 15, correctly rounded: a product with the rounded 1/15 and one correction
  const float c = 1.f / 15.f;
  const float y = f32_mul(range, c);
  const float w = f32_fma(f32_fma(-y, 15.f, range), c, y);
  uint32_t s = int4_bf16_bits(w);
  if (!ok || w < 0x1p-100f) s = 0u;
  q.step = f32_of(s << 16);
  q.least = least;
  q.keep = ok ? 0xffffffffu : 0u;
#if defined(__CUDA_ARCH__)
  float x;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(q.step));
  q.inv = s ? x : 0.f;
#else
  q.inv = s ? 1.f / q.step : 0.f;
#endif
  q.pair = (ok ? f32_bits(least) >> 16 : 0x7fc0u) | (s << 16);
  return q;
}

// The code of x in the low 4 bits of the result, whose other bits are those of
// kInt4Bias: the quotient correctly rounded, then rounded to a whole number by the
// add. y is off by 2 units at the most, its remainder is exact (a step has 8 bits),
// and the correction by it, which the error of inv touches 2^22 times smaller, gives a
// tie of the exact quotient as it is.
constexpr uint32_t kInt4Bias = 0x4b400000u;  // 1.5 * 2^23
DATTN_HD uint32_t int4_code_biased(float x, const Int4Grid& q) {
  const float d = f32_add(x, -q.least);
  const float y = f32_mul(d, q.inv);
  const float z = f32_fma(f32_fma(-y, q.step, d), q.inv, y);
  return f32_bits(f32_add(z, 12582912.f));
}
DATTN_HD uint32_t int4_code(float x, const Int4Grid& q) { return (int4_code_biased(x, q) & 15u) & q.keep; }

}  // namespace dattn
