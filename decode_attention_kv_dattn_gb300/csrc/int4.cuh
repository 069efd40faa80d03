// Device helpers of the 4-bit cache's kernels: a group's extent, its grid and its codes
// (int4_format.h) from packed bf16 values.
#pragma once

#include "common.cuh"
#include "int4_format.h"
#include "mma.cuh"
#include "qk_norm.cuh"
#include "rope_angle.h"
#include "round_f64.h"

namespace dattn {

__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// (largest, -least) of the values packed in w[0..N), as one bf16 pair: the join of
// two such pairs is a maximum.
template <int N>
__device__ __forceinline__ uint32_t extent(const uint32_t (&w)[N]) {
  uint32_t mx = w[0], mn = w[0];
#pragma unroll
  for (int i = 1; i < N; ++i) {
    mx = max2_nan(mx, w[i]);
    mn = min2_nan(mn, w[i]);
  }
  mn ^= 0x80008000u;
  // (the halves of each, beside one another)
  return max2_nan(__byte_perm(mx, mn, 0x5410), __byte_perm(mx, mn, 0x7632));
}
__device__ __forceinline__ Int4Grid grid_of(uint32_t e) { return int4_grid(-bf16_hi(e), bf16_lo(e)); }

// Two floats at a time (the packed fp32 instructions: half the issue slots).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void split(F2 a, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 wide2(uint32_t w) { return f2(bf16_lo(w), bf16_hi(w)); }

// Codes of N values (N / 2 words), the first in the low 4 bits: int4_code_biased of each.
template <int N>
__device__ __forceinline__ uint32_t codes(const uint32_t* w, const Int4Grid& q) {
  const F2 least = f2(-q.least, -q.least), inv = f2(q.inv, q.inv), step = f2(-q.step, -q.step), magic = f2(12582912.f, 12582912.f);
  constexpr uint32_t bias = kInt4Bias * (N == 8 ? 0x11111111u : 0x1111u);
  uint32_t r = 0;
#pragma unroll
  for (int i = N / 2 - 1; i >= 0; --i) {
    const F2 d = add2(wide2(w[i]), least);
    const F2 y = mul2(d, inv);
    const F2 z = add2(fma2(fma2(y, step, d), inv, y), magic);
    float c0, c1;
    split(z, c0, c1);
    r = (r * 16u + __float_as_uint(c1)) * 16u + __float_as_uint(c0);
  }
  return (r - bias) & q.keep;
}

// A key's entry in a 4-bit cache is x c - y s (y c + x s on the other side) with c and s to 64
// bits, rounded to fp32 and then to bf16: a code is a step of the grid, which an entry
// that is off by one of bf16's may change by a whole one, so the entry is that of
// arithmetic in 64 bits. It is formed in fp32 with a bound of its error, and where both
// ends of the bound round alike, that is the entry. The bound is kTurnError of |x c| + |v|,
// and 2^-110 for what underflows.

// Dim d of a key row at pos: with c and s in two fp32 terms and exact products, which decide
// five of six such values at a fifth of the price, or in 64 bits.
__device__ __noinline__ inline uint32_t key_exact(const uint16_t* row, const uint16_t* kn, double inv, int64_t pos, const uint64_t* steps,
                                                  int r, int d) {
  auto at = [&](int x) { return kn ? qk_norm_apply(row[x], kn[x], inv) : row[x]; };
  const uint16_t xb = at(d);
  if (d >= r) return xb;
  const int half = r / 2;
  const bool first = d < half;
  const uint64_t step = steps[first ? d : d - half];
  const float x = bf16_to_f32(xb), y = bf16_to_f32(at(first ? d + half : d - half)) * (first ? -1.f : 1.f);
  {
    float c, s, cl, sl;
    rope_cos_sin_near(pos, step, c, s, cl, sl);
    const float p = f32_mul(x, c), q = f32_mul(y, s), sum = f32_add(p, q), b = f32_add(sum, -p);
    float low = f32_add(f32_add(p, -f32_add(sum, -b)), f32_add(q, -b));  // p + q - sum, exactly
    low = f32_add(low, f32_add(f32_fma(x, c, -p), f32_fma(y, s, -q)));
    low = f32_fma(x, cl, f32_fma(y, sl, low));
    const float e = f32_fma(f32_add(fabsf(p), fabsf(q)), 0x1.1p-25f, 0x1p-110f);
    const uint32_t w = pack_bf16x2(f32_add(sum, f32_add(low, -e)), f32_add(sum, f32_add(low, e)));
    if ((w >> 16) == (w & 0xffffu)) return w & 0xffffu;
  }
  int64_t cq, sq;
  rope_cos_sin_q62(pos, step, cq, sq);
  const double c = static_cast<double>(cq) * 0x1p-62, s = static_cast<double>(sq) * 0x1p-62;
  return pack_bf16x2(static_cast<float>(fma(static_cast<double>(y), s, static_cast<double>(x) * c)), 0.f) & 0xffffu;
}

}  // namespace dattn
