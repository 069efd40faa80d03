// A warp's arithmetic over blocks of a 4-bit cache (int4_format.h).
//
// With code c, step s and least value b of a (key k, group G of 64 dims):
//   score    q . K_k = sum_G [ s_kG (q_G . c_kG) + b_kG sum(q_G) ]
//   output   O_d    += sum_k p_k s_kG (c_kd - 8)  +  sum_k p_k (b_kG + 8 s_kG)     (d in G)
// so the codes enter the tensor cores as they are - whole numbers, exact in fp16 -
// and the grid is applied to 4 scores (K) or folded into the weights (V): a group of
// 64 dims costs a few FMAs instead of one for every value. The products are not with
// c0 and c1 of a byte but with c0 and the byte c0 + 16 c1, which one mask or byte permute
// each brings into a half: q0 c0 + q1 c1 = (q0 - q1 / 16) c0 + (q1 / 16) (c0 + 16 c1),
// and the outputs of c1 are taken apart at the end.
//
// Columns of the MMAs: head h's high and low term side by side (2 h, 2 h + 1), so a
// lane's score and output fragments belong to one head (t = lane % 4, and t + 4 with
// NT = 2), and a head's hi + lo is one add without a shuffle.
//
// Precision: that of fp32 sums (0.9 - 1.2e-7 of the outputs' size, against 64 bits).
//  * q's factors and the weights p s enter as two fp16 terms, 22 bits, where fp16 holds
//    them (a dim of q is off by 2^-22 of itself, or 2^-29 of the head's largest where that
//    is more): q is scaled by a power of two that brings the head's largest to 2^18 .. 2^19
//    (2^14 .. 2^15 as a byte's factor, which is a sixteenth), the weights by f_hG, a power of
//    two for each head and group that keeps the largest p s of what has been summed in
//    2^5 .. 2^15. It follows the product, up and down: a key may have a step as large as it
//    likes beside no weight, in one head or in all, and takes no bits from the others'. (With
//    f of the largest step alone, a value 2^24 times the others' size and of no weight cost
//    the outputs 3e-3 of theirs, one of 2^32 all.) The running maximum is a whole number and
//    only moved when a score passes it by 6 (p is at most 2^6), and the products are only
//    looked at where a step times f is above 2^9, which saves the cross-lane maxima of every
//    group of keys.
//  * An MMA lines its products up by the operands' exponents and drops what lies below, and
//    a subnormal operand counts as 2^-14 there, however small. A code masked out of its
//    word is a subnormal, c 2^-24: as it is it costs c0's products 6 bits and the bytes' 2.
//    The keys' bytes can stand that (their factors are a sixteenth of c0's); c0 and the
//    values' operands are made normal numbers by one more operation each (the mask sets
//    the exponent of 1024, which is then taken off): with subnormals alone the outputs were
//    off by 2 - 4e-6.
//  * The values' codes are centred (c - 8): sums of codes 0 .. 15 grow with the context
//    while the outputs do not, and the 7.5 sum(p s) in them, taken off at the end, left
//    errors of 4e-5 over a million tokens.
//  * The MMAs' sums are cut off, not rounded, so long chains shrink: each pair of blocks is
//    summed from zero and added in fp32 (one chain: 7.5e-6 over 262,144 tokens).
// All of it together takes 8 x 262,144 tokens from 198 to 248 us, 64 ragged streams from 42
// to 48, 32 x 16,384 of 24 / 4 heads from 148 to 176 (of it the scales of heads and products
// instead of groups and steps 2). Where a step passes 2^9 / f in most blocks, as with 64
// times the values' size in every second token and little weight there, 13% come on top.
#pragma once

#include "common.cuh"
#include "int4_format.h"
#include "mma.cuh"

namespace dattn {

// The MMAs and the transpose as pure functions, which the compiler may move past one
// another (8 x 262,144 tokens 201 -> 193 us against the volatile ones of mma.cuh).
__device__ __forceinline__ void mma_codes(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_codes_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {  // d = A * B
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t less(uint32_t x, uint32_t y) {  // of fp16 pairs
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ void add4(float (&o)[4], const float (&x)[4]) {  // o += x, two at a time
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    uint64_t a, b;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(o[e]), "f"(o[e + 1]));
    asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(x[e]), "f"(x[e + 1]));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o[e]), "=f"(o[e + 1]) : "l"(a));
  }
}
__device__ __forceinline__ uint32_t scaled(uint32_t x) {  // (x - 1024) 2^-10 of an fp16 pair
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0x14001400u), "r"(0xbc00bc00u));
  return r;
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// q of the 4 NT heads (fp32 [4 NT][D], base-2 scale) as B fragments, and what the
// scores need: sums of q over each group, in the units of the accumulators, and
// the factor from those units to the score, for the lane's score heads.
template <int D, int NT>
__device__ __forceinline__ void int4_query(const float* qs, int lane, uint32_t (&qb)[D / 16][NT][2], float (&qsum)[NT][D / 64],
                                           float (&inv)[NT]) {
  constexpr unsigned full = 0xffffffffu;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float* src = qs + (4 * nt + (g >> 1)) * D;
    float mx = 0.f, sum[D / 64];
#pragma unroll
    for (int G = 0; G < D / 64; ++G) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(src + G * 64 + t * 16 + 4 * i);
        mx = fmaxf(fmaxf(mx, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
        s += (x.x + x.y) + (x.z + x.w);
      }
      s += __shfl_xor_sync(full, s, 1);
      sum[G] = s + __shfl_xor_sync(full, s, 2);
    }
    mx = fmaxf(mx, __shfl_xor_sync(full, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(full, mx, 2));
    // 2^(18 - floor(log2 mx)), 2^100 at the most (a head of zeros)
    const int e = 272 - static_cast<int>(__float_as_uint(mx) >> 23);
    const float S = __uint_as_float(static_cast<uint32_t>(min(max(e, 1), 227)) << 23);
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      // dims i of the word: halves 0 .. 3 and 4 .. 7, bytes (0, 1) and (2, 3) of a half; c0
      // is an operand in units of 2^-10, a byte in units of 2^-24
      const float* x = src + (w >> 1) * 64 + t * 16 + (w & 1) * 8;
      const float4 a = *reinterpret_cast<const float4*>(x), b = *reinterpret_cast<const float4*>(x + 4);
      const float z = S * 0.0625f;
      uint32_t hi, lo;
      split_f16x2(fmaf(a.y, -z, a.x * S) * 0x1p-14f, fmaf(b.y, -z, b.x * S) * 0x1p-14f, hi, lo);
      qb[2 * w][nt][0] = g & 1 ? lo : hi;
      split_f16x2(a.y * z, b.y * z, hi, lo);
      qb[2 * w][nt][1] = g & 1 ? lo : hi;
      split_f16x2(fmaf(a.w, -z, a.z * S) * 0x1p-14f, fmaf(b.w, -z, b.z * S) * 0x1p-14f, hi, lo);
      qb[2 * w + 1][nt][0] = g & 1 ? lo : hi;
      split_f16x2(a.w * z, b.w * z, hi, lo);
      qb[2 * w + 1][nt][1] = g & 1 ? lo : hi;
    }
    // accumulators hold S 2^-24 times q . c
    const float unit = S * 0x1p-24f, back = 0x1p24f / S;
#pragma unroll
    for (int G = 0; G < D / 64; ++G) qsum[nt][G] = __shfl_sync(full, sum[G] * unit, 8 * t);
    inv[nt] = __shfl_sync(full, back, 8 * t);
  }
}

// One warp's running state over the 16-key blocks that it takes.
template <int D, int NT>
struct Int4Warp {
  static constexpr int KS = D / 16, NG = D / 64, MT = D / 16;
  // At 16 m-tiles and two column tiles the outputs alone are 128 registers: q's
  // fragments then stay in shared memory.
  static constexpr bool kSharedQ = D == 256 && NT == 2;
  static constexpr int kQBytes = KS * 256 * NT + 32 * 4 * NT * (NG + 1);  // of one unit's fragments, sums and factors

  uint32_t qb[kSharedQ ? 1 : KS][NT][2];
  float qsum[NT][NG], inv[NT];
  float o[MT][NT][4];
  float m[NT], l[NT], cst[NT][NG];  // base-2 maximum, sum of weights, sum of p (b + 8 s)
  float f[NT][NG];                  // power of two of the weights of the lane's head and group G

  // The fragments into shared memory (kSharedQ), and the warp's own part of them.
  static __device__ __forceinline__ void put_query(const float* qs, uint8_t* dst, int lane) {
    uint32_t q[KS][NT][2];
    float s[NT][NG], v[NT];
    int4_query<D, NT>(qs, lane, q, s, v);
    __syncwarp();  // (dst may be where qs is)
    static_assert(!kSharedQ || NT == 2, "16 bytes of a lane: a k-step's two column tiles");
#pragma unroll
    for (int i = 0; i < KS; ++i)
      *reinterpret_cast<uint4*>(dst + i * 512 + lane * 16) = make_uint4(q[i][0][0], q[i][0][1], q[i][NT - 1][0], q[i][NT - 1][1]);
    float* x = reinterpret_cast<float*>(dst + KS * 256 * NT);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int G = 0; G < NG; ++G) x[(nt * (NG + 1) + G) * 32 + lane] = s[nt][G];
      x[(nt * (NG + 1) + NG) * 32 + lane] = v[nt];
    }
    __syncwarp();
  }
  __device__ __forceinline__ void get_query(const float* qs, const uint8_t* src, int lane) {
    if constexpr (kSharedQ) {
      const float* x = reinterpret_cast<const float*>(src + KS * 256 * NT);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int G = 0; G < NG; ++G) qsum[nt][G] = x[(nt * (NG + 1) + G) * 32 + lane];
        inv[nt] = x[(nt * (NG + 1) + NG) * 32 + lane];
      }
    } else {
      int4_query<D, NT>(qs, lane, qb, qsum, inv);
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = -INFINITY;
      l[nt] = 0.f;
#pragma unroll
      for (int G = 0; G < NG; ++G) {
        cst[nt][G] = 0.f;
        f[nt][G] = 0x1p100f;
      }
    }
  }

  // The steps of keys g and g + 8 of a block's values, groups G and G + 1, and the least values.
  static __device__ __forceinline__ void pairs(const uint8_t* vb, int row, int G, float (&st)[2], float (&ls)[2]) {
    const uint2 p = *reinterpret_cast<const uint2*>(vb + 8 * D + row * (4 * NG) + G * 4);
    st[0] = bf16_hi(p.x), ls[0] = bf16_lo(p.x);
    st[1] = bf16_hi(p.y), ls[1] = bf16_lo(p.y);
  }

  // 2^(e - 127), or 0 where that is no normal number (e < 1).
  static __device__ __forceinline__ float power(int e) { return e > 0 ? __uint_as_float(static_cast<uint32_t>(e) << 23) : 0.f; }

  // A score passed its head's maximum by 6, or a weight p s may pass its scale: both are
  // brought up to date and what was summed so far is rescaled, by powers of two. The
  // maximum's rise by d makes all of the past 2^-d times as large, which f takes back
  // as far as the new keys let it. (Large steps of keys of little weight change nothing.)
  template <int N>
  __device__ __forceinline__ void rescale(const float (&s)[N][NT][2], const uint8_t* vb, int pitch, int g) {
    constexpr unsigned full = 0xffffffffu;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mx = m[nt];
#pragma unroll
      for (int b = 0; b < N; ++b) mx = fmaxf(mx, fmaxf(s[b][nt][0], s[b][nt][1]));
      mx = fmaxf(mx, __shfl_xor_sync(full, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(full, mx, 8));
      mx = ceilf(fmaxf(mx, __shfl_xor_sync(full, mx, 16)));
      const int d = mx == m[nt] ? 0 : static_cast<int>(fminf(mx - m[nt], 1000.f));
      const float fac = power(127 - d);
      m[nt] = mx;
      l[nt] *= fac;
      const float ms = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int G = 0; G < NG; ++G) {
        cst[nt][G] *= fac;
        float x = 0.f;  // the largest p s of the new keys
#pragma unroll
        for (int b = 0; b < N; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            x = fmaxf(x, exp2_fast(s[b][nt][i] - ms) *
                             bf16_hi(*reinterpret_cast<const uint32_t*>(vb + b * pitch + 8 * D + (g + 8 * i) * (4 * NG) + G * 4)));
        x = fmaxf(x, __shfl_xor_sync(full, x, 4));
        x = fmaxf(x, __shfl_xor_sync(full, x, 8));
        x = fmaxf(x, __shfl_xor_sync(full, x, 16));
        // the past's stays where it is, or x f in 2^5 .. 2^6 if that is less
        const int e = static_cast<int>(__float_as_uint(f[nt][G]) >> 23);
        const int en = max(min(min(e + d, 227), x > 0.f ? 259 - static_cast<int>(__float_as_uint(x) >> 23) : 227), 1);
        f[nt][G] = power(en);
        const float r = power(127 + en - e - d);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[G * 4 + j][nt][i] *= r;
      }
    }
  }

  // The values' grids of the keys that do not count, in shared memory: they may hold
  // anything (0 x NaN is NaN). Ends with a warp barrier.
  static __device__ __forceinline__ void clear_rows(uint8_t* vb, uint32_t mask, int lane) {
    for (int i = lane; i < kInt4Block * NG; i += 32)
      if (!((mask >> (i / NG)) & 1u)) *reinterpret_cast<uint32_t*>(vb + 8 * D + i * 4) = 0u;
    fence_proxy_async_smem();  // before the stage is refilled by bulk copies
    __syncwarp();
  }

  // N blocks of 16 keys at once (their chains of products, exponentials and transposes
  // run beside one another): kb, vb are the K and V bytes of the first in shared memory,
  // the others follow; bit r of mask[b] says whether key r of block b counts (one of
  // them does; the others' V grids are zero), qf the unit's fragments with kSharedQ.
  template <int N>
  __device__ __forceinline__ void blocks(const uint8_t* kb, const uint8_t* vb, const uint32_t (&mask)[N], const uint8_t* qf,
                                         int lane) {
    constexpr unsigned full = 0xffffffffu;
    constexpr uint32_t m0 = 0x000f000fu, m1 = 0x00ff00ffu;
    constexpr int pitch = int4_block_bytes(D);
    const int g = lane >> 2, t = lane & 3;
    // ---- scores of keys g and g + 8 of each block for the lane's heads
    float s[N][NT][2];
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[b][nt][0] = s[b][nt][1] = 0.f;
#pragma unroll
    for (int sec = 0; sec < D / 128; ++sec) {
      uint4 xa[N], xb[N];
      uint2 pa[N], pb[N];
#pragma unroll
      for (int b = 0; b < N; ++b) {
        const uint8_t* src = kb + b * pitch;
        xa[b] = *reinterpret_cast<const uint4*>(src + sec * 1024 + g * 64 + t * 16);
        xb[b] = *reinterpret_cast<const uint4*>(src + sec * 1024 + g * 64 + t * 16 + 512);
        pa[b] = *reinterpret_cast<const uint2*>(src + 8 * D + g * (4 * NG) + sec * 8);
        pb[b] = *reinterpret_cast<const uint2*>(src + 8 * D + (g + 8) * (4 * NG) + sec * 8);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int G = sec * 2 + k;
        float acc[N][NT][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int ks = (G * 2 + j) * 2 + i;
            uint32_t q[NT][2];
            if constexpr (kSharedQ) {
              const uint4 v = *reinterpret_cast<const uint4*>(qf + ks * 512 + lane * 16);
              q[0][0] = v.x, q[0][1] = v.y, q[NT - 1][0] = v.z, q[NT - 1][1] = v.w;
            } else {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) q[nt][0] = qb[ks][nt][0], q[nt][1] = qb[ks][nt][1];
            }
#pragma unroll
            for (int b = 0; b < N; ++b) {
              const uint32_t wa = k ? (j ? xa[b].w : xa[b].z) : (j ? xa[b].y : xa[b].x);
              const uint32_t wb = k ? (j ? xb[b].w : xb[b].z) : (j ? xb[b].y : xb[b].x);
              const uint32_t ba = i ? prmt(wa, 0u, 0x4341u) : wa & m1, bb = i ? prmt(wb, 0u, 0x4341u) : wb & m1;
              const uint32_t a[4] = {scaled((ba & m0) | 0x64006400u), scaled((bb & m0) | 0x64006400u), ba, bb};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (j + i == 0) mma_codes_first(acc[b][nt], a, q[nt][0], q[nt][1]);
                else mma_codes(acc[b][nt], a, q[nt][0], q[nt][1]);
              }
            }
          }
        }
#pragma unroll
        for (int b = 0; b < N; ++b) {
          const uint32_t p0 = k ? pa[b].y : pa[b].x, p1 = k ? pb[b].y : pb[b].x;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float(&c)[4] = acc[b][nt];
            s[b][nt][0] = fmaf(bf16_hi(p0), c[0] + c[1], fmaf(bf16_lo(p0), qsum[nt][G], s[b][nt][0]));
            s[b][nt][1] = fmaf(bf16_hi(p1), c[2] + c[3], fmaf(bf16_lo(p1), qsum[nt][G], s[b][nt][1]));
          }
        }
      }
    }
    // ---- do the maximum and the weights' scales still hold?
    float top[NT];  // the lane's largest step, times f
    {
      uint32_t mx[NG];
#pragma unroll
      for (int G = 0; G < NG; ++G) mx[G] = 0u;
#pragma unroll
      for (int b = 0; b < N; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int G = 0; G < NG; G += 2) {
            const uint2 p = *reinterpret_cast<const uint2*>(vb + b * pitch + 8 * D + (g + 8 * i) * (4 * NG) + G * 4);
            // (steps are not negative: the larger pair as a number has the larger step)
            mx[G] = max(mx[G], p.x);
            mx[G + 1] = max(mx[G + 1], p.y);
          }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        top[nt] = 0.f;
#pragma unroll
        for (int G = 0; G < NG; ++G) top[nt] = fmaxf(top[nt], __uint_as_float(mx[G] & 0xffff0000u) * f[nt][G]);
      }
    }
    bool move = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) move = move || top[nt] > 512.f;
#pragma unroll
    for (int b = 0; b < N; ++b) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        s[b][nt][0] *= inv[nt];
        s[b][nt][1] *= inv[nt];
      }
      if (mask[b] != 0xffffu) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (!((mask[b] >> g) & 1u)) s[b][nt][0] = -INFINITY;
          if (!((mask[b] >> (g + 8)) & 1u)) s[b][nt][1] = -INFINITY;
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) move = move || fmaxf(s[b][nt][0], s[b][nt][1]) > m[nt] + 6.f;
    }
    if (__any_sync(full, move)) rescale<N>(s, vb, pitch, g);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float ms = m[nt] == -INFINITY ? 0.f : m[nt];
#pragma unroll
      for (int b = 0; b < N; ++b) {  // (the scores become the weights)
        s[b][nt][0] = exp2_fast(s[b][nt][0] - ms);
        s[b][nt][1] = exp2_fast(s[b][nt][1] - ms);
        l[nt] += s[b][nt][0] + s[b][nt][1];
      }
    }
    // ---- outputs, a group of 64 dims at a time: its weights as B fragments, hi and lo
    // beside one another, then its four m-tiles
#pragma unroll
    for (int G = 0; G < NG; G += 2) {
      float s0[N][2], s1[N][2], l0[N][2], l1[N][2];
#pragma unroll
      for (int b = 0; b < N; ++b) {
        pairs(vb + b * pitch, g, G, s0[b], l0[b]);
        pairs(vb + b * pitch, g + 8, G, s1[b], l1[b]);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t pb[N][NT][2];
        uint4 x[N];
#pragma unroll
        for (int b = 0; b < N; ++b) {
          x[b] = *reinterpret_cast<const uint4*>(vb + b * pitch + (G + k) * 512 + lane * 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float p0 = s[b][nt][0], p1 = s[b][nt][1];
            cst[nt][G + k] = fmaf(p0, fmaf(8.f, s0[b][k], l0[b][k]), fmaf(p1, fmaf(8.f, s1[b][k], l1[b][k]), cst[nt][G + k]));
            uint32_t hi, lo;
            split_f16x2((p0 * s0[b][k]) * f[nt][G + k], (p1 * s1[b][k]) * f[nt][G + k], hi, lo);
            pb[b][nt][0] = transposed(prmt(hi, lo, 0x5410u));
            pb[b][nt][1] = transposed(prmt(hi, lo, 0x7632u));
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float sum[NT][4];
#pragma unroll
            for (int b = 0; b < N; ++b) {
              const uint32_t wa = j ? x[b].y : x[b].x, wb = j ? x[b].w : x[b].z;
              const uint32_t ba = i ? prmt(wa, 0x64646464u, 0x4341u) : (wa & m1) | 0x64006400u;
              const uint32_t bb = i ? prmt(wb, 0x64646464u, 0x4341u) : (wb & m1) | 0x64006400u;
              const uint32_t a[4] = {less((ba & m0) | 0x64006400u, 0x64086408u), less(ba, 0x64886488u),
                                     less((bb & m0) | 0x64006400u, 0x64086408u), less(bb, 0x64886488u)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (b == 0) mma_codes_first(sum[nt], a, pb[b][nt][0], pb[b][nt][1]);
                else mma_codes(sum[nt], a, pb[b][nt][0], pb[b][nt][1]);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) add4(o[(G + k) * 4 + j * 2 + i][nt], sum[nt]);
          }
      }
    }
  }

  // The state: outputs [4 NT][D] relative to m, and m and l of each head.
  __device__ __forceinline__ void finish(float* os, float* ml, int GP, int lane) {
    constexpr unsigned full = 0xffffffffu;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt] += __shfl_xor_sync(full, l[nt], 4);
      l[nt] += __shfl_xor_sync(full, l[nt], 8);
      l[nt] += __shfl_xor_sync(full, l[nt], 16);
      if (g == 0) {
        ml[4 * nt + t] = m[nt];
        ml[GP + 4 * nt + t] = l[nt];
      }
#pragma unroll
      for (int G = 0; G < NG; ++G) {
        float c = cst[nt][G];
        c += __shfl_xor_sync(full, c, 4);
        c += __shfl_xor_sync(full, c, 8);
        c += __shfl_xor_sync(full, c, 16);
        const float back = 1.f / f[nt][G];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float4 v;
          const float(&a)[4] = o[G * 4 + j * 2][nt];
          const float(&b)[4] = o[G * 4 + j * 2 + 1][nt];
          const float a0 = a[0] + a[1], b0 = b[0] + b[1];
          v.x = fmaf(a0, back, c);
          v.y = fmaf(((a[2] + a[3]) - a0) * 0.0625f, back, c);
          v.z = fmaf(b0, back, c);
          v.w = fmaf(((b[2] + b[3]) - b0) * 0.0625f, back, c);
          *reinterpret_cast<float4*>(os + (4 * nt + t) * D + G * 64 + g * 8 + j * 4) = v;
        }
      }
    }
  }
};

}  // namespace dattn
