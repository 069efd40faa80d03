// The streaming warp's arithmetic over a 4-bit cache (int4_format.h), for
// decode_kernel.
//
// With code c, step s and least value b of a (key k, group G of 64 dims):
//   score    q . K_k = sum_G [ s_kG (q_G . c_kG) + b_kG sum(q_G) ]
//   output   O_d    += sum_k p_k s_kG c_kd  +  sum_k p_k b_kG     (d in G)
// so the codes enter the tensor cores as they are - whole numbers, exact in fp16 -
// and the grid is applied to 4 scores (K) or folded into the weights (V): a group of
// 64 dims costs a few FMAs instead of one for every value. A code becomes an fp16
// operand by a mask alone: bits 0-3 of a half are the subnormal c 2^-24, bits 4-7 are
// c 2^-20, and a shift by 8 brings the other two codes there; 5 instructions for 8
// values. The power of two between the two kinds is taken out of q's terms (K) or of
// the finished outputs (V).
//
// Columns of the MMAs: head h's high and low term side by side (2 h, 2 h + 1), so a
// lane's score and output fragments belong to one head (t = lane % 4, and t + 4 with
// NT = 2), and a head's hi + lo is one add without a shuffle.
//
// Precision. q and the weights p s enter as two fp16 terms, 22 bits, where fp16 holds
// them: q is scaled by a power of two that brings the head's largest to 2^10 .. 2^11
// (2^15 for the dims that need the factor 16), the weights by f_G, a power of two that
// follows the largest step seen so far (step f_G in 2^6 .. 2^8), p being at most 2^6:
// the running maximum is only moved when a score passes it by 6, which saves the
// cross-lane maximum of every group of keys. Sums are fp32.
#pragma once

#include "common.cuh"
#include "int4_format.h"
#include "mma.cuh"

namespace dattn {

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
    // 2^(10 - floor(log2 mx)), 2^100 at the most (a head of zeros)
    const int e = 264 - static_cast<int>(__float_as_uint(mx) >> 23);
    const float S = __uint_as_float(static_cast<uint32_t>(min(max(e, 1), 227)) << 23);
    const float S16 = S * 16.f;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      const float* x = src + (w >> 1) * 64 + t * 16 + (w & 1) * 8;
      const float4 a = *reinterpret_cast<const float4*>(x), b = *reinterpret_cast<const float4*>(x + 4);
      uint32_t hi, lo;
      split_f16x2(a.x * S16, b.x * S16, hi, lo);
      qb[2 * w][nt][0] = g & 1 ? lo : hi;
      split_f16x2(a.y * S, b.y * S, hi, lo);
      qb[2 * w][nt][1] = g & 1 ? lo : hi;
      split_f16x2(a.z * S16, b.z * S16, hi, lo);
      qb[2 * w + 1][nt][0] = g & 1 ? lo : hi;
      split_f16x2(a.w * S, b.w * S, hi, lo);
      qb[2 * w + 1][nt][1] = g & 1 ? lo : hi;
    }
    // accumulators hold S 2^-20 times q . c
    const float unit = S * 0x1p-20f, back = 0x1p20f / S;
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
  // fragments then stay in shared memory, written by the helper warp.
  static constexpr bool kSharedQ = D == 256 && NT == 2;
  static constexpr int kQBytes = KS * 512 + 32 * 4 * NT * (NG + 1);  // of one unit's fragments, sums and factors

  uint32_t qb[kSharedQ ? 1 : KS][NT][2];
  float qsum[NT][NG], inv[NT];
  float o[MT][NT][4];
  float m[NT], l[NT], cst[NT][NG];  // base-2 maximum, sum of weights, sum of p b
  float f[NG];                      // power of two of the weights of group G

  // The helper warp's share with kSharedQ, and the streaming warps' with or without.
  static __device__ __forceinline__ void put_query(const float* qs, uint8_t* dst, int lane) {
    uint32_t q[KS][NT][2];
    float s[NT][NG], v[NT];
    int4_query<D, NT>(qs, lane, q, s, v);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      *reinterpret_cast<uint4*>(dst + ks * 512 + lane * 16) = make_uint4(q[ks][0][0], q[ks][0][1], q[ks][NT - 1][0], q[ks][NT - 1][1]);
    float* x = reinterpret_cast<float*>(dst + KS * 512);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int G = 0; G < NG; ++G) x[(nt * (NG + 1) + G) * 32 + lane] = s[nt][G];
      x[(nt * (NG + 1) + NG) * 32 + lane] = v[nt];
    }
  }
  __device__ __forceinline__ void get_query(const float* qs, const uint8_t* src, int lane) {
    if constexpr (kSharedQ) {
      const float* x = reinterpret_cast<const float*>(src + KS * 512);
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
      for (int G = 0; G < NG; ++G) cst[nt][G] = 0.f;
    }
#pragma unroll
    for (int G = 0; G < NG; ++G) f[G] = 0x1p100f;
  }

  // A score passed its head's maximum by 6, or a step its group's scale: both are
  // brought up to date and what was summed so far is rescaled.
  __device__ __forceinline__ void rescale(const float (&s)[NT][2], const float (&st)[2][NG]) {
    constexpr unsigned full = 0xffffffffu;
    float fac[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mx = fmaxf(s[nt][0], s[nt][1]);
      mx = fmaxf(mx, __shfl_xor_sync(full, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(full, mx, 8));
      mx = fmaxf(m[nt], fmaxf(mx, __shfl_xor_sync(full, mx, 16)));
      fac[nt] = mx == -INFINITY ? 1.f : exp2_fast(m[nt] - mx);
      m[nt] = mx;
      l[nt] *= fac[nt];
    }
#pragma unroll
    for (int G = 0; G < NG; ++G) {
      float x = fmaxf(st[0][G], st[1][G]);
      x = fmaxf(x, __shfl_xor_sync(full, x, 4));
      x = fmaxf(x, __shfl_xor_sync(full, x, 8));
      x = fmaxf(x, __shfl_xor_sync(full, x, 16));
      float ratio = 1.f;
      if (x * f[G] > 256.f) {
        // x f in 2^6 .. 2^7
        const int e = 260 - static_cast<int>(__float_as_uint(x) >> 23);
        const float fn = __uint_as_float(static_cast<uint32_t>(min(max(e, 1), 227)) << 23);
        ratio = fn * (1.f / f[G]);
        f[G] = fn;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        cst[nt][G] *= fac[nt];
        const float r = fac[nt] * ratio;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[G * 4 + j][nt][e] *= r;
      }
    }
  }

  // One block of 16 keys: kb, vb are its K and V bytes in shared memory, bit r of mask
  // says whether key r counts (at least one does), qf the unit's fragments with kSharedQ.
  __device__ __forceinline__ void block(const uint8_t* kb, const uint8_t* vb, uint32_t mask, const uint8_t* qf, int lane) {
    constexpr unsigned full = 0xffffffffu;
    constexpr uint32_t m0 = 0x000f000fu, m1 = 0x00f000f0u;
    const int g = lane >> 2, t = lane & 3;
    // ---- scores of keys g and g + 8 for the lane's heads
    float s[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = 0.f;
#pragma unroll
    for (int sec = 0; sec < D / 128; ++sec) {
      const uint4 xa = *reinterpret_cast<const uint4*>(kb + sec * 1024 + g * 64 + t * 16);
      const uint4 xb = *reinterpret_cast<const uint4*>(kb + sec * 1024 + g * 64 + t * 16 + 512);
      const uint2 pa = *reinterpret_cast<const uint2*>(kb + 8 * D + g * (4 * NG) + sec * 8);
      const uint2 pb = *reinterpret_cast<const uint2*>(kb + 8 * D + (g + 8) * (4 * NG) + sec * 8);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int G = sec * 2 + k;
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t wa = k ? (j ? xa.w : xa.z) : (j ? xa.y : xa.x), wb = k ? (j ? xb.w : xb.z) : (j ? xb.y : xb.x);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int ks = (G * 2 + j) * 2 + i;
            const uint32_t a[4] = {wa & m0, wb & m0, wa & m1, wb & m1};
            if constexpr (kSharedQ) {
              const uint4 q = *reinterpret_cast<const uint4*>(qf + ks * 512 + lane * 16);
              mma_f16(acc[0], a, q.x, q.y);
              mma_f16(acc[NT - 1], a, q.z, q.w);
            } else {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], a, qb[ks][nt][0], qb[ks][nt][1]);
            }
            wa >>= 8;
            wb >>= 8;
          }
        }
        const uint32_t p0 = k ? pa.y : pa.x, p1 = k ? pb.y : pb.x;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          s[nt][0] = fmaf(bf16_hi(p0), acc[nt][0] + acc[nt][1], fmaf(bf16_lo(p0), qsum[nt][G], s[nt][0]));
          s[nt][1] = fmaf(bf16_hi(p1), acc[nt][2] + acc[nt][3], fmaf(bf16_lo(p1), qsum[nt][G], s[nt][1]));
        }
      }
    }
    // ---- the values' grids of the same keys; keys that do not count weigh nothing
    const bool on0 = (mask >> g) & 1u, on1 = (mask >> (g + 8)) & 1u;
    float st[2][NG], ls[2][NG], top = 0.f;
#pragma unroll
    for (int G = 0; G < NG; G += 2) {
      uint2 pa = *reinterpret_cast<const uint2*>(vb + 8 * D + g * (4 * NG) + G * 4);
      uint2 pb = *reinterpret_cast<const uint2*>(vb + 8 * D + (g + 8) * (4 * NG) + G * 4);
      if (!on0) pa = make_uint2(0u, 0u);
      if (!on1) pb = make_uint2(0u, 0u);
      st[0][G] = bf16_hi(pa.x), ls[0][G] = bf16_lo(pa.x);
      st[0][G + 1] = bf16_hi(pa.y), ls[0][G + 1] = bf16_lo(pa.y);
      st[1][G] = bf16_hi(pb.x), ls[1][G] = bf16_lo(pb.x);
      st[1][G + 1] = bf16_hi(pb.y), ls[1][G + 1] = bf16_lo(pb.y);
#pragma unroll
      for (int x = G; x < G + 2; ++x) top = fmaxf(top, fmaxf(st[0][x], st[1][x]) * f[x]);
    }
    bool move = top > 256.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      s[nt][0] = on0 ? s[nt][0] * inv[nt] : -INFINITY;
      s[nt][1] = on1 ? s[nt][1] * inv[nt] : -INFINITY;
      move = move || fmaxf(s[nt][0], s[nt][1]) > m[nt] + 6.f;
    }
    if (__any_sync(full, move)) rescale(s, st);
    float p[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float ms = m[nt] == -INFINITY ? 0.f : m[nt];
      p[nt][0] = exp2_fast(s[nt][0] - ms);
      p[nt][1] = exp2_fast(s[nt][1] - ms);
      l[nt] += p[nt][0] + p[nt][1];
    }
    // ---- outputs, a group of 64 dims at a time: its weights as B fragments, hi and lo
    // beside one another, then its four m-tiles
#pragma unroll
    for (int G = 0; G < NG; ++G) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        cst[nt][G] = fmaf(p[nt][0], ls[0][G], fmaf(p[nt][1], ls[1][G], cst[nt][G]));
        uint32_t hi, lo;
        split_f16x2(p[nt][0] * (st[0][G] * f[G]), p[nt][1] * (st[1][G] * f[G]), hi, lo);
        pb[nt][0] = movm_t(prmt(hi, lo, 0x5410u));
        pb[nt][1] = movm_t(prmt(hi, lo, 0x7632u));
      }
      const uint4 x = *reinterpret_cast<const uint4*>(vb + G * 512 + lane * 16);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t wa = j ? x.y : x.x, wb = j ? x.w : x.z;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a[4] = {wa & m0, wa & m1, wb & m0, wb & m1};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(o[G * 4 + j * 2 + i][nt], a, pb[nt][0], pb[nt][1]);
          wa >>= 8;
          wb >>= 8;
        }
      }
    }
  }

  // The state: outputs [4 NT][D] relative to m, and m and l of each head.
  __device__ __forceinline__ void finish(float* os, float* ml, bool any, int GP, int lane) {
    constexpr unsigned full = 0xffffffffu;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt] += __shfl_xor_sync(full, l[nt], 4);
      l[nt] += __shfl_xor_sync(full, l[nt], 8);
      l[nt] += __shfl_xor_sync(full, l[nt], 16);
      if (g == 0) {
        ml[4 * nt + t] = any ? m[nt] : -INFINITY;
        ml[GP + 4 * nt + t] = any ? l[nt] : 0.f;
      }
      if (!any) continue;
#pragma unroll
      for (int G = 0; G < NG; ++G) {
        float c = cst[nt][G];
        c += __shfl_xor_sync(full, c, 4);
        c += __shfl_xor_sync(full, c, 8);
        c += __shfl_xor_sync(full, c, 16);
        const float back = 1.f / f[G];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float4 v;
          const float(&a)[4] = o[G * 4 + j * 2][nt];
          const float(&b)[4] = o[G * 4 + j * 2 + 1][nt];
          v.x = fmaf((a[0] + a[1]) * 0x1p24f, back, c);
          v.y = fmaf((a[2] + a[3]) * 0x1p20f, back, c);
          v.z = fmaf((b[0] + b[1]) * 0x1p24f, back, c);
          v.w = fmaf((b[2] + b[3]) * 0x1p20f, back, c);
          *reinterpret_cast<float4*>(os + (4 * nt + t) * D + G * 64 + g * 8 + j * 4) = v;
        }
      }
    }
  }
};

}  // namespace dattn
