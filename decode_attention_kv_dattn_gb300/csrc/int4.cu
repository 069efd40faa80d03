// Entries of a 4-bit cache (int4_format.h): quantised as they are written, and read
// back. And the read-back of the other cache formats.
//
// Both are bound by memory: append reads 4 bytes a (key, value) pair of dims and
// writes 9/8, the read-back the other way round. A warp takes one block of 16 tokens
// of one KV head, K or V, in the lanes' order of the block itself: what it stores (or
// loads) is 16 bytes a lane in one piece, what it loads (or stores) of the bf16 rows
// whole 128-byte lines, and a group's least and largest value are 2 (K) or 3 (V)
// shuffles away.
#include "bf16_exact.h"
#include "common.cuh"
#include "int4.cuh"
#include "kernels.h"
#include "mma.cuh"
#include "qk_norm.cuh"
#include "rope_angle.h"
#include "round_f64.h"

namespace dattn {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxWarps = 8;

// The tokens of block blockIdx.x of call row b and where the block is.
struct BlockSpan {
  int t0;          // the block's first token, as an index into the row's new tokens (may be negative)
  int cnt;
  int64_t block;   // of the pool, for KV head 0
  __device__ __forceinline__ bool has(int r) const { return t0 + r >= 0 && t0 + r < cnt; }
};

__device__ __forceinline__ bool find_block(const CacheView& c, int Hkv, int b, int start, int cnt, int t_max, int* err,
                                           BlockSpan& s) {
  const bool report = threadIdx.x == 0;
  if (cnt < 0 || cnt > t_max) {
    if (report && blockIdx.x == 0) raise_error(err, ERR_INDEX);
    return false;
  }
  if (start < 0 && cnt > 0 && report && blockIdx.x == 0) raise_error(err, ERR_INDEX);  // (the tokens before 0)
  if (cnt == 0) return false;
  const int64_t at = static_cast<int64_t>(max(start, 0) / kInt4Block) + blockIdx.x;
  const int64_t t0 = at * kInt4Block - start;
  if (t0 >= cnt) return false;
  const int bpp = c.P / kInt4Block;
  const int64_t pi = at / bpp;
  const int pg = pi < c.bt_stride ? c.block_table[static_cast<int64_t>(b) * c.bt_stride + pi] : -1;
  if (pg < 0 || pg >= c.n_rows) {
    if (report) raise_error(err, ERR_INDEX);
    return false;
  }
  s.t0 = static_cast<int>(t0);
  s.cnt = cnt;
  s.block = static_cast<int64_t>(pg) * Hkv * bpp + (at - pi * bpp);
  return true;
}

// cos and sin of pair j of the block's token r: pairs 2 c, 2 c + 1 as (cos, cos, sin, sin),
// 16 bytes, in an order that spreads what 8 lanes (two tokens, four runs of 8 such) read
// at a time over the banks.
__device__ __forceinline__ int turn_at(int D, int r, int c) {
  const int q = c >> 3;
  return r * (D / 4) + (c & ~7) + ((c & 7) ^ ((q & 3) | ((r & 1) << 2)));
}

// Where the new keys of a token are: its row, position and norm, and the layer's rotation.
struct KeyRow {
  const uint16_t* row;
  const uint16_t* kn;
  const uint64_t* step;
  int64_t pos;
  double inv;
  int r;
  // Dims d, d + 1 (d even) in 64 bits: what the short arithmetic below cannot decide, and
  // rotations that it does not take.
  __device__ __forceinline__ uint32_t exact2(int d) const {
    return key_exact(row, kn, inv, pos, step, r, d) | (key_exact(row, kn, inv, pos, step, r, d + 1) << 16);
  }
};

// bf16 of two values known to within e0 and e1: false where that does not tell.
__device__ __forceinline__ bool settled(F2 v, F2 e, uint32_t& w) {
  float a, b, c, d;
  split(add2(v, e), a, b);
  split(fma2(e, f2(-1.f, -1.f), v), c, d);
  w = pack_bf16x2(c, d);
  return w == pack_bf16x2(a, b);
}

__device__ __forceinline__ void load16(const uint16_t* p, uint32_t (&w)[8]) {
  const uint4 x = ld_nc_v4(p), y = ld_nc_v4(p + 8);
  w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
}

// A normalised value is the bf16 nearest to the exact one, formed in fp32 with a bound of
// 2^-22, a turned one as key_exact says, with kTurnError; about one in 3,000 is not
// decided so and goes to exact2 (7 instructions a value against ~30 of an exact sum for all,
// which took 1,490 us for the prompts below).
//
// Sixteen values from dim d on, normalised; the words that key_pair has to settle into open.
__device__ __forceinline__ void normed(const KeyRow& a, uint32_t (&x)[8], int d, uint32_t& open) {
  if (!a.kn) return;
  uint32_t kw[8];
  load16(a.kn + d, kw);
  const float f = static_cast<float>(a.inv);
  if (!(f >= 0x1p-120f && f <= 0x1p120f)) open = 0xffu;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const F2 v = mul2(mul2(wide2(x[i]), wide2(kw[i])), f2(f, f));
    float v0, v1;
    split(v, v0, v1);
    const F2 e = fma2(f2(fabsf(v0), fabsf(v1)), f2(0x1p-22f, 0x1p-22f), f2(0x1p-110f, 0x1p-110f));
    if (!settled(v, e, x[i])) open |= 1u << i;
  }
}

// x + y s with the bound of its error, into w; whether it settled.
__device__ __forceinline__ bool turned(F2 x, F2 y, F2 s, uint32_t& w) {
  const F2 v = fma2(y, s, x);
  float x0, x1, v0, v1;
  split(x, x0, x1);
  split(v, v0, v1);
  return settled(v, fma2(f2(fabsf(x0) + fabsf(v0), fabsf(x1) + fabsf(v1)), f2(kTurnError, kTurnError), f2(0x1p-110f, 0x1p-110f)), w);
}

// The words of w, dims d0 on, that are open.
__device__ __forceinline__ void settle(const KeyRow& a, int d0, uint32_t open, uint32_t (&w)[8]) {
  while (open) {
    const int i = __ffs(open) - 1;
    open &= open - 1;
    const uint32_t v = a.exact2(d0 + 2 * i);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j == i) w[j] = v;
  }
}

// Sixteen values of a key row from dim d0 on, normalised and turned where ROT says so;
// cs: turn_at of the block's token tok.
template <int D, bool ROT>
__device__ __forceinline__ void key_words(const KeyRow& a, int tok, int d0, const float4* cs, uint32_t (&w)[8]) {
  load16(a.row + d0, w);
  if constexpr (ROT) {
    const int half = a.r / 2;
    uint32_t open = 0;
    if (half % 16 != 0) {
      open = 0xffu;  // (a lane's dims may lie on both sides of the rotation's border)
    } else {
      normed(a, w, d0, open);
      if (d0 < a.r) {
        const bool first = d0 < half;
        const int p0 = first ? d0 + half : d0 - half;
        uint32_t p[8];
        load16(a.row + p0, p);
        normed(a, p, p0, open);
        const uint32_t sign = first ? 0x80008000u : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 f = cs[turn_at(D, tok, (first ? d0 : p0) / 2 + i)];
          if (!turned(mul2(wide2(w[i]), f2(f.x, f.y)), wide2(p[i] ^ sign), f2(f.z, f.w), w[i])) open |= 1u << i;
        }
      }
    }
    settle(a, d0, open, w);
  }
}

// The same of both sides of a rotation, w from dim d0 and p from d0 + half on.
template <int D>
__device__ __forceinline__ void key_words2(const KeyRow& a, int tok, int d0, const float4* cs, uint32_t (&w)[8], uint32_t (&p)[8]) {
  const int p0 = d0 + a.r / 2;
  load16(a.row + d0, w);
  load16(a.row + p0, p);
  uint32_t wopen = 0, popen = 0;
  normed(a, w, d0, wopen);
  normed(a, p, p0, popen);
  wopen = popen = wopen | popen;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 f = cs[turn_at(D, tok, d0 / 2 + i)];
    const F2 x = wide2(w[i]), y = wide2(p[i]), c = f2(f.x, f.y), s = f2(f.z, f.w);
    if (!turned(mul2(x, c), y, mul2(s, f2(-1.f, -1.f)), w[i])) wopen |= 1u << i;
    if (!turned(mul2(y, c), x, s, p[i])) popen |= 1u << i;
  }
  settle(a, d0, wopen, w);
  settle(a, p0, popen, p);
}

// One CTA per block of 16 tokens of a call row; its warps share out (KV head, K or V):
// keys first, so that every warp of many heads has keys and values (a rotated key costs
// twice a value, and warps with keys alone would share two of the SM's four schedulers).
// Tokens that the call does not bring stay as they are. Bound by issue (70% of the slots, ~20
// instructions a value) and by loads that nothing of the warp's covers (the largest stall):
// 64 ragged prompts (126,000 tokens of 8 heads of 128, rotated) 219 us, not rotated 145, where
// their 660 MB take 98. Two kinds of keys cost more: a rotation whose half is not a multiple
// of 16 has every dim of a key formed by key_exact (rotary_dim 40 / 80 595 /
// 868 us, 64 204), and a key norm has a warp sum its 16 rows in fp64, one behind the other
// (1,634 us not rotated, 1,772 rotated; 2 heads of 256 rotated by 64 104 -> 602). With keys turned by rope_cos_sin, which is off by up to 1.5e-7 and moved 50
// of 65 million codes, 205 (3 instead of 4 CTAs an SM 224; keys and values by turns 233;
// one side of a rotation in a lane 215), with one exact step behind the bound 255.
template <int D, bool ROT>
__global__ void __launch_bounds__(kMaxWarps * 32, 4) int4_append_kernel(const AppendArgs a) {
  constexpr int NG = D / kInt4Group;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y;
  BlockSpan s;
  if (!find_block(a.c, a.Hkv, b, a.start_index[b], a.count[b], a.Tmax, a.err, s)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int bpp = a.c.P / kInt4Block;
  __shared__ float4 cs[ROT ? kInt4Block * D / 4 : 1];
  const int64_t pos = ROT && a.start_pos ? a.start_pos[b] : 0;
  if constexpr (ROT) {
    const int half = a.r / 2;
    for (int e = threadIdx.x; e < kInt4Block * half; e += blockDim.x) {
      const int r = e / half, i = e - r * half;
      float* f = reinterpret_cast<float*>(cs + turn_at(D, r, i >> 1)) + (i & 1);
      if (s.has(r)) rope_cos_sin_near(pos + s.t0 + r, a.rope_step[i], f[0], f[2]);
    }
    __syncthreads();
  }
  const int warps = blockDim.x >> 5;
  for (int task = warp; task < 2 * a.Hkv; task += warps) {
    const int h = task < a.Hkv ? task : task - a.Hkv;
    const bool value = task >= a.Hkv;
    const uint16_t* src = (value ? a.v : a.k) + ((static_cast<int64_t>(b) * a.in_T + a.row0 + s.t0) * a.Hkv + h) * D;
    const int64_t pitch = static_cast<int64_t>(a.Hkv) * D;
    uint8_t* dst = reinterpret_cast<uint8_t*>(value ? a.c.v : a.c.k) + (s.block + static_cast<int64_t>(h) * bpp) * int4_block_bytes(D);
    if (!value) {
      // keys: tokens g and g + 8, 16 dims a lane of every group
      double inv0 = 0.0, inv1 = 0.0;
      if (ROT && a.k_norm) {
        for (int r = 0; r < kInt4Block; ++r) {
          if (!s.has(r)) continue;
          const double v = qk_norm_inv(src + r * pitch, D, a.norm_eps, lane);
          if (r == g) inv0 = v;
          if (r == g + 8) inv1 = v;
        }
      }
      auto key = [&](int r, int i) {
        return KeyRow{src + r * pitch, a.k_norm, a.rope_step, pos + s.t0 + r, i ? inv1 : inv0, a.r};
      };
      auto put = [&](const uint32_t (&w)[8], int r, int G, bool on) {
        uint32_t e = extent(w);
        e = max2_nan(e, __shfl_xor_sync(kFull, e, 1));
        e = max2_nan(e, __shfl_xor_sync(kFull, e, 2));
        const Int4Grid q = grid_of(e);
        if (!on) return;
        *reinterpret_cast<uint2*>(dst + int4_key_word(r, G * 8 + t * 2)) = make_uint2(codes<8>(w, q), codes<8>(w + 4, q));
        if (t == 0) *reinterpret_cast<uint32_t*>(dst + int4_pair(D, r, G)) = q.pair;
      };
      // where the two sides of the rotation are whole groups, a lane has both of a pair
      const int across = ROT && a.r > 0 && a.r % 128 == 0 ? a.r / 128 : 0;
#pragma unroll 1
      for (int x = 0; x < 2 * across; ++x) {  // (group, token g or g + 8)
        const int i = x & 1, r = g + 8 * i, G = x >> 1;
        const bool on = s.has(r);
        uint32_t w[8] = {}, p[8] = {};
        if (on) key_words2<D>(key(r, i), r, G * 64 + t * 16, cs, w, p);
        put(w, r, G, on);
        put(p, r, G + across, on);
      }
#pragma unroll 1
      for (int x = 4 * across; x < 2 * NG; ++x) {
        const int i = x & 1, r = g + 8 * i, G = x >> 1;
        const bool on = s.has(r);
        uint32_t w[8] = {};
        if (on) key_words<D, ROT>(key(r, i), r, G * 64 + t * 16, cs, w);
        put(w, r, G, on);
      }
    } else {
      // values: tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9, 8 dims a lane of every group
      int tok[4];
      bool on[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tok[i] = 2 * t + (i & 1) + 8 * (i >> 1);
        on[i] = s.has(tok[i]);
      }
#pragma unroll 1
      for (int G = 0; G < NG; ++G) {
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = on[i] ? ld_nc_v4(src + tok[i] * pitch + G * 64 + g * 8) : make_uint4(0u, 0u, 0u, 0u);
        uint32_t half[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t e = extent(w);
          e = max2_nan(e, __shfl_xor_sync(kFull, e, 4));
          e = max2_nan(e, __shfl_xor_sync(kFull, e, 8));
          e = max2_nan(e, __shfl_xor_sync(kFull, e, 16));
          const Int4Grid q = grid_of(e);
          half[i][0] = codes<4>(w, q) & 0xffffu;
          half[i][1] = codes<4>(w + 2, q) & 0xffffu;
          if (g == 0 && on[i]) *reinterpret_cast<uint32_t*>(dst + int4_pair(D, tok[i], G)) = q.pair;
        }
        uint8_t* d = dst + G * 512 + lane * 16;
        if (on[0] && on[1] && on[2] && on[3]) {
          *reinterpret_cast<uint4*>(d) = make_uint4(half[0][0] | (half[1][0] << 16), half[0][1] | (half[1][1] << 16),
                                                    half[2][0] | (half[3][0] << 16), half[2][1] | (half[3][1] << 16));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (on[i])
#pragma unroll
              for (int j = 0; j < 2; ++j)
                *reinterpret_cast<uint16_t*>(dst + int4_value_half(tok[i], G * 16 + g * 2 + j)) = static_cast<uint16_t>(half[i][j]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- read back
//
// What these kernels write is the caller's, who may give it to a decode as its new token,
// and a decode reads its inputs before it waits for the launch ahead of it: the launch
// behind them is made in the stream's full order (launch_order.h), unless it waits before
// all else.

// Two codes (low 4 bits of each half of w) to their values as a bf16 pair, rounded
// once: the codes become bf16 by their place in 128..143, exactly.
__device__ __forceinline__ uint32_t values2(uint32_t w, uint32_t step2, uint32_t least2) {
  uint32_t c, r;
  const uint32_t x = (w & 0x000f000fu) | 0x43004300u;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(x), "r"(0xc300c300u));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(c), "r"(step2), "r"(least2));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kMaxWarps * 32) int4_read_kernel(const ReadArgs a) {
  constexpr int NG = D / kInt4Group;
  pdl_wait();
  const int b = blockIdx.y;
  BlockSpan s;
  if (!find_block(a.c, a.Hkv, b, a.start_index[b], a.count[b], a.Tmax, a.err, s)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int bpp = a.c.P / kInt4Block;
  for (int task = warp; task < 2 * a.Hkv; task += blockDim.x >> 5) {
    const int h = task >> 1;
    uint16_t* dst = (task & 1 ? a.v : a.k) + ((static_cast<int64_t>(b) * a.Tmax + s.t0) * a.Hkv + h) * D;
    const int64_t pitch = static_cast<int64_t>(a.Hkv) * D;
    const uint8_t* src = reinterpret_cast<const uint8_t*>(task & 1 ? a.c.v : a.c.k) + (s.block + static_cast<int64_t>(h) * bpp) * int4_block_bytes(D);
    if ((task & 1) == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = g + 8 * i;
        if (!s.has(r)) continue;
#pragma unroll
        for (int sec = 0; sec < D / 128; ++sec) {
          const uint4 x = *reinterpret_cast<const uint4*>(src + int4_key_word(r, sec * 16 + t * 2));
          const uint2 pr = *reinterpret_cast<const uint2*>(src + int4_pair(D, r, sec * 2));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t pair = k ? pr.y : pr.x;
            const uint32_t least2 = __byte_perm(pair, 0u, 0x1010), step2 = __byte_perm(pair, 0u, 0x3232);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w = k ? (j ? x.w : x.z) : (j ? x.y : x.x);
              // dims (0, 4), (1, 5), (2, 6), (3, 7)
              const uint32_t v0 = values2(w, step2, least2), v1 = values2(w >> 4, step2, least2);
              const uint32_t v2 = values2(w >> 8, step2, least2), v3 = values2(w >> 12, step2, least2);
              *reinterpret_cast<uint4*>(dst + r * pitch + sec * 128 + k * 64 + t * 16 + j * 8) =
                  make_uint4(__byte_perm(v0, v1, 0x5410), __byte_perm(v2, v3, 0x5410), __byte_perm(v0, v1, 0x7632),
                             __byte_perm(v2, v3, 0x7632));
            }
          }
        }
      }
    } else {
#pragma unroll
      for (int G = 0; G < NG; ++G) {
        const uint4 x = *reinterpret_cast<const uint4*>(src + G * 512 + lane * 16);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int r0 = 2 * t + 8 * p;
          const uint32_t pa = *reinterpret_cast<const uint32_t*>(src + int4_pair(D, r0, G));
          const uint32_t pb = *reinterpret_cast<const uint32_t*>(src + int4_pair(D, r0 + 1, G));
          const uint32_t least2 = __byte_perm(pa, pb, 0x5410), step2 = __byte_perm(pa, pb, 0x7632);
          uint32_t even[4], odd[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w = p ? (j ? x.w : x.z) : (j ? x.y : x.x);
            const uint32_t v0 = values2(w, step2, least2), v1 = values2(w >> 4, step2, least2);
            const uint32_t v2 = values2(w >> 8, step2, least2), v3 = values2(w >> 12, step2, least2);
            even[2 * j] = __byte_perm(v0, v1, 0x5410);
            even[2 * j + 1] = __byte_perm(v2, v3, 0x5410);
            odd[2 * j] = __byte_perm(v0, v1, 0x7632);
            odd[2 * j + 1] = __byte_perm(v2, v3, 0x7632);
          }
          uint16_t* d = dst + r0 * pitch + G * 64 + g * 8;
          if (s.has(r0)) *reinterpret_cast<uint4*>(d) = make_uint4(even[0], even[1], even[2], even[3]);
          if (s.has(r0 + 1)) *reinterpret_cast<uint4*>(d + pitch) = make_uint4(odd[0], odd[1], odd[2], odd[3]);
        }
      }
    }
  }
}

// E4M3 value times scale in fp32, for one rounding to bf16 in all: a product (28 bits)
// that fp32 rounds onto the middle between two bf16 values goes back to its own side.
__device__ __forceinline__ float scaled_e4m3(uint8_t x, float scale) {
  const float v = e4m3_to_f32(x), p = v * scale, e = fmaf(v, scale, -p);
  const uint32_t b = __float_as_uint(p);
  if ((b & 0xffffu) != 0x8000u || !(e > 0.f || e < 0.f)) return p;
  return __uint_as_float((e > 0.f) == (p > 0.f) ? b + 1u : b - 1u);
}

// bf16 and E4M3 caches, paged or ring: one warp per token, 8 dims a lane and step.
template <bool F8>
__global__ void __launch_bounds__(kMaxWarps * 32) read_kernel(const ReadArgs a) {
  pdl_wait();
  const CacheView& c = a.c;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kMaxWarps + (threadIdx.x >> 5);
  const int cnt = a.count[b];
  if (cnt < 0 || cnt > a.Tmax || (!c.paged && cnt > c.R)) {
    if (t == 0 && lane == 0) raise_error(a.err, ERR_INDEX);
    return;
  }
  if (t >= cnt) return;
  const int64_t idx = static_cast<int64_t>(a.start_index[b]) + t;
  int row = -1;
  const int rows = c.paged ? c.P : c.R;  // of a head
  if (idx >= 0) {
    if (c.paged) {
      if (idx / c.P < c.bt_stride) row = c.block_table[static_cast<int64_t>(b) * c.bt_stride + idx / c.P];
    } else {
      row = c.stream_rows ? c.stream_rows[b] : b;
    }
  }
  if (row < 0 || row >= c.n_rows) {
    if (lane == 0) raise_error(a.err, ERR_INDEX);
    return;
  }
  const int64_t src0 = (static_cast<int64_t>(row) * a.Hkv * rows + idx % rows) * a.D;
  const int64_t dst0 = (static_cast<int64_t>(b) * a.Tmax + t) * a.Hkv * a.D;
  for (int e = lane; e < a.Hkv * a.D / 8; e += 32) {
    const int h = e / (a.D / 8), d = (e - h * (a.D / 8)) * 8;
    const int64_t o = src0 + static_cast<int64_t>(h) * rows * a.D + d;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint16_t* pool = i ? c.v : c.k;
      uint4* dst = reinterpret_cast<uint4*>((i ? a.v : a.k) + dst0 + h * a.D + d);
      if constexpr (F8) {
        const float scale = i ? a.v_scale : a.k_scale;
        const uint2 x = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(pool) + o);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t two = (j < 2 ? x.x : x.y) >> (16 * (j & 1));
          w[j] = pack_bf16x2(scaled_e4m3(static_cast<uint8_t>(two), scale), scaled_e4m3(static_cast<uint8_t>(two >> 8), scale));
        }
        *dst = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        *dst = *reinterpret_cast<const uint4*>(pool + o);
      }
    }
  }
}

// Blocks that `tokens` tokens in a row may touch.
unsigned block_count(int tokens) { return static_cast<unsigned>((static_cast<int64_t>(tokens) + kInt4Block - 2) / kInt4Block + 1); }

}  // namespace

cudaError_t launch_append_int4(const AppendArgs& a, cudaStream_t s) {
  const dim3 grid(block_count(a.Tmax), a.B), block(32 * (2 * a.Hkv < kMaxWarps ? 2 * a.Hkv : kMaxWarps));
  const bool rot = a.rotate && (a.r > 0 || a.k_norm);
  auto k = a.D == 128 ? (rot ? int4_append_kernel<128, true> : int4_append_kernel<128, false>)
                      : (rot ? int4_append_kernel<256, true> : int4_append_kernel<256, false>);
  return launch_pdl_waiting(k, grid, block, 0, s, a);
}

cudaError_t launch_read(const ReadArgs& a, bool int4, bool f8, cudaStream_t s) {
  if (int4) {
    const dim3 grid(block_count(a.Tmax), a.B), block(32 * (2 * a.Hkv < kMaxWarps ? 2 * a.Hkv : kMaxWarps));
    return launch_pdl_waiting(a.D == 128 ? int4_read_kernel<128> : int4_read_kernel<256>, grid, block, 0, s, a);
  }
  const dim3 grid((static_cast<unsigned>(a.Tmax) + kMaxWarps - 1) / kMaxWarps, a.B);
  return launch_pdl_waiting(f8 ? read_kernel<true> : read_kernel<false>, grid, dim3(kMaxWarps * 32), 0, s, a);
}

}  // namespace dattn
