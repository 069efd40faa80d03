// Decode over selected pages: the page summaries, their scores against the new
// token's query and the selection (one launch), and the attention over the
// selected pages (another).
//
// Definition. A page's summary is the mean of its P keys as they are stored
// (E4M3: times k_scale), rounded to bf16: the rounding halves what a score
// reads, and a mean only ranks pages. The score of page p for a unit is
//   s_p = max over the group's query heads g of <rot(q_g), summary_p>,
// a real number; the selection is the pages kept for certain (the first and
// the newest ones) and the best of the rest, ties to the lowest page.
//
// Method. Scores of many pages lie arbitrarily near the border, so the
// selection is made twice: the tensor cores screen every page in bf16 x bf16
// with fp32 sums (q as hi + lo bf16 terms), with a bound e on how far a
// screened score may be from the real one; pages whose screened score is more
// than 2e above the k-th largest are in, those more than 2e below are out, and
// the few between are scored again in fp64 and ranked.
#include <cuda_bf16.h>

#include <algorithm>

#include "bf16_exact.h"
#include "common.cuh"
#include "mma.cuh"
#include "qk_norm.cuh"
#include "round_f64.h"

namespace dattn {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;             // of an attention CTA: several CTAs an SM, so that one's prologue or merge
                                      // runs beside another's pass over its keys
constexpr int kList = 1024;           // pages near the border ranked in shared memory
constexpr int kBins = 1024;           // histogram bins of the threshold search
constexpr int kStaged = 16384;        // scores held in shared memory during the selection
constexpr int kMaxSplits = 160;       // CTAs of a unit in the attention
constexpr float kWeightUp = 32768.f;  // E4M3: the softmax weights' factor in fp16

// The cached tokens of stream b as every paged call reads them: clamped to the
// call's bound, with the error reported once.
__device__ __forceinline__ int stream_length(const CacheView& c, int b, int max_len, bool report, int* err) {
  int n = c.seq_len[b];
  const int cap = static_cast<int>(min(static_cast<int64_t>(max_len), static_cast<int64_t>(c.bt_stride) * c.P));
  if (n < 0 || n > cap) {
    if (report) raise_error(err, ERR_LENGTH);
    n = n < 0 ? 0 : cap;
  }
  return n;
}

// Physical page of a stream's logical page; a bad entry reads page 0 and is
// reported (as in the decode kernel).
__device__ __forceinline__ int physical_page(const CacheView& c, int b, int p, int* err) {
  int pg = c.block_table[static_cast<int64_t>(b) * c.bt_stride + p];
  if (pg < 0 || pg >= c.n_rows) {
    raise_error(err, ERR_INDEX);
    pg = 0;
  }
  return pg;
}

// 16 bytes of the cache, read once: past the L1, which holds nothing of a row
// that an earlier launch may still have been writing.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// The E4M3 byte nearest x / scale (ties to even, saturating at 448; scale > 0).
// y, the fp32 quotient, lies on the same side of every border between two bytes
// as the exact one, unless it is that border (a number of at most 5 significant
// bits): then the sign of the remainder says which side.
__device__ __forceinline__ uint8_t e4m3_of_quotient(float x, float scale) {
  float y = __fdiv_rn(x, scale);
  const float r = fmaf(-y, scale, x);  // exact
  const int bits = __float_as_int(y);
  if ((bits & 0x7ffff) == 0 && r != 0.f && y != 0.f && fabsf(y) < 448.f)
    y = __int_as_float((r > 0.f) == (y > 0.f) ? bits + 1 : bits - 1);
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3));
}

// A norm's square: infinite where it is no number, so that maxima keep it.
__device__ __forceinline__ float nan_to_inf(float x) { return x == x ? x : INFINITY; }

// ---------------------------------------------------------------- summaries

// One warp per (completed page, KV head): 16-byte loads, every lane the same
// dims of a few rows at a time, fp32 sums joined across the warp's row groups.
// Bound by reading the keys once; the page's rows of one head are contiguous.
// 64 prompts of 64 - 4,096 tokens, 8 heads of 128, pages of 16: 274 MB in 45 us
// (6.1 TB/s); after one decode step of 64 streams 2.4 us in a graph.
template <int D, bool F8>
__global__ void __launch_bounds__(256) summarize_kernel(const SummarizeArgs a) {
  constexpr int EPL = F8 ? 16 : 8;          // elements of a 16-byte load
  constexpr int LPR = D / EPL;              // lanes of a row
  constexpr int RPI = 32 / LPR;             // rows of a warp's load
  constexpr int UN = 4;                     // loads in flight a lane
  pdl_wait();
  pdl_trigger();
  const CacheView& c = a.c;
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int64_t job = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int cnt = a.count[b], start = a.start_index[b];
  if (cnt < 0 || cnt > a.max_tokens || start < 0 || cnt > INT32_MAX - start) {
    if (job == 0 && lane == 0) raise_error(a.err, ERR_INDEX);
    return;
  }
  const int i = static_cast<int>(job / a.Hkv), h = static_cast<int>(job - static_cast<int64_t>(i) * a.Hkv);
  const int first = start / c.P, done = (start + cnt) / c.P;
  // (the grid covers a table's pages, whatever max_tokens says; the others are none)
  if (job == 0 && lane == 0 && first < done && done > c.bt_stride) raise_error(a.err, ERR_INDEX);
  if (i >= done - first) return;
  const int p = first + i;
  const int pg = p < c.bt_stride ? c.block_table[static_cast<int64_t>(b) * c.bt_stride + p] : -1;
  if (pg < 0 || pg >= c.n_rows) {
    if (lane == 0) raise_error(a.err, ERR_INDEX);
    return;
  }
  const int64_t base = (static_cast<int64_t>(pg) * a.Hkv + h) * c.P * D;
  const uint8_t* src = reinterpret_cast<const uint8_t*>(c.k) + base * (F8 ? 1 : 2);
  const int row0 = lane / LPR, col = lane % LPR;
  float acc[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
  for (int r = row0; r < c.P; r += RPI * UN) {
    uint4 w[UN];
#pragma unroll
    for (int x = 0; x < UN; ++x)
      if (r + x * RPI < c.P)
        w[x] = *reinterpret_cast<const uint4*>(src + (static_cast<int64_t>(r + x * RPI) * D + col * EPL) * (F8 ? 1 : 2));
      else
        w[x] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int x = 0; x < UN; ++x) {
      const uint32_t v[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if constexpr (F8) {
          const uint32_t lo = e4m3x2_lo(v[y]), hi = e4m3x2_hi(v[y]);
          const float2 l2 = __half22float2(*reinterpret_cast<const __half2*>(&lo));
          const float2 h2 = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          acc[4 * y] += l2.x;
          acc[4 * y + 1] += l2.y;
          acc[4 * y + 2] += h2.x;
          acc[4 * y + 3] += h2.y;
        } else {
          acc[2 * y] += bf16_lo(v[y]);
          acc[2 * y + 1] += bf16_hi(v[y]);
        }
      }
    }
  }
#pragma unroll
  for (int w = LPR; w < 32; w <<= 1)
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] += __shfl_xor_sync(kFull, acc[e], w);
  if (row0 == 0) {
    const float inv = 1.f / static_cast<float>(c.P);
    uint32_t o[EPL / 2];
#pragma unroll
    for (int e = 0; e < EPL / 2; ++e) {
      float x = acc[2 * e] * inv, y = acc[2 * e + 1] * inv;
      if constexpr (F8) {
        x *= a.k_scale;
        y *= a.k_scale;
      }
      o[e] = pack_bf16x2(x, y);
    }
    uint16_t* dst = a.summary + (static_cast<int64_t>(pg) * a.Hkv + h) * D + col * EPL;
#pragma unroll
    for (int e = 0; e < EPL / 8; ++e)
      *reinterpret_cast<uint4*>(dst + 8 * e) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
  }
}

// ---------------------------------------------------------------- the new token's query

// The group's queries, normalised, rotated in fp32 and scaled. A thread has one
// pair of dims (d0, d1) of the heads g0, g0 + STEP, ...: its angle is worked out
// once, and all its loads are in flight together. Caller inputs only, so this
// runs before the wait for the launch before.
template <int D, int GP, int NTH>
struct QueryPairs {
  static constexpr int PAIRS = D / 2, STEP = NTH / PAIRS, ITER = (GP + STEP - 1) / STEP;
  int d0, d1, g0;
  uint16_t x[ITER], y[ITER];  // before the rotation
  float v0[ITER], v1[ITER];   // heads past the group's are zeros

  __device__ __forceinline__ void load(const PageArgs& a, int b, int h, float scale, double* inv_s) {
    const uint16_t* q = a.q + (static_cast<int64_t>(b) * a.Hkv + h) * a.G * D;
    const int p = threadIdx.x % PAIRS, half = a.r / 2;
    g0 = threadIdx.x / PAIRS;
    d0 = p < half ? p : a.r + 2 * (p - half);
    d1 = p < half ? p + half : d0 + 1;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int g = g0 + i * STEP;
      x[i] = g < a.G ? q[g * D + d0] : 0;
      y[i] = g < a.G ? q[g * D + d1] : 0;
    }
    float cf = 1.f, sf = 0.f;
    if (p < half) rope_cos_sin(a.pos[b], a.rope_step[p], cf, sf);
    if (a.q_norm) {
      for (int g = threadIdx.x >> 5; g < a.G; g += NTH / 32) {
        const double inv = qk_norm_inv(q + g * D, D, a.norm_eps, threadIdx.x & 31);
        if ((threadIdx.x & 31) == 0) inv_s[g] = inv;
      }
      __syncthreads();
      const uint16_t w0 = a.q_norm[d0], w1 = a.q_norm[d1];
#pragma unroll
      for (int i = 0; i < ITER; ++i)
        if (g0 + i * STEP < a.G) {
          x[i] = qk_norm_apply(x[i], w0, inv_s[g0 + i * STEP]);
          y[i] = qk_norm_apply(y[i], w1, inv_s[g0 + i * STEP]);
        }
    }
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const float xf = bf16_to_f32(x[i]), yf = bf16_to_f32(y[i]);
      v0[i] = (p < half ? fmaf(xf, cf, -yf * sf) : xf) * scale;
      v1[i] = (p < half ? fmaf(yf, cf, xf * sf) : yf) * scale;
    }
  }
};

// ---------------------------------------------------------------- scores and selection

// fp64 to an unsigned key of the same order (NaN above everything).
__device__ __forceinline__ uint64_t order_key(double x) {
  if (x != x) x = INFINITY;
  const uint64_t v = static_cast<uint64_t>(__double_as_longlong(x + 0.0));  // -0 as +0
  return (v >> 63) ? ~v : (v | 0x8000000000000000ull);
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return x;
}

// Block-wide sum and maximum, known to every thread (`buf`: a word a warp).
template <int NTH>
__device__ __forceinline__ int block_sum(int x, int* buf) {
  x = __reduce_add_sync(kFull, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  return __reduce_add_sync(kFull, (threadIdx.x & 31) < NTH / 32 ? buf[threadIdx.x & 31] : 0);
}
template <int NTH>
__device__ __forceinline__ float block_max(float x, int* buf) {
  x = warp_max(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = __float_as_int(x);
  __syncthreads();
  return warp_max((threadIdx.x & 31) < NTH / 32 ? __int_as_float(buf[threadIdx.x & 31]) : -INFINITY);
}

// Join of `parts` CTAs of a unit: true in all threads of the last one to arrive,
// which then sees what the others wrote before. The counter is left at zero.
__device__ __forceinline__ bool last_to_arrive(int* counter, int parts, int* flag) {
  __syncthreads();
  if (parts == 1) return true;
  if (threadIdx.x == 0) {
    // (release: the block's writes, after the barrier; acquire: the other blocks')
    int before;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    const bool last = before == parts - 1;
    if (last) *counter = 0;
    *flag = last;
  }
  __syncthreads();
  return *flag != 0;
}

struct SelectShared {
  alignas(16) int hist[kBins];
  int list[kList];
  alignas(16) float value[kList];
  alignas(16) uint64_t list_key[kList];
  uint64_t step[128];  // the rotation's phase steps
  int buf[32];
  int n_list, bin, above, inside, flag;
  float threshold;
  double inv[8];
};

// Which candidates the exact scores are needed for: those with screened scores
// in [dn, up] (all, where the screen does not hold).
struct Border {
  float dn, up;
  bool screened;
  __device__ __forceinline__ bool near(float x) const { return !screened || (x <= up && x >= dn); }
};

// The exact score of a summary held 2 dims a lane with one query head, as a key,
// by one warp.
template <int D>
__device__ __forceinline__ uint64_t exact_key(const uint32_t (&w)[D / 64], const double* q, int lane) {
  double y0 = 0.0, y1 = 0.0;
#pragma unroll
  for (int x = 0; x < D / 64; ++x) {
    const double2 qd = *reinterpret_cast<const double2*>(q + 64 * x + lane * 2);
    y0 = fma(qd.x, static_cast<double>(bf16_lo(w[x])), y0);
    y1 = fma(qd.y, static_cast<double>(bf16_hi(w[x])), y1);
  }
  double z = y0 + y1;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
  return order_key(z);
}

// `want` of the many pages near the border (equal summaries, or values beyond
// the fp32 range): their keys go to memory and the border is found bit by bit,
// first of the keys, then of the page among equal keys. Apart, for it is rarely
// run and the selection's cost is mostly its instructions' first fetch.
template <int D, int NTH>
__device__ __noinline__ void select_of_many(const PageArgs& a, int u, int b, int h, int lo, int N, int want,
                                            const float* sc, const double* q64, Border border, uint32_t* bits,
                                            int* buf) {
  const int t = threadIdx.x, lane = t & 31;
  uint64_t* keys = a.keys + static_cast<int64_t>(u) * a.pitch;
  for (int i = t >> 5; i < N; i += NTH / 32) {
    if (!border.near(__ldcg(sc + i))) continue;
    const uint16_t* src =
        a.summary + (static_cast<int64_t>(physical_page(a.c, b, lo + i, a.err)) * a.Hkv + h) * D + lane * 2;
    uint32_t w[D / 64];
#pragma unroll
    for (int x = 0; x < D / 64; ++x) w[x] = *reinterpret_cast<const uint32_t*>(src + 64 * x);
    uint64_t key = 0;
    for (int g = 0; g < a.G; ++g) key = max(key, exact_key<D>(w, q64 + g * D, lane));
    if (lane == 0) keys[i] = key;
  }
  __syncthreads();
  uint64_t T = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t cand = T | (1ull << bit);
    int x = 0;
    for (int i = t; i < N; i += NTH) x += border.near(__ldcg(sc + i)) && keys[i] >= cand;
    if (block_sum<NTH>(x, buf) >= want) T = cand;
  }
  int x = 0;
  for (int i = t; i < N; i += NTH) x += border.near(__ldcg(sc + i)) && keys[i] > T;
  const int ties = want - block_sum<NTH>(x, buf);  // of the pages with key T, the lowest
  int step = 1;
  while (step < N) step <<= 1;
  int last = -1;  // the largest candidate up to which fewer than `ties` of them lie
  for (; step >= 1; step >>= 1) {
    const int cand = last + step;
    if (cand >= N) continue;
    int y = 0;
    for (int i = t; i <= cand; i += NTH) y += border.near(__ldcg(sc + i)) && keys[i] == T;
    if (block_sum<NTH>(y, buf) < ties) last = cand;
  }
  for (int i = t; i < N; i += NTH)
    if (border.near(__ldcg(sc + i)) && (keys[i] > T || (keys[i] == T && i <= last + 1)))
      atomicOr(&bits[i >> 5], 1u << (i & 31));
}

// The selection of one unit from its screened scores, by one CTA. Candidate i is
// page lo + i; a warp's 32 scores are consecutive candidates, so one ballot is a
// word of the bitmap of those selected. q_raw: the group's (normalised) bf16
// queries [G][D] in shared memory. What it costs is mostly latency - of the
// passes' dependent steps and of fetching its instructions - so its loops are
// short rather than unrolled.
template <int D, int NTH>
__device__ void select_unit(const PageArgs& a, int u, int b, int h, int pages, const uint16_t* q_raw, uint8_t* dyn,
                            SelectShared& s) {
  constexpr int W = NTH / 32;
  const CacheView& c = a.c;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int lo = a.keep_first, N = pages - a.keep_last - lo;
  const int k = a.num_pages - a.keep_first - a.keep_last;  // 0 <= k < N
  uint32_t* bits = reinterpret_cast<uint32_t*>(dyn);
  double* q64 = reinterpret_cast<double*>(dyn + a.q64_off);
  const float* gsc = a.scores + static_cast<int64_t>(u) * a.pitch + lo;
  float* staged = reinterpret_cast<float*>(dyn + a.staged_off);
  // A pass over the candidates: f(candidate, score) by whole warps of
  // consecutive candidates; past the last one, candidate N and -inf. Scores come
  // through shared memory, `staged` at a time (all of them, if they fit: then
  // only the first pass loads them), several loads in flight a thread.
  const int cap = a.staged;
  bool loaded = false;
  auto pass = [&](auto f) {
    for (int s0 = 0; s0 < N; s0 += cap) {
      const int n = min(cap, N - s0), full = (n + 127) & ~127;
      if (!loaded) {
        __syncthreads();
        for (int i0 = t; i0 < full; i0 += 16 * NTH) {
          float x[16];
#pragma unroll
          for (int y = 0; y < 16; ++y) x[y] = i0 + y * NTH < n ? __ldcg(gsc + s0 + i0 + y * NTH) : -INFINITY;
#pragma unroll
          for (int y = 0; y < 16; ++y)
            if (i0 + y * NTH < full) staged[i0 + y * NTH] = x[y];
        }
        __syncthreads();
        loaded = N <= cap;
      }
      for (int i0 = warp * 128 + lane; i0 < full; i0 += 4 * NTH) {
        float x[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) x[y] = staged[i0 + y * 32];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (i0 + y * 32 - lane < n) f(min(s0 + i0 + y * 32, N), x[y]);
      }
    }
  };
  // ---- the screened scores' range and error bound
  float mn = INFINITY, mx = -INFINITY, cn = 0.f;
  const float qn = __ldcg(a.qnorm + u);
  for (int x = lo / a.chunk_pages + lane; x < a.chunks && x * a.chunk_pages < lo + N; x += 32) {
    const float* info = a.cinfo + (static_cast<int64_t>(u) * a.chunks + x) * 3;
    mn = fminf(mn, __ldcg(info));
    mx = fmaxf(mx, __ldcg(info + 1));
    cn = fmaxf(cn, __ldcg(info + 2));
  }
  for (int x = t; x < kBins; x += NTH) s.hist[x] = 0;
  if (t == 0) s.n_list = 0;
  mn = -warp_max(-mn);
  mx = warp_max(mx);
  cn = warp_max(cn);
  // Error of a screened score, relative to |q| |summary|: the tensor cores'
  // fp32 sums, D / 16 steps of 17 addends that may each lose 2^-23 of the
  // largest (D 2^-23 1.07 in all; what the lo terms add is 2^-9 of that), q
  // as two bf16 terms (2^-17) and the fp32 rotation (2^-20): below D 2^-22
  // for D >= 128. Sums below the fp32 range add 2^-100.
  const float e = fmaf(static_cast<float>(D) * 2.3841858e-7f * cn, qn, 7.9e-31f);
  // (a NaN or overflow anywhere makes e, mn or mx fail this)
  Border border{-INFINITY, INFINITY, e < 1e36f && mx < 1e38f && mn > -1e38f && k > 0};
  // append to the list by the lanes of `mask` (a whole warp calls)
  auto append = [&](uint32_t mask, int i, float x) {
    int at = 0;
    if (lane == 0) at = atomicAdd(&s.n_list, __popc(mask));
    at = __shfl_sync(kFull, at, 0) + __popc(mask & ((1u << lane) - 1u));
    if ((mask >> lane & 1u) && at < kList) {
      s.list[at] = i;
      s.value[at] = x;
    }
  };
  auto select = [&](int i) { atomicOr(&bits[i >> 5], 1u << (i & 31)); };
  int want = k, m = 0;  // still to be chosen, of the m pages near the border in the list
  bool listed = false;
  if (border.screened) {
    // ---- the k-th largest screened score lies in [a0, a1]: narrowed by
    // histograms of equal value ranges
    float a0 = mn, a1 = mx;
    const float size = fmaxf(fabsf(mn), fabsf(mx));
    // counts above each bin of the histogram, from the top: where the kk-th
    // largest lies (s.bin), and how many are above and in that bin
    auto find_bin = [&](int above, int kk) {
      __syncthreads();
      constexpr int BPT = kBins / NTH;  // bins of a thread
      int own[BPT], mine = 0;
#pragma unroll
      for (int x = 0; x < BPT; ++x) {
        own[x] = s.hist[kBins - 1 - (t * BPT + x)];
        mine += own[x];
      }
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s.buf[warp] = incl;
      __syncthreads();
      int top = above + incl - mine + __reduce_add_sync(kFull, lane < warp ? s.buf[lane] : 0);
#pragma unroll
      for (int x = 0; x < BPT; ++x) {
        if (top < kk && kk <= top + own[x]) {
          s.bin = kBins - 1 - (t * BPT + x);
          s.above = top;
          s.inside = own[x];
        }
        top += own[x];
      }
      __syncthreads();
    };
    // ---- few candidates: all of them listed, and ranked below (64 streams of 8
    // heads: 96 - 120 candidates 45.4 us this way, 46.9 by histograms; 215 - 251
    // candidates 53.8 and 49.6)
    if (N <= 128) {
      __syncthreads();
      for (int i = t; i < N; i += NTH) {
        s.list[i] = i;
        s.value[i] = __ldcg(gsc + i);
      }
      if (t == 0) s.n_list = N;
      __syncthreads();
      listed = true;
    }
    // ---- long streams, by way of the 16-page tiles' maxima: the k-th largest of
    // them has k scores at or above it, so the k-th largest score is no less,
    // and only tiles that reach it have scores to look at (1 x 1,048,576 tokens
    // 25.4 us, 29.5 without; where tiles are fewer than twice what is chosen it
    // does not pay: 64 x 16,384 tokens 48.7 us with, 45.9 without)
    const int tile0 = lo >> 4, tiles = ((lo + N - 1) >> 4) - tile0 + 1;
    if (!listed && tiles >= 2 * k && a1 > a0) {
      const float* gtm = a.tile_max + static_cast<int64_t>(u) * a.tile_pitch + tile0;
      const float inv = static_cast<float>(kBins) / (a1 - a0);
      if (inv > 0.f && inv < 1e38f) {
        int* near_tiles = reinterpret_cast<int*>(s.list_key);
        __syncthreads();
        for (int x = t; x < tiles; x += NTH)
          atomicAdd(&s.hist[min(kBins - 1, static_cast<int>((__ldcg(gtm + x) - a0) * inv))], 1);
        find_bin(0, k);
        if (s.above + s.inside <= kList - 256) {
          const float edge = a0 + s.bin / inv - 2.5f * e - 2e-6f * size;
          for (int x = t; x < tiles; x += NTH)
            if (__ldcg(gtm + x) >= edge) {
              const int at = atomicAdd(&s.n_list, 1);
              if (at < kList) near_tiles[at] = x;
            }
          __syncthreads();
          const int found = min(s.n_list, kList);
          const bool all = s.n_list <= kList;
          __syncthreads();
          if (t == 0) s.n_list = 0;
          __syncthreads();
          for (int x0 = warp * 2; x0 < found; x0 += 2 * W) {  // 16 lanes a tile
            const int x = x0 + (lane >> 4);
            const int i = x < found ? (near_tiles[x] + tile0) * 16 + (lane & 15) - lo : -1;
            const float y = i >= 0 && i < N ? __ldcg(gsc + i) : -INFINITY;
            const uint32_t mask = __ballot_sync(kFull, y >= edge);
            if (mask) append(mask, i, y);
          }
          __syncthreads();
          listed = all && s.n_list <= kList;
        }
        if (!listed) {
          __syncthreads();
          for (int x = t; x < kBins; x += NTH) s.hist[x] = 0;
          if (t == 0) s.n_list = 0;
        }
      }
    }
    int above = 0;  // scores above a1
    for (int round = 0; round < 8 && !listed; ++round) {
      const float inv = a1 > a0 ? static_cast<float>(kBins) / (a1 - a0) : 0.f;
      if (!(inv > 0.f && inv < 1e38f)) break;  // one value, or too narrow to cut
      auto bin_of = [&](float x) { return min(kBins - 1, static_cast<int>((x - a0) * inv)); };
      __syncthreads();
      if (round > 0) {
        for (int x = t; x < kBins; x += NTH) s.hist[x] = 0;
        __syncthreads();
      }
      pass([&](int i, float x) {
        if (x >= a0 && x <= a1) atomicAdd(&s.hist[bin_of(x)], 1);
      });
      find_bin(above, k);
      const int bin = s.bin, inside = s.inside;
      above = s.above;
      if (above + inside <= kList - 256) {
        // few enough: every score that can matter - down to 2 e below the bin's
        // lower edge, and what rounding may have moved that edge - in the list
        const float edge = a0 + bin / inv - 2.5f * e - 2e-6f * size;
        pass([&](int i, float x) {
          const uint32_t mask = __ballot_sync(kFull, x >= edge);
          if (mask) append(mask, i, x);
        });
        __syncthreads();
        listed = s.n_list <= kList;
        break;
      }
      // the bin's own range
      float b0 = INFINITY, b1 = -INFINITY;
      pass([&](int i, float x) {
        if (x >= a0 && x <= a1 && bin_of(x) == bin) {
          b0 = fminf(b0, x);
          b1 = fmaxf(b1, x);
        }
      });
      a0 = -block_max<NTH>(-b0, s.buf);
      a1 = block_max<NTH>(b1, s.buf);
      if (inside <= 256) break;  // (a bracket of [a0, a1] is narrow enough)
    }
    if (listed) {
      // the k-th largest by rank in the list
      const int all = s.n_list;
      for (int y = t; y < all; y += NTH) {
        const float w = s.value[y];
        int more = 0, same = 0;
        int x = 0;
        for (; x + 4 <= all; x += 4) {
          const float4 z = *reinterpret_cast<const float4*>(s.value + x);
          more += (z.x > w) + (z.y > w) + (z.z > w) + (z.w > w);
          same += (z.x == w) + (z.y == w) + (z.z == w) + (z.w == w);
        }
        for (; x < all; ++x) {
          more += s.value[x] > w;
          same += s.value[x] == w;
        }
        if (more < k && k <= more + same) s.threshold = w;  // equal scores write the same
      }
      for (int w = t; w < (N + 31) / 32; w += NTH) bits[w] = 0;
      __syncthreads();
      a0 = a1 = s.threshold;
    }
    border.up = __fadd_ru(a1, 2.f * e);
    border.dn = __fsub_rd(a0, 2.f * e);
  }
  if (listed) {
    // ---- in, out, or near the border, from the list; those near it move to
    // its front
    const int all = s.n_list;
    int i[kList / NTH], in = 0;
#pragma unroll
    for (int y = 0; y < kList / NTH; ++y) {
      const int x = t + y * NTH;
      i[y] = -1;
      if (x < all) {
        const float v = s.value[x];
        if (v > border.up) {
          select(s.list[x]);
          ++in;
        } else if (v >= border.dn) {
          i[y] = s.list[x];
        }
      }
    }
    want = k - block_sum<NTH>(in, s.buf);
    if (t == 0) s.n_list = 0;
    __syncthreads();
#pragma unroll
    for (int y = 0; y < kList / NTH; ++y)
      if (i[y] >= 0) s.list[atomicAdd(&s.n_list, 1)] = i[y];
    __syncthreads();
    m = s.n_list;
  } else {
    __syncthreads();
    if (t == 0) s.n_list = 0;
    __syncthreads();
    // ---- the same from the scores
    int in = 0;
    const float up = border.up;
    const bool screened = border.screened;
    pass([&](int i, float x) {
      const uint32_t mask = __ballot_sync(kFull, i < N && screened && x > up);
      const uint32_t close = __ballot_sync(kFull, i < N && k > 0 && border.near(x));
      if (close) append(close, i, x);
      if (lane == 0) bits[i >> 5] = mask;
      in += __popc(mask);
    });
    want = k - block_sum<NTH>(lane == 0 ? in : 0, s.buf);  // k > 0: 1 <= want <= m
    m = s.n_list;
  }
  // ---- the pages near the border again in fp32: a lane's 2 E products and five
  // levels of sums, on the fp32 query
  constexpr int E = D / 64;
  uint32_t ahead[E];
  auto fetch = [&](int x) {  // the summary of list entry x, 2 dims a lane
    const uint16_t* src =
        a.summary + (static_cast<int64_t>(physical_page(c, b, lo + s.list[x], a.err)) * a.Hkv + h) * D + lane * 2;
#pragma unroll
    for (int y = 0; y < E; ++y) ahead[y] = *reinterpret_cast<const uint32_t*>(src + 64 * y);
  };
  if (want < m && m <= 4 * W && border.screened) {
    const float* qf = reinterpret_cast<const float*>(dyn + a.qf_off);
    for (int x = warp; x < m; x += W) {
      fetch(x);
      float best = -INFINITY;
      for (int g = 0; g < a.G; ++g) {
        float y0 = 0.f, y1 = 0.f;
#pragma unroll
        for (int y = 0; y < E; ++y) {
          const float2 qd = *reinterpret_cast<const float2*>(qf + g * D + 64 * y + lane * 2);
          y0 = fmaf(qd.x, bf16_lo(ahead[y]), y0);
          y1 = fmaf(qd.y, bf16_hi(ahead[y]), y1);
        }
        float z = y0 + y1;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
        best = fmaxf(best, z);
      }
      if (lane == 0) s.value[x] = best;
    }
    __syncthreads();
    // Error, relative to |q| |summary|: 4 products a chain, the join and five
    // sums (10 roundings of 2^-24: 6.0e-7) and the query: cosine and sine within
    // 1.5e-7 each and two roundings (at most 1.5e-7 sqrt(2) + 2^-23: 3.4e-7).
    const float e2 = fmaf(1.2e-6f * cn, qn, 7.9e-31f);
    int sure = 0, i = -1;
    if (t < m) {
      const float v = s.value[t];
      int over = 0, may = 0;  // those surely above this one; those possibly above or equal
      for (int x = 0; x < m; ++x) {
        over += s.value[x] > v + 2.f * e2;
        may += x != t && s.value[x] >= v - 2.f * e2;
      }
      if (may < want) {  // surely among the best
        select(s.list[t]);
        sure = 1;
      } else if (over < want) {
        i = s.list[t];
      }
    }
    const int taken = block_sum<NTH>(sure, s.buf);
    want -= taken;
    if (t == 0) s.n_list = 0;
    __syncthreads();
    if (i >= 0) s.list[atomicAdd(&s.n_list, 1)] = i;
    __syncthreads();
    m = s.n_list;
  }
  if (want == m && m <= kList) {
    for (int x = t; x < m; x += NTH) select(s.list[x]);
  } else if (want == m) {
    for (int i = t; i < N; i += NTH)
      if (border.near(__ldcg(gsc + i))) select(i);
  } else {
    // ---- exact scores of the pages near the border: q rotated in fp64. A warp
    // has a page and a head at a time; the first summaries load meanwhile.
    const bool few = m <= kList;
    if (few && warp < m * a.G) fetch(warp / a.G);
    const int half = a.r / 2;
    const int64_t pos = a.pos[b];
    double2* turn = reinterpret_cast<double2*>(s.hist);  // [half] cos, sin
    for (int p = t; p < half; p += NTH) {
      int64_t cq, sq;
      rope_cos_sin_q62(pos, s.step[p], cq, sq);
      turn[p] = make_double2(static_cast<double>(cq) * 2.168404344971009e-19, static_cast<double>(sq) * 2.168404344971009e-19);
    }
    for (int x = t; x < min(m, kList); x += NTH) s.list_key[x] = 0;
    __syncthreads();
    for (int i = t; i < a.G * (D / 2); i += NTH) {
      const int g = i / (D / 2), p = i - g * (D / 2);
      const int d0 = p < half ? p : a.r + 2 * (p - half);
      const int d1 = p < half ? p + half : d0 + 1;
      const double x = bf16_to_f32(q_raw[g * D + d0]), y = bf16_to_f32(q_raw[g * D + d1]);
      const double2 cs = p < half ? turn[p] : make_double2(1.0, 0.0);
      q64[g * D + d0] = p < half ? x * cs.x - y * cs.y : x;
      q64[g * D + d1] = p < half ? y * cs.x + x * cs.y : y;
    }
    __syncthreads();
    if (few) {
      for (int x = warp; x < m * a.G; x += W) {
        const uint64_t key = exact_key<D>(ahead, q64 + (x % a.G) * D, lane);
        if (lane == 0) atomicMax(reinterpret_cast<unsigned long long*>(&s.list_key[x / a.G]), key);
        if (x + W < m * a.G) fetch((x + W) / a.G);
      }
      __syncthreads();
      for (int y = t; y < m; y += NTH) {
        const uint64_t key = s.list_key[y];
        const int i = s.list[y];
        int before = 0;
        for (int x = 0; x < m; ++x) before += s.list_key[x] > key || (s.list_key[x] == key && s.list[x] < i);
        if (before < want) select(i);
      }
    } else {
      select_of_many<D, NTH>(a, u, b, h, lo, N, want, gsc, q64, border, bits, s.buf);
    }
  }
  __syncthreads();

  // ---- the pages in ascending order: the first ones, the selected, the newest
  int32_t* table = a.table + static_cast<int64_t>(u) * a.num_pages;
  int32_t* sel = a.selected ? a.selected + static_cast<int64_t>(u) * a.num_pages : nullptr;
  const int32_t* pt = c.block_table + static_cast<int64_t>(b) * c.bt_stride;
  const int words = (N + 31) / 32;
  int done = 0;
  for (int w0 = 0; w0 < words; w0 += NTH) {
    const int w = w0 + t;
    uint32_t mask = w < words ? bits[w] : 0;
    const int mine = __popc(mask);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) s.buf[warp] = incl;
    __syncthreads();
    const int of = lane < W ? s.buf[lane] : 0;
    int at = done + incl - mine + __reduce_add_sync(kFull, lane < warp ? of : 0);
    done += __reduce_add_sync(kFull, of);
    for (; mask; mask &= mask - 1, ++at) {
      const int i = w * 32 + __ffs(mask) - 1;
      // (at < k) the list in shared memory where it fits: then all threads
      // fetch the table's entries at once
      if (k <= kBins)
        s.hist[at] = i;
      else
        table[lo + at] = i;
    }
  }
  __syncthreads();
  for (int i = t; i < a.num_pages; i += NTH) {
    int p;
    if (i < lo)
      p = i;
    else if (i < lo + k)
      p = lo + (k <= kBins ? s.hist[i - lo] : table[i]);
    else
      p = lo + N + (i - lo - k);
    table[i] = pt[p];
    if (sel) sel[i] = p;
  }
}

// Screened scores, and the selection by the CTA that finishes a unit's last
// chunk (a per-unit counter). A warp takes 16 pages at a time as the rows of an
// m16n8k16 A operand. The sum over the dims may run in any order, so a lane's
// 16-byte load of a summary (8 dims) is its k-elements of two MMAs, without a
// trip through shared memory; the query's B operand uses the same order and
// stays in registers. Columns: the group's heads as bf16 hi and, 4 (or one
// 8-column tile) further, what is left as bf16 lo.
// Bound by reading the candidates' summaries once (D * 2 bytes a page and
// head) only where there are many - E4M3 64 x 16,384 tokens, 128 units of about
// 980 pages: 64 MB in 7.3 us of the CTAs' 16; the squared norm that the error
// bound needs is one bf16x2 FMA a loaded word. The rest is the chain of a unit's
// selection: q 1.6 us, scores 2 - 3, the chunks' join 1.5 - 2, the border 2 - 4,
// exact scores and the pages in order 2. In all (under ncu) 15 us at 1 x
// 1,048,576 tokens, 21 at 8 x 262,144, 18 at 64 ragged streams, 24 at E4M3 64 x
// 16,384, 12 at 1 x 5,003.
template <int D, int NT, int NTH>
__global__ void __launch_bounds__(NTH, NTH == 256 ? (D == 128 ? 4 : 2) : 1) page_select_kernel(const PageArgs a) {
  constexpr int W = NTH / 32;
  constexpr int GP = NT * 4;
  constexpr int J = D / 32;                 // 32-dim blocks: one 16-byte load a row and lane
  constexpr int PITCH = D + 32;             // bf16 a query row in shared memory
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ __align__(16) uint16_t qb[8 * NT * PITCH];
  __shared__ SelectShared sh;
  __shared__ uint16_t q_raw[GP * D];
  __shared__ float wmax[3][W];
  const CacheView& c = a.c;
  const int u = blockIdx.y, chunk = blockIdx.x;
  const int b = u / a.Hkv, h = u - b * a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = stream_length(c, b, a.max_len, chunk == 0 && h == 0, a.err);
  const int pages = (n + c.P - 1) / c.P;
  const int lo = a.keep_first, hi = pages - a.keep_last;  // the candidates
  const int t0 = chunk * a.chunk_pages;                   // this CTA's pages
  const bool work = pages > a.num_pages && t0 < hi && t0 + a.chunk_pages > lo;
  const int c_first = lo / a.chunk_pages;                 // the unit's first chunk with candidates
  if (work) {
    QueryPairs<D, GP, NTH> qp;
    qp.load(a, b, h, 1.f, sh.inv);
    for (int p = threadIdx.x; p < a.r / 2; p += NTH) sh.step[p] = a.rope_step[p];
    float* qf = reinterpret_cast<float*>(dyn + a.qf_off);  // [GP][D]
#pragma unroll
    for (int i = 0; i < qp.ITER; ++i) {
      const int g = qp.g0 + i * qp.STEP;
      if (g >= GP) break;
      const uint16_t h0 = f32_to_bf16(qp.v0[i]), h1 = f32_to_bf16(qp.v1[i]);
      qb[g * PITCH + qp.d0] = h0;
      qb[g * PITCH + qp.d1] = h1;
      qb[(GP + g) * PITCH + qp.d0] = f32_to_bf16(qp.v0[i] - bf16_to_f32(h0));
      qb[(GP + g) * PITCH + qp.d1] = f32_to_bf16(qp.v1[i] - bf16_to_f32(h1));
      q_raw[g * D + qp.d0] = qp.x[i];
      q_raw[g * D + qp.d1] = qp.y[i];
      qf[g * D + qp.d0] = qp.v0[i];
      qf[g * D + qp.d1] = qp.v1[i];
    }
    __syncthreads();
    // the largest query norm of the group, for the error bound
    if (chunk == c_first) {
      float best = 0.f;
      for (int g = warp; g < a.G; g += W) {
        float ss = 0.f;
        for (int d = lane; d < D; d += 32) ss = fmaf(qf[g * D + d], qf[g * D + d], ss);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
        best = fmaxf(best, nan_to_inf(ss));
      }
      if (lane == 0) wmax[0][warp] = best;
    }
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  if (!work) {
    if (chunk == 0 && pages <= a.num_pages) {
      // every page
      for (int i = threadIdx.x; i < a.num_pages; i += NTH) {
        const int64_t at = static_cast<int64_t>(u) * a.num_pages + i;
        if (i < pages) a.table[at] = c.block_table[static_cast<int64_t>(b) * c.bt_stride + i];
        if (a.selected) a.selected[at] = i < pages ? i : -1;
      }
    }
    return;
  }
  if (chunk == c_first && threadIdx.x == 0) {
    float best = 0.f;
    for (int w = 0; w < W; ++w) best = fmaxf(best, wmax[0][w]);
    a.qnorm[u] = sqrtf(best) * 1.001f + 8.7e-19f;  // (squares below the range)
  }
  uint32_t bq[NT][J][4];
  {
    const int col = lane >> 2, sub = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint4 w = *reinterpret_cast<const uint4*>(qb + (t * 8 + col) * PITCH + j * 32 + sub * 8);
        bq[t][j][0] = w.x;
        bq[t][j][1] = w.y;
        bq[t][j][2] = w.z;
        bq[t][j][3] = w.w;
      }
  }
  const int r0 = lane >> 2, sub = lane & 3;
  float* out = a.scores + static_cast<int64_t>(u) * a.pitch;
  float norm_max = 0.f, s_min = INFINITY, s_max = -INFINITY;
  const int t1 = min(t0 + a.chunk_pages, hi);
  for (int t = t0 + warp * 16; t < t1; t += W * 16) {
    if (t + 16 <= lo) continue;
    uint4 w[2][J];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int p = t + r0 + 8 * x;
      if (p >= lo && p < hi) {
        const int pg = physical_page(c, b, p, a.err);
        const uint16_t* src = a.summary + (static_cast<int64_t>(pg) * a.Hkv + h) * D + sub * 8;
#pragma unroll
        for (int j = 0; j < J; ++j) w[x][j] = *reinterpret_cast<const uint4*>(src + j * 32);
      } else {
#pragma unroll
        for (int j = 0; j < J; ++j) w[x][j] = make_uint4(0, 0, 0, 0);
      }
    }
    float acc[NT][4];
#pragma unroll
    for (int y = 0; y < NT; ++y) acc[y][0] = acc[y][1] = acc[y][2] = acc[y][3] = 0.f;
    __nv_bfloat162 sq[2];
    sq[0] = sq[1] = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint32_t a0[4] = {w[0][j].x, w[1][j].x, w[0][j].y, w[1][j].y};
      const uint32_t a1[4] = {w[0][j].z, w[1][j].z, w[0][j].w, w[1][j].w};
#pragma unroll
      for (int y = 0; y < NT; ++y) {
        mma_bf16(acc[y], a0, bq[y][j][0], bq[y][j][1]);
        mma_bf16(acc[y], a1, bq[y][j][2], bq[y][j][3]);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t v[4] = {w[x][j].x, w[x][j].y, w[x][j].z, w[x][j].w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&v[y]);
          sq[x] = __hfma2(m, m, sq[x]);
        }
      }
    }
    // norms: at most 64 bf16 additions of one lane, each off by 2^-9 of the sum
    // at most, so 1.25 covers them; squares below the range add 2^-60
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float ss = __low2float(sq[x]) + __high2float(sq[x]);
      ss += __shfl_xor_sync(kFull, ss, 1);
      ss += __shfl_xor_sync(kFull, ss, 2);
      norm_max = fmaxf(norm_max, nan_to_inf(ss));
    }
    // scores: column 2 sub, 2 sub + 1 of rows r0 and r0 + 8
    float s[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float v0 = acc[0][2 * x], v1 = acc[0][2 * x + 1];
      int g;
      if constexpr (NT == 1) {
        v0 += __shfl_xor_sync(kFull, v0, 2);
        v1 += __shfl_xor_sync(kFull, v1, 2);
        g = (2 * sub) & 3;
      } else {
        v0 += acc[NT - 1][2 * x];
        v1 += acc[NT - 1][2 * x + 1];
        g = 2 * sub;
      }
      // a score that is no number ranks first
      v0 = nan_to_inf(v0);
      v1 = nan_to_inf(v1);
      s[x] = fmaxf(g < a.G ? v0 : -INFINITY, g + 1 < a.G ? v1 : -INFINITY);
      s[x] = fmaxf(s[x], __shfl_xor_sync(kFull, s[x], 1));
      if constexpr (NT == 2) s[x] = fmaxf(s[x], __shfl_xor_sync(kFull, s[x], 2));
    }
    float tile_max = -INFINITY;
    if (sub < 2) {
      const int p = t + r0 + 8 * sub;
      if (p >= lo && p < hi) {
        const float x = sub ? s[1] : s[0];
        out[p] = x;
        s_min = fminf(s_min, x);
        s_max = fmaxf(s_max, x);
        tile_max = x;
      }
    }
    tile_max = warp_max(tile_max);
    if (lane == 0) a.tile_max[static_cast<int64_t>(u) * a.tile_pitch + (t >> 4)] = tile_max;
  }
  norm_max = warp_max(norm_max);
  s_max = warp_max(s_max);
  s_min = -warp_max(-s_min);
  __syncthreads();
  if (lane == 0) {
    wmax[0][warp] = norm_max;
    wmax[1][warp] = s_max;
    wmax[2][warp] = s_min;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < W; ++w) {
      norm_max = fmaxf(norm_max, wmax[0][w]);
      s_max = fmaxf(s_max, wmax[1][w]);
      s_min = fminf(s_min, wmax[2][w]);
    }
    float* info = a.cinfo + (static_cast<int64_t>(u) * a.chunks + chunk) * 3;
    info[0] = s_min;
    info[1] = s_max;
    info[2] = sqrtf(norm_max * 1.25f) + 8.7e-19f;  // 2^-60
  }
  // ---- the unit's last chunk selects
  if (!last_to_arrive(a.done + u, (hi - 1) / a.chunk_pages - c_first + 1, &sh.flag)) return;
  select_unit<D, NTH>(a, u, b, h, pages, q_raw, dyn, sh);
}

// ---------------------------------------------------------------- attention over the selected pages

// One CTA per (unit, split of its selected keys); a warp takes 16 keys of a page
// at a time, straight from memory into registers: nothing is shared between
// warps before the end.
//   S (16 keys x 8 heads)  = K (16 x D) . Q^T (D x 8)
//   O^T (D x 8 heads)     += V^T (D x 16) . P^T (16 x 8)
// on mma.sync m16n8k16 with fp32 sums. The sum over the dims may run in any
// order, so a lane's 16-byte load of a K row is its k-elements of two (E4M3:
// four) MMAs; a lane's 16 bytes of a V row, transposed 8 x 8 in registers, are
// rows of V^T in an order that only the final store has to know. Q and P are
// split into three bf16 terms (24 bits; K and V enter exactly); E4M3 is widened
// to fp16, with Q and P as two fp16 terms (22 bits, which fp16's range allows for
// P down to 2^-18: P is split at 2^15 times its value, so smaller weights lose at
// most 2^-40 each, of sums that are 1 or more). Terms are MMAs into the same
// accumulator.
// Few selected keys a unit: what counts is the chain of dependent steps, so
// there is no ring to fill, and q is rotated and split while the selection is
// still running.
// Bound by the keys' bytes where units are many: 64 ragged streams of 8 heads
// of 128, 32 pages of 16 tokens each, read 128 MB in the loop's 21 us (6.1
// TB/s) of 36 in all under ncu. With few units by the chain: 13 us at 1 x 5,003
// tokens, 15 at 1 x 1,048,576 (64 pages of 64), of which the loop is 3 - 5.
// Groups prefetched to the L2 cache ahead of the registers' changed nothing to
// speak of (64 ragged streams 47.4 - 54 us for 0 - 8 of them).
template <int D, bool F8>
struct AttendGeo {
  static constexpr int TERMS = F8 ? 2 : 3;
  static constexpr int J = F8 ? D / 64 : D / 32;      // 16-byte loads of a row and lane
  static constexpr int DPJ = F8 ? 64 : 32;            // dims of a quad's load
  static constexpr int PITCH = D + 32;                // 16-bit elements of a query row in shared memory: two rows'
                                                      // 64 bytes of a quad side by side in the banks
  static constexpr int QB = TERMS * 8 * PITCH * 2;    // bytes
  static constexpr int TILES = D / 16;                // M tiles of O^T
};

template <int D, bool F8>
__global__ void __launch_bounds__(kWarps * 32, D == 128 ? 4 : 2) page_attend_kernel(const PageArgs a) {
  using Gm = AttendGeo<D, F8>;
  constexpr int TERMS = Gm::TERMS, J = Gm::J, NTH = kWarps * 32, PO = D + 1;
  extern __shared__ __align__(16) uint8_t dyn[];
  uint16_t* qb = reinterpret_cast<uint16_t*>(dyn);       // [TERMS][8][PITCH]
  float* qf = reinterpret_cast<float*>(dyn + Gm::QB);    // [8][D], then the warps' outputs [kWarps][G][PO] (an odd
                                                         // pitch: a store's lanes hit 32 banks)
  __shared__ double inv_s[9];
  __shared__ float ms[kWarps + 1][8], ls[kWarps + 1][8];
  __shared__ float fw[kMaxSplits][8], lw[8];  // weights of the states that are joined, and their sums
  __shared__ uint16_t kn_s[D];
  __shared__ float vn_s[D];
  __shared__ int flag;
  const CacheView& c = a.c;
  const int u = blockIdx.x / a.splits, sp = blockIdx.x - u * a.splits;
  const int b = u / a.Hkv, h = u - b * a.Hkv, G = a.G;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int r0 = lane >> 2, sub = lane & 3;

  // ---- the query (base-2 scores) and, in split 0, the new token: its K entry
  // and value as they are stored
  float q_up = 1.f;  // E4M3: a power of two that brings the query to the top of the fp16 range, and back
  {
    QueryPairs<D, 8, NTH> qp;
    qp.load(a, b, h, a.q_scale, inv_s);
    float q_down = 1.f;
    if constexpr (F8) {
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < qp.ITER; ++i) mx = fmaxf(mx, fmaxf(fabsf(qp.v0[i]), fabsf(qp.v1[i])));
      mx = block_max<NTH>(mx, reinterpret_cast<int*>(&ms[0][0]));
      // 2^ex <= mx < 2^(ex + 1): the largest element comes to [2^14, 2^15), so that
      // the second term's last place, 2^-24, is 2^-38 of it or less and heads (and
      // dims) far below the largest keep their 22 bits too; both powers are normal
      // numbers
      const int ex = min(max(((__float_as_int(mx) >> 23) & 255) - 127, -112), 127);
      q_up = __int_as_float((127 + ex - 14) << 23);
      q_down = __int_as_float((127 - ex + 14) << 23);
    }
#pragma unroll
    for (int i = 0; i < qp.ITER; ++i) {
      const int g = qp.g0 + i * qp.STEP;
      if (g >= 8) break;
      float x0 = qp.v0[i], x1 = qp.v1[i];
      qf[g * D + qp.d0] = x0;
      qf[g * D + qp.d1] = x1;
      x0 *= q_down;
      x1 *= q_down;
#pragma unroll
      for (int y = 0; y < TERMS; ++y) {
        uint16_t* row = qb + (y * 8 + g) * Gm::PITCH;
        const uint32_t w = F8 ? pack_f16x2(x0, x1) : pack_bf16x2(x0, x1);
        row[qp.d0] = static_cast<uint16_t>(w);
        row[qp.d1] = static_cast<uint16_t>(w >> 16);
        if constexpr (F8) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
          x0 -= f.x;
          x1 -= f.y;
        } else {
          x0 -= bf16_lo(w);
          x1 -= bf16_hi(w);
        }
      }
    }
  }
  if (sp == 0) {
    const uint16_t* kn = a.k_new + static_cast<int64_t>(u) * D;
    const uint16_t* vn = a.v_new + static_cast<int64_t>(u) * D;
    if (a.k_norm) {
      if (warp == 0) {
        const double inv = qk_norm_inv(kn, D, a.norm_eps, lane);
        if (lane == 0) inv_s[8] = inv;
      }
      __syncthreads();
    }
    auto key = [&](int d) { return a.k_norm ? qk_norm_apply(kn[d], a.k_norm[d], inv_s[8]) : kn[d]; };
    const int half = a.r / 2;
    const int64_t pos = a.pos[b];
    for (int p = t; p < D / 2; p += NTH) {
      const int d0 = p < half ? p : a.r + 2 * (p - half);
      const int d1 = p < half ? p + half : d0 + 1;
      uint16_t x = key(d0), y = key(d1);
      if (p < half) {
        float cf, sf;
        rope_cos_sin(pos, a.rope_step[p], cf, sf);
        const uint32_t cb = __float_as_uint(cf), sb = __float_as_uint(sf);
        const uint16_t x1 = bf16_dot2(x, cb, y, sb ^ 0x80000000u);  // x c - y s
        y = bf16_dot2(y, cb, x, sb);                                // y c + x s
        x = x1;
      }
      kn_s[d0] = x;
      kn_s[d1] = y;
    }
    __syncthreads();
    for (int d = t; d < D; d += NTH) {
      float v = bf16_to_f32(vn[d]);
      if constexpr (F8) {
        // the stored bytes, and the values they stand for
        const uint8_t k8 = e4m3_of_quotient(bf16_to_f32(kn_s[d]), a.k_scale);
        const uint8_t v8 = e4m3_of_quotient(v, a.v_scale);
        kn_s[d] = static_cast<uint16_t>(k8 | (v8 << 8));
        v = e4m3_to_f32(v8);  // (v_scale is applied at the end)
      }
      vn_s[d] = v;
    }
    __syncthreads();
    for (int g = warp; g < G; g += kWarps) {
      float dot = 0.f;
      for (int d = lane; d < D; d += 32)
        dot = fmaf(qf[g * D + d], F8 ? e4m3_to_f32(static_cast<uint8_t>(kn_s[d] & 255)) : bf16_to_f32(kn_s[d]), dot);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
      if (lane == 0) {
        ms[kWarps][g] = dot;
        ls[kWarps][g] = 1.f;
      }
    }
  }
  const float gate_raw = a.gate && t < G ? bf16_to_f32(a.gate[static_cast<int64_t>(u) * G + t]) : 0.f;
  const int n = stream_length(c, b, a.max_len, false, a.err);
  const int pages = (n + c.P - 1) / c.P;
  const int m = min(pages, a.num_pages);       // selected pages; the last one holds the newest tokens
  const int gpp = (c.P + 15) / 16;             // 16-key groups of a page
  const int groups = m * gpp, stride = kWarps * a.splits;
  const int last_rows = n - (pages - 1) * c.P;
  __syncthreads();

  // the selection is the launch before's
  pdl_wait();
  pdl_trigger();
  const int32_t* table = a.table + static_cast<int64_t>(u) * a.num_pages;
  const int gi0 = sp * kWarps + warp;
  const int mine = gi0 < groups ? (groups - 1 - gi0) / stride + 1 : 0;  // groups of this warp
  float o[Gm::TILES][4];
#pragma unroll
  for (int i = 0; i < Gm::TILES; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float mrun[2] = {-INFINITY, -INFINITY}, lrun[2] = {0.f, 0.f};  // columns (heads) 2 sub, 2 sub + 1
  uint4 kw[2][J], vw[2][J];
  int my_pg = 0;
  // the pages of this warp's groups it .. it + 31, one per lane
  auto pages_of = [&](int it) {
    const int gi = gi0 + (it + lane) * stride;
    my_pg = 0;
    if (it + lane < mine) {
      my_pg = __ldcg(table + gi / gpp);
      if (my_pg < 0 || my_pg >= c.n_rows) {
        raise_error(a.err, ERR_INDEX);
        my_pg = 0;
      }
    }
  };
  // group `it`: its first row of the pools and its keys (none in a page's rows
  // past the last token)
  auto group_of = [&](int it, int64_t& row, int& valid) {
    const int gi = gi0 + it * stride;
    const int pi = gi / gpp, gr = gi - pi * gpp;
    valid = min(16, (pi == m - 1 ? last_rows : c.P) - gr * 16);
    row = (static_cast<int64_t>(__shfl_sync(kFull, my_pg, it & 31)) * a.Hkv + h) * c.P + gr * 16;
  };
  auto load = [&](const uint16_t* pool, int64_t row, int valid, uint4 (&w)[2][J]) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const bool in = r0 + 8 * x < valid;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(pool) + (row + r0 + 8 * x) * (D * (F8 ? 1 : 2)) + sub * 16;
#pragma unroll
      for (int j = 0; j < J; ++j) w[x][j] = in ? ld_stream(src + 64 * j) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  int64_t row = 0, row_next = 0;
  int valid = 0, valid_next = 0;
  if (mine > 0) {
    pages_of(0);
    group_of(0, row, valid);
    load(c.k, row, valid, kw);
    load(c.v, row, valid, vw);
  }
  for (int it = 0; it < mine; ++it) {
    const bool more = it + 1 < mine;
    if (more) {
      if (((it + 1) & 31) == 0) pages_of(it + 1);
      group_of(it + 1, row_next, valid_next);
    }
    // ---- scores, in independent chains of MMAs
    float sa[2 * TERMS][4];
#pragma unroll
    for (int x = 0; x < 2 * TERMS; ++x) sa[x][0] = sa[x][1] = sa[x][2] = sa[x][3] = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint32_t k0[4] = {kw[0][j].x, kw[0][j].y, kw[0][j].z, kw[0][j].w};
      const uint32_t k1[4] = {kw[1][j].x, kw[1][j].y, kw[1][j].z, kw[1][j].w};
      if constexpr (F8) {
        uint32_t af[4][4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          af[z][0] = e4m3x2_lo(k0[z]);
          af[z][1] = e4m3x2_lo(k1[z]);
          af[z][2] = e4m3x2_hi(k0[z]);
          af[z][3] = e4m3x2_hi(k1[z]);
        }
#pragma unroll
        for (int y = 0; y < TERMS; ++y) {
          const uint16_t* qp = qb + (y * 8 + r0) * Gm::PITCH + j * Gm::DPJ + sub * (Gm::DPJ / 4);
          const uint4 q0 = *reinterpret_cast<const uint4*>(qp), q1 = *reinterpret_cast<const uint4*>(qp + 8);
          mma_f16(sa[2 * y], af[0], q0.x, q0.y);
          mma_f16(sa[2 * y + 1], af[1], q0.z, q0.w);
          mma_f16(sa[2 * y], af[2], q1.x, q1.y);
          mma_f16(sa[2 * y + 1], af[3], q1.z, q1.w);
        }
      } else {
        const uint32_t a0[4] = {k0[0], k1[0], k0[1], k1[1]};
        const uint32_t a1[4] = {k0[2], k1[2], k0[3], k1[3]};
#pragma unroll
        for (int y = 0; y < TERMS; ++y) {
          const uint4 q0 =
              *reinterpret_cast<const uint4*>(qb + (y * 8 + r0) * Gm::PITCH + j * Gm::DPJ + sub * (Gm::DPJ / 4));
          mma_bf16(sa[2 * y], a0, q0.x, q0.y);
          mma_bf16(sa[2 * y + 1], a1, q0.z, q0.w);
        }
      }
    }
    if (more) load(c.k, row_next, valid_next, kw);  // in flight behind the softmax and P V
    float s[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      s[x] = 0.f;
#pragma unroll
      for (int y = 2 * TERMS - 1; y >= 0; --y) s[x] += sa[y][x];
      if constexpr (F8) s[x] *= q_up;
    }
    if (r0 >= valid) s[0] = s[1] = -INFINITY;
    if (r0 + 8 >= valid) s[2] = s[3] = -INFINITY;
    // ---- softmax over the keys, one column (head) at a time
    float p[4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float mx = fmaxf(s[x], s[2 + x]);
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, w));
      const float mnew = fmaxf(mrun[x], mx);
      const float ref = mnew == -INFINITY ? 0.f : mnew;  // (scores of -inf alone weigh nothing)
      const float al = exp2_fast(mrun[x] - ref);
      p[x] = exp2_fast(s[x] - ref);
      p[2 + x] = exp2_fast(s[2 + x] - ref);
      lrun[x] = fmaf(lrun[x], al, p[x] + p[2 + x]);
      if (al != 1.f) {
#pragma unroll
        for (int i = 0; i < Gm::TILES; ++i) {
          o[i][x] *= al;
          o[i][2 + x] *= al;
        }
      }
      mrun[x] = mnew;
    }
    // ---- P^T, in terms (E4M3: of 2^15 P, the largest power of two below the fp16
    // range; taken back exactly from the outputs)
    uint32_t pt[TERMS][2];
    if constexpr (F8) {
#pragma unroll
      for (int x = 0; x < 4; ++x) p[x] *= kWeightUp;
    }
#pragma unroll
    for (int y = 0; y < TERMS; ++y) {
      const uint32_t w0 = F8 ? pack_f16x2(p[0], p[1]) : pack_bf16x2(p[0], p[1]);
      const uint32_t w1 = F8 ? pack_f16x2(p[2], p[3]) : pack_bf16x2(p[2], p[3]);
      pt[y][0] = movm_t(w0);
      pt[y][1] = movm_t(w1);
      if (y + 1 < TERMS) {
        if constexpr (F8) {
          const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&w0));
          const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&w1));
          p[0] -= f0.x;
          p[1] -= f0.y;
          p[2] -= f1.x;
          p[3] -= f1.y;
        } else {
          p[0] -= bf16_lo(w0);
          p[1] -= bf16_hi(w0);
          p[2] -= bf16_lo(w1);
          p[3] -= bf16_hi(w1);
        }
      }
    }
    // ---- O^T
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint32_t v0[4] = {vw[0][j].x, vw[0][j].y, vw[0][j].z, vw[0][j].w};
      const uint32_t v1[4] = {vw[1][j].x, vw[1][j].y, vw[1][j].z, vw[1][j].w};
      if constexpr (F8) {
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const uint32_t af[4] = {movm_t(e4m3x2_lo(v0[z])), movm_t(e4m3x2_hi(v0[z])), movm_t(e4m3x2_lo(v1[z])),
                                  movm_t(e4m3x2_hi(v1[z]))};
#pragma unroll
          for (int y = 0; y < TERMS; ++y) mma_f16(o[4 * j + z], af, pt[y][0], pt[y][1]);
        }
      } else {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const uint32_t af[4] = {movm_t(v0[2 * z]), movm_t(v0[2 * z + 1]), movm_t(v1[2 * z]), movm_t(v1[2 * z + 1])};
#pragma unroll
          for (int y = 0; y < TERMS; ++y) mma_bf16(o[2 * j + z], af, pt[y][0], pt[y][1]);
        }
      }
    }
    if (more) {
      load(c.v, row_next, valid_next, vw);  // in flight behind the next group's scores
      row = row_next;
      valid = valid_next;
    }
  }

  // ---- the warps' states together, and the new token's
#pragma unroll
  for (int x = 0; x < 2; ++x) {
#pragma unroll
    for (int w = 4; w < 32; w <<= 1) lrun[x] += __shfl_xor_sync(kFull, lrun[x], w);
    if (r0 == 0) {
      ms[warp][2 * sub + x] = mrun[x];
      ls[warp][2 * sub + x] = lrun[x];
    }
  }
  __syncthreads();  // (qf is read no more)
#pragma unroll
  for (int i = 0; i < Gm::TILES; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int g = 2 * sub + (x & 1);
      // tile i's rows x / 2 * 8 + r0: which 16-bit pair (of a lane's 16 bytes)
      // and lane of the quad they came from
      const int j = i / (F8 ? 4 : 2), w = (i % (F8 ? 4 : 2)) * 2 + (x >> 1);
      const int d = j * Gm::DPJ + (r0 >> 1) * (Gm::DPJ / 4) + 2 * w + (r0 & 1);
      if (g < G) qf[(warp * G + g) * PO + d] = F8 ? o[i][x] * (1.f / kWeightUp) : o[i][x];
    }
  __syncthreads();
  const int parts = kWarps + (sp == 0 ? 1 : 0);
  // weights of `n` states (m and l of state w, head g at mp[w][g], lp[w][g]):
  // fw[w][g] = 2^(m - max m) and their sum of l; a warp per head
  auto weights = [&](int n, auto m_of, auto l_of, float* top) {
    for (int g = warp; g < G; g += kWarps) {
      float mw[kMaxSplits / 32], lv[kMaxSplits / 32], mm = -INFINITY;
#pragma unroll
      for (int x = 0; x < kMaxSplits / 32; ++x) {
        const int w = lane + 32 * x;
        mw[x] = w < n ? m_of(w, g) : -INFINITY;
        lv[x] = w < n ? l_of(w, g) : 0.f;
      }
#pragma unroll
      for (int x = 0; x < kMaxSplits / 32; ++x) mm = fmaxf(mm, mw[x]);
      mm = warp_max(mm);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float l = 0.f;
#pragma unroll
      for (int x = 0; x < kMaxSplits / 32; ++x) {
        const float f = exp2_fast(mw[x] - ref);
        if (lane + 32 * x < n) fw[lane + 32 * x][g] = f;
        l = fmaf(lv[x], f, l);
      }
#pragma unroll
      for (int w = 16; w >= 1; w >>= 1) l += __shfl_xor_sync(kFull, l, w);
      if (lane == 0) {
        lw[g] = l;
        if (top) top[g] = mm;
      }
    }
    __syncthreads();
  };
  const int64_t ps = (G * (D + 2) + 3) & ~3;  // floats of a partial state
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * ps;
  const bool single = a.splits == 1;
  // (the heads' factors: v_scale, the gate, 1 / sum)
  auto factors = [&]() {
    if (t < G) {
      float f = 1.f / lw[t];
      if constexpr (F8) f *= a.v_scale;
      if (a.gate) f /= 1.f + expf(-gate_raw);
      lw[t] = f;
    }
    __syncthreads();
  };
  float* dst = a.out + static_cast<int64_t>(u) * G * D;
  weights(parts, [&](int w, int g) { return ms[w][g]; }, [&](int w, int g) { return ls[w][g]; },
          single ? nullptr : part + G * D);
  if (single)
    factors();
  else if (t < G)
    part[G * D + G + t] = lw[t];
#pragma unroll 4
  for (int e = t; e < G * D; e += NTH) {
    const int g = e / D, d = e - g * D;
    float x = sp == 0 ? vn_s[d] * fw[kWarps][g] : 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x = fmaf(qf[(w * G + g) * PO + d], fw[w][g], x);
    if (single)
      dst[e] = x * lw[g];
    else
      part[e] = x;
  }
  // ---- the new entry into its slot: no key of it is read as valid by this
  // call, and masked rows' values are replaced by zeros. A stream whose length was
  // clamped has no slot: the one after the bound holds a token of it.
  if (sp == 0 && a.write_back && c.seq_len[b] == n) {
    const int pi = n / c.P;
    const int pg = pi < c.bt_stride ? c.block_table[static_cast<int64_t>(b) * c.bt_stride + pi] : -1;
    if (pg < 0 || pg >= c.n_rows) {
      if (t == 0) raise_error(a.err, ERR_INDEX);
    } else {
      const int64_t at = ((static_cast<int64_t>(pg) * a.Hkv + h) * c.P + n % c.P) * D;
      for (int d = t; d < D; d += NTH) {
        if constexpr (F8) {
          reinterpret_cast<uint8_t*>(c.k)[at + d] = static_cast<uint8_t>(kn_s[d] & 255);
          reinterpret_cast<uint8_t*>(c.v)[at + d] = static_cast<uint8_t>(kn_s[d] >> 8);
        } else {
          c.k[at + d] = kn_s[d];
          c.v[at + d] = a.v_new[static_cast<int64_t>(u) * D + d];
        }
      }
    }
  }
  if (single) return;
  // ---- the unit's last split joins them, in their order
  if (!last_to_arrive(a.counters + u, a.splits, &flag)) return;
  const float* p0 = a.part + static_cast<int64_t>(u) * a.splits * ps;
  // 4 elements a thread at a time, in the splits' order, BATCH of them in flight;
  // the first ones load while the weights are worked out
  constexpr int BATCH = 16;
  float4 y[BATCH];
  auto load_batch = [&](int e, int w0) {
#pragma unroll
    for (int w = 0; w < BATCH; ++w)
      y[w] = w0 + w < a.splits && e < G * D ? __ldcg(reinterpret_cast<const float4*>(p0 + (w0 + w) * ps + e))
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  load_batch(t * 4, 0);
  weights(a.splits, [&](int w, int g) { return __ldcg(p0 + w * ps + G * D + g); },
          [&](int w, int g) { return __ldcg(p0 + w * ps + G * D + G + g); }, nullptr);
  factors();
  for (int e = t * 4; e < G * D; e += NTH * 4) {
    const int g = e / D;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w0 = 0; w0 < a.splits; w0 += BATCH) {
#pragma unroll
      for (int w = 0; w < BATCH; ++w) {
        const float f = w0 + w < a.splits ? fw[w0 + w][g] : 0.f;
        x.x = fmaf(y[w].x, f, x.x);
        x.y = fmaf(y[w].y, f, x.y);
        x.z = fmaf(y[w].z, f, x.z);
        x.w = fmaf(y[w].w, f, x.w);
      }
      if (w0 + BATCH < a.splits)
        load_batch(e, w0 + BATCH);
      else
        load_batch(e + NTH * 4, 0);
    }
    const float f = lw[g];
    *reinterpret_cast<float4*>(dst + e) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
  }
}

}  // namespace

cudaError_t launch_summarize(const SummarizeArgs& a, int D, cudaStream_t s) {
  const int64_t pages = std::min<int64_t>((static_cast<int64_t>(a.max_tokens) + a.c.P - 1) / a.c.P, a.c.bt_stride);
  const dim3 grid(static_cast<unsigned>((pages * a.Hkv + 7) / 8), a.B);
  auto k = D == 128 ? (a.f8 ? summarize_kernel<128, true> : summarize_kernel<128, false>)
                    : (a.f8 ? summarize_kernel<256, true> : summarize_kernel<256, false>);
  return launch_pdl(k, grid, dim3(256), 0, s, a);
}

// Threads of the score and selection kernel: 16 warps for long streams, whose
// selection is one CTA's passes over all scores, 8 otherwise (more CTAs an SM).
// Calls with 8 / 16 warps: 1 x 1,048,576 tokens (16,384 pages) 27.4 / 25.3 us, 8
// x 262,144 (4,096) 40.2 / 39.3, E4M3 64 x 16,384 (1,024) 45.4 / 44.8, 64 ragged
// (up to 256) 49.4 / 61.5, 1 x 5,003 (313) 20.5 / 21.7.
static int select_threads(int pages) { return pages > 2048 ? 512 : 256; }

int page_chunk_pages(int units, int pages, int num_sms) {
  // Every CTA first rotates the group's queries, so: as many 16-page tiles a
  // warp as leave the grid within the 16 warps an SM that run at once (with 8 /
  // 16 / 32: 8 x 262,144 tokens 59.3 / 39.3 / 37.9 us, E4M3 64 x 16,384 49.0 /
  // 46.0 / 48.9, 1 x 1,048,576 116 / 25.4 / 25.7).
  const int threads = select_threads(pages), tile = threads / 2;
  const int64_t tiles = (pages + tile - 1) / tile;
  const int64_t ctas = std::max<int64_t>(1, static_cast<int64_t>(512 / threads) * num_sms / units);
  return tile * static_cast<int>(std::max<int64_t>(1, (tiles + ctas - 1) / ctas));
}

int page_splits(int units, int groups, int num_sms) {
  // A group a warp where there are few of them (one / two / four: 1 x 5,003
  // tokens 20.0 / 20.4 / 23.7 us, 1 x 1,048,576 25.4 / 25.5 / 28.3); no more CTAs
  // than run at once, two an SM at D = 256 (one / two / four: 8 x 262,144 tokens
  // 44.9 / 39.3 / 43.5 us, E4M3 64 x 16,384 56.4 / 46.0 / 51.6).
  int s = 2 * num_sms / units;
  s = std::min(s, (groups + kWarps - 1) / kWarps);
  return std::min(std::max(s, 1), kMaxSplits);
}

template <int NTH>
static cudaError_t select_launch(const PageArgs& a, int D, size_t smem, cudaStream_t s) {
  auto k = D == 128 ? (a.G <= 4 ? page_select_kernel<128, 1, NTH> : page_select_kernel<128, 2, NTH>)
                    : (a.G <= 4 ? page_select_kernel<256, 1, NTH> : page_select_kernel<256, 2, NTH>);
  static std::atomic<uint64_t> opted[4];
  const cudaError_t e = opt_in_smem(k, kSelectSmemMax, opted[(D == 128 ? 0 : 2) + (a.G <= 4 ? 0 : 1)]);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(a.chunks, a.B * a.Hkv), dim3(NTH), smem, s, a);
}

cudaError_t launch_page_select(PageArgs a, int D, cudaStream_t s) {
  const int pages = static_cast<int>((static_cast<int64_t>(a.max_len) + a.c.P - 1) / a.c.P);
  const size_t bits = (static_cast<size_t>(pages) + 31) / 32 * 4;
  a.q64_off = static_cast<int>((bits + 15) / 16 * 16);
  a.qf_off = a.q64_off + a.G * 8 * D;
  a.staged_off = a.qf_off + (a.G <= 4 ? 4 : 8) * 4 * D;
  a.staged = (std::min(pages, kStaged) + 127) / 128 * 128;
  size_t smem = a.staged_off + static_cast<size_t>(a.staged) * 4;
  if (pages <= a.num_pages) smem = 0;  // no stream has more pages than it may read
  if (smem > static_cast<size_t>(kSelectSmemMax)) return cudaErrorNotSupported;
  return select_threads(pages) == 512 ? select_launch<512>(a, D, smem, s) : select_launch<256>(a, D, smem, s);
}

template <int D, bool F8>
static cudaError_t attend_launch(const PageArgs& a, cudaStream_t s) {
  auto k = page_attend_kernel<D, F8>;
  // the query's terms, then its fp32 values or the warps' outputs
  const auto bytes = [](int G) { return AttendGeo<D, F8>::QB + std::max(8 * D, kWarps * G * (D + 1)) * 4; };
  static std::atomic<uint64_t> opted{0};
  const cudaError_t e = opt_in_smem(k, bytes(8), opted);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(a.B * a.Hkv * a.splits), dim3(kWarps * 32), bytes(a.G), s, a);
}

cudaError_t launch_page_attend(const PageArgs& a, int D, bool f8, cudaStream_t s) {
  if (D == 128) return f8 ? attend_launch<128, true>(a, s) : attend_launch<128, false>(a, s);
  return f8 ? attend_launch<256, true>(a, s) : attend_launch<256, false>(a, s);
}

}  // namespace dattn
