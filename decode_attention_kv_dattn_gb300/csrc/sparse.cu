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
constexpr int NT_ = 256;              // threads of every kernel here
constexpr int kWarps = NT_ / 32;
constexpr int kList = 1024;           // pages near the border ranked in shared memory
constexpr int kBins = 1024;           // histogram bins of the threshold search
constexpr int kStaged = 16384;        // scores held in shared memory during the selection

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

// A norm's square: infinite where it is no number, so that maxima keep it.
__device__ __forceinline__ float nan_to_inf(float x) { return x == x ? x : INFINITY; }

// ---------------------------------------------------------------- summaries

// One warp per (completed page, KV head): 16-byte loads, every lane the same
// dims of a few rows at a time, fp32 sums joined across the warp's row groups.
// Bound by reading the keys once; the page's rows of one head are contiguous.
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
  const int job = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int cnt = a.count[b], start = a.start_index[b];
  if (cnt < 0 || cnt > a.max_tokens || start < 0 || cnt > INT32_MAX - start) {
    if (job == 0 && lane == 0) raise_error(a.err, ERR_INDEX);
    return;
  }
  const int i = job / a.Hkv, h = job - i * a.Hkv;
  const int p = start / c.P + i;
  if (p >= (start + cnt) / c.P) return;
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

// The group's queries [G][D] in fp32, normalised, rotated and scaled, into
// qf[g * D + d]; heads G .. GP - 1 are zeros. Caller inputs only, so it runs
// before the wait for the launch before. Ends with a block barrier.
template <int D, int GP>
__device__ __forceinline__ void rotate_queries(const PageArgs& a, int b, int h, float scale, float* qf, double* inv_s) {
  const uint16_t* q = a.q + (static_cast<int64_t>(b) * a.Hkv + h) * a.G * D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (a.q_norm) {
    for (int g = warp; g < a.G; g += kWarps) {
      const double inv = qk_norm_inv(q + g * D, D, a.norm_eps, lane);
      if (lane == 0) inv_s[g] = inv;
    }
    __syncthreads();
  }
  const int half = a.r / 2;
  const int64_t pos = a.pos[b];
  for (int i = threadIdx.x; i < GP * (D / 2); i += NT_) {
    const int g = i / (D / 2), p = i - g * (D / 2);
    const int d0 = p < half ? p : a.r + 2 * (p - half);
    const int d1 = p < half ? p + half : d0 + 1;
    float v0 = 0.f, v1 = 0.f;
    if (g < a.G) {
      uint16_t x = q[g * D + d0], y = q[g * D + d1];
      if (a.q_norm) {
        x = qk_norm_apply(x, a.q_norm[d0], inv_s[g]);
        y = qk_norm_apply(y, a.q_norm[d1], inv_s[g]);
      }
      const float xf = bf16_to_f32(x), yf = bf16_to_f32(y);
      float cf = 1.f, sf = 0.f;
      if (p < half) rope_cos_sin(pos, a.rope_step[p], cf, sf);
      v0 = p < half ? fmaf(xf, cf, -yf * sf) : xf;
      v1 = p < half ? fmaf(yf, cf, xf * sf) : yf;
    }
    qf[g * D + d0] = v0 * scale;
    qf[g * D + d1] = v1 * scale;
  }
  __syncthreads();
}

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

// Block-wide sum, minimum and maximum, known to every thread (`buf`: kWarps
// words of shared memory).
__device__ __forceinline__ int block_sum(int x, int* buf) {
  x = __reduce_add_sync(kFull, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += buf[w];
  return s;
}
__device__ __forceinline__ float block_max(float x, int* buf) {
  x = warp_max(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = __float_as_int(x);
  __syncthreads();
  float s = __int_as_float(buf[0]);
#pragma unroll
  for (int w = 1; w < kWarps; ++w) s = fmaxf(s, __int_as_float(buf[w]));
  return s;
}

struct SelectShared {
  int hist[kBins];
  int list[kList];
  uint64_t list_key[kList];
  int buf[kWarps];
  int n_in, n_list, bin, above, inside;
  float threshold;
  double inv[8];
};

// The selection of one unit from its screened scores, by one CTA.
template <int D>
__device__ void select_unit(const PageArgs& a, int u, int b, int h, int n, int pages, uint8_t* dyn, SelectShared& s) {
  const CacheView& c = a.c;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int lo = a.keep_first, hi = pages - a.keep_last;
  const int k = a.num_pages - a.keep_first - a.keep_last;  // 0 <= k < hi - lo
  const int words = (pages + 31) / 32;
  uint32_t* bits = reinterpret_cast<uint32_t*>(dyn);
  double* q64 = reinterpret_cast<double*>(dyn + a.q64_off);
  const float* gsc = a.scores + static_cast<int64_t>(u) * a.pitch;
  const float* sc = gsc;
  for (int w = t; w < words; w += NT_) {
    // the pages kept for certain: below lo, from hi on
    uint32_t m = 0;
    const int p = w * 32;
    if (lo > p) m |= lo - p >= 32 ? ~0u : (1u << (lo - p)) - 1u;
    if (hi < p + 32) m |= hi <= p ? ~0u : ~0u << (hi - p);
    if (pages < p + 32) m &= (1u << (pages - p)) - 1u;
    bits[w] = m;
  }
  if (t == 0) s.n_in = s.n_list = 0;
  if (k > 0) {
    // ---- the screened scores' range and error bound
    float mn = INFINITY, mx = -INFINITY, cn = 0.f;
    if (hi - lo <= kStaged) {
      float* staged = reinterpret_cast<float*>(dyn + a.staged_off);
#pragma unroll 8
      for (int p = lo + t; p < hi; p += NT_) {
        const float x = __ldcg(gsc + p);
        staged[p - lo] = x;
        mn = fminf(mn, x);
        mx = fmaxf(mx, x);
      }
      sc = staged - lo;
    } else {
#pragma unroll 8
      for (int p = lo + t; p < hi; p += NT_) {
        const float x = __ldcg(gsc + p);
        mn = fminf(mn, x);
        mx = fmaxf(mx, x);
      }
    }
    for (int x = lo / a.chunk_pages + t; x < a.chunks && x * a.chunk_pages < hi; x += NT_)
      cn = fmaxf(cn, __ldcg(a.cnorm + static_cast<int64_t>(u) * a.chunks + x));
    mn = -block_max(-mn, s.buf);
    mx = block_max(mx, s.buf);
    cn = block_max(cn, s.buf);
    // Error of a screened score, relative to |q| |summary|: the tensor cores'
    // fp32 sums, D / 16 steps of 17 addends that may each lose 2^-23 of the
    // largest (D 2^-23 1.07 in all; what the lo terms add is 2^-9 of that), q
    // as two bf16 terms (2^-17) and the fp32 rotation (2^-20): below D 2^-22
    // for D >= 128. Sums below the fp32 range add 2^-100.
    const float e = fmaf(static_cast<float>(D) * 2.3841858e-7f * cn, __ldcg(a.qnorm + u), 7.9e-31f);
    // (a NaN or overflow anywhere makes e, mn or mx fail this)
    const bool screened = e < 1e36f && mx < 1e38f && mn > -1e38f;
    float up = INFINITY, dn = -INFINITY;  // in above up, out below dn
    if (screened) {
      // ---- the k-th largest screened score lies in [a0, a1]: narrowed by
      // histograms of equal value ranges until its bin holds at most kList
      // scores, which are then ranked
      float a0 = mn, a1 = mx;
      int want = k;
      for (int round = 0; round < 8; ++round) {
        const float inv = a1 > a0 ? static_cast<float>(kBins) / (a1 - a0) : 0.f;
        if (!(inv > 0.f && inv < 1e38f)) break;  // one value, or too narrow to cut
        auto bin_of = [&](float x) { return min(kBins - 1, static_cast<int>((x - a0) * inv)); };
        __syncthreads();
        for (int x = t; x < kBins; x += NT_) s.hist[x] = 0;
        if (t == 0) s.n_list = 0;
        __syncthreads();
#pragma unroll 8
        for (int p = lo + t; p < hi; p += NT_) {
          const float x = sc[p];
          if (x >= a0 && x <= a1) atomicAdd(&s.hist[bin_of(x)], 1);
        }
        __syncthreads();
        // counts above each bin, from the top: thread t holds 4 bins
        constexpr int BPT = kBins / NT_;
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
        int above = incl - mine;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) above += w < warp ? s.buf[w] : 0;
#pragma unroll
        for (int x = 0; x < BPT; ++x) {
          if (above < want && want <= above + own[x]) {
            s.bin = kBins - 1 - (t * BPT + x);
            s.above = above;
            s.inside = own[x];
          }
          above += own[x];
        }
        __syncthreads();
        const int bin = s.bin, inside = s.inside;
        want -= s.above;
        float b0 = INFINITY, b1 = -INFINITY;  // the bin's own range
#pragma unroll 8
        for (int p = lo + t; p < hi; p += NT_) {
          const float x = sc[p];
          if (x >= a0 && x <= a1 && bin_of(x) == bin) {
            b0 = fminf(b0, x);
            b1 = fmaxf(b1, x);
            if (inside <= kList) s.list[atomicAdd(&s.n_list, 1)] = __float_as_int(x);
          }
        }
        if (inside <= kList) {
          // the score with `want - 1` larger ones before it
          __syncthreads();
          for (int y = t; y < inside; y += NT_) {
            const float v = __int_as_float(s.list[y]);
            int more = 0, same = 0;
            for (int x = 0; x < inside; ++x) {
              const float w = __int_as_float(s.list[x]);
              more += w > v;
              same += w == v;
            }
            if (more < want && want <= more + same) s.threshold = v;  // equal scores write the same
          }
          __syncthreads();
          a0 = a1 = s.threshold;
          break;
        }
        a0 = -block_max(-b0, s.buf);
        a1 = block_max(b1, s.buf);
      }
      up = __fadd_ru(a1, 2.f * e);
      dn = __fsub_rd(a0, 2.f * e);
      __syncthreads();
      if (t == 0) s.n_list = 0;
    }
    __syncthreads();
    // ---- in, out, or near the border
    int in = 0;
#pragma unroll 8
    for (int p = lo + t; p < hi; p += NT_) {
      const float x = sc[p];
      if (screened && x > up) {
        atomicOr(&bits[p >> 5], 1u << (p & 31));
        ++in;
      } else if (!screened || x >= dn) {
        const int y = atomicAdd(&s.n_list, 1);
        if (y < kList) s.list[y] = p;
      }
    }
    const int want = k - block_sum(in, s.buf);  // 1 <= want <= m
    const int m = s.n_list;
    auto near = [&](int p) {
      const float x = sc[p];
      return !screened || (x <= up && x >= dn);
    };
    if (want == m) {
      if (m <= kList) {
        for (int x = t; x < m; x += NT_) atomicOr(&bits[s.list[x] >> 5], 1u << (s.list[x] & 31));
      } else {
        for (int p = lo + t; p < hi; p += NT_)
          if (near(p)) atomicOr(&bits[p >> 5], 1u << (p & 31));
      }
    } else {
      // ---- exact scores of the pages near the border: q rotated in fp64
      const uint16_t* q = a.q + (static_cast<int64_t>(b) * a.Hkv + h) * a.G * D;
      if (a.q_norm) {
        if (warp < a.G) {
          const double inv = qk_norm_inv(q + warp * D, D, a.norm_eps, lane);
          if (lane == 0) s.inv[warp] = inv;
        }
        __syncthreads();
      }
      const int half = a.r / 2;
      const int64_t pos = a.pos[b];
      for (int p = t; p < D / 2; p += NT_) {
        const int d0 = p < half ? p : a.r + 2 * (p - half);
        const int d1 = p < half ? p + half : d0 + 1;
        double cd = 1.0, sd = 0.0;
        // the phase in turns is an exact 64-bit fraction; signed, times 2 for
        // half turns: int64 -> 2^-63 of a half turn
        if (p < half)
          sincospi(static_cast<double>(static_cast<int64_t>(static_cast<uint64_t>(pos) * a.rope_step[p])) *
                       1.0842021724855044e-19,
                   &sd, &cd);
        for (int g = 0; g < a.G; ++g) {
          uint16_t x = q[g * D + d0], y = q[g * D + d1];
          if (a.q_norm) {
            x = qk_norm_apply(x, a.q_norm[d0], s.inv[g]);
            y = qk_norm_apply(y, a.q_norm[d1], s.inv[g]);
          }
          const double xd = bf16_to_f32(x), yd = bf16_to_f32(y);
          q64[g * D + d0] = xd * cd - yd * sd;
          q64[g * D + d1] = yd * cd + xd * sd;
        }
      }
      __syncthreads();
      auto exact_key = [&](int p) {  // by one warp
        const int pg = physical_page(c, b, p, a.err);
        const uint16_t* src = a.summary + (static_cast<int64_t>(pg) * a.Hkv + h) * D;
        double best = -INFINITY;
        double mv[D / 32];
#pragma unroll
        for (int x = 0; x < D / 32; ++x) mv[x] = bf16_to_f32(src[lane + 32 * x]);
        for (int g = 0; g < a.G; ++g) {
          double v = 0.0;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) v = fma(q64[g * D + lane + 32 * x], mv[x], v);
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
          if (v != v) v = INFINITY;
          best = v > best ? v : best;
        }
        return order_key(best);
      };
      if (m <= kList) {
        for (int x = warp; x < m; x += kWarps) {
          const uint64_t key = exact_key(s.list[x]);
          if (lane == 0) s.list_key[x] = key;
        }
        __syncthreads();
        for (int y = t; y < m; y += NT_) {
          const uint64_t key = s.list_key[y];
          const int p = s.list[y];
          int before = 0;
          for (int x = 0; x < m; ++x) before += s.list_key[x] > key || (s.list_key[x] == key && s.list[x] < p);
          if (before < want) atomicOr(&bits[p >> 5], 1u << (p & 31));
        }
      } else {
        // many pages near the border (equal summaries, or values beyond the
        // fp32 range): their keys go to memory and the border is found bit by
        // bit, first of the keys, then of the page among equal keys
        uint64_t* keys = a.keys + static_cast<int64_t>(u) * a.pitch;
        for (int p = lo + warp; p < hi; p += kWarps) {
          if (!near(p)) continue;
          const uint64_t key = exact_key(p);
          if (lane == 0) keys[p] = key;
        }
        __syncthreads();
        uint64_t T = 0;
        for (int bit = 63; bit >= 0; --bit) {
          const uint64_t cand = T | (1ull << bit);
          int x = 0;
          for (int p = lo + t; p < hi; p += NT_) x += near(p) && keys[p] >= cand;
          if (block_sum(x, s.buf) >= want) T = cand;
        }
        int x = 0;
        for (int p = lo + t; p < hi; p += NT_) x += near(p) && keys[p] > T;
        const int ties = want - block_sum(x, s.buf);  // of the pages with key T, the lowest
        int step = 1;
        while (step < hi - lo) step <<= 1;
        int last = lo - 1;  // the largest page up to which fewer than `ties` of them lie
        for (; step >= 1; step >>= 1) {
          const int cand = last + step;
          if (cand >= hi) continue;
          int y = 0;
          for (int p = lo + t; p <= cand; p += NT_) y += near(p) && keys[p] == T;
          if (block_sum(y, s.buf) < ties) last = cand;
        }
        for (int p = lo + t; p < hi; p += NT_)
          if (near(p) && (keys[p] > T || (keys[p] == T && p <= last + 1))) atomicOr(&bits[p >> 5], 1u << (p & 31));
      }
    }
  }
  __syncthreads();

  // ---- the selected pages in ascending order
  int32_t* table = a.table + static_cast<int64_t>(u) * a.num_pages;
  int32_t* sel = a.selected ? a.selected + static_cast<int64_t>(u) * a.num_pages : nullptr;
  int done = 0;
  for (int w0 = 0; w0 < words; w0 += NT_) {
    const int w = w0 + t;
    uint32_t m = w < words ? bits[w] : 0;
    const int mine = __popc(m);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) s.buf[warp] = incl;
    __syncthreads();
    int at = done + incl - mine;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      at += x < warp ? s.buf[x] : 0;
      done += s.buf[x];
    }
    while (m) {
      const int p = w * 32 + __ffs(m) - 1;
      m &= m - 1;
      if (at < a.num_pages) {
        table[at] = c.block_table[static_cast<int64_t>(b) * c.bt_stride + p];
        if (sel) sel[at] = p;
      }
      ++at;
    }
  }
  (void)n;
}

// Screened scores, and the selection by the CTA that finishes a unit's last
// chunk (a per-unit counter). A warp takes 16 pages at a time as the rows of an
// m16n8k16 A operand. The sum over the dims may run in any order, so a lane's
// 16-byte load of a summary (8 dims) is its k-elements of two MMAs, without a
// trip through shared memory; the query's B operand uses the same order and
// stays in registers. Columns: the group's heads as bf16 hi and, 4 (or one
// 8-column tile) further, what is left as bf16 lo.
// Bound by reading the candidates' summaries once (D * 2 bytes a page and
// head); the squared norm that the error bound needs is one bf16x2 FMA a
// loaded word.
template <int D, int NT>
__global__ void __launch_bounds__(NT_) page_select_kernel(const PageArgs a) {
  constexpr int GP = NT * 4;
  constexpr int J = D / 32;                 // 32-dim blocks: one 16-byte load a row and lane
  constexpr int PITCH = D + 8;              // bf16 a query row in shared memory
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ __align__(16) uint16_t qb[8 * NT * PITCH];
  __shared__ SelectShared sh;
  __shared__ float wmax[kWarps];
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
    float* qf = reinterpret_cast<float*>(dyn + a.q64_off);  // [GP][D] (the selection's fp64 query later)
    rotate_queries<D, GP>(a, b, h, 1.f, qf, sh.inv);
    for (int e = threadIdx.x; e < GP * D; e += NT_) {
      const int g = e / D, d = e - g * D;
      const float x = qf[e];
      const uint16_t hb = f32_to_bf16(x);
      qb[g * PITCH + d] = hb;
      qb[(GP + g) * PITCH + d] = f32_to_bf16(x - bf16_to_f32(hb));
    }
    // the largest query norm of the group, for the error bound
    if (chunk == c_first) {
      float best = 0.f;
      for (int g = warp; g < a.G; g += kWarps) {
        float ss = 0.f;
        for (int d = lane; d < D; d += 32) ss = fmaf(qf[g * D + d], qf[g * D + d], ss);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
        best = fmaxf(best, nan_to_inf(ss));
      }
      if (lane == 0) wmax[warp] = best;
    }
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  if (!work) {
    if (chunk == 0 && pages <= a.num_pages) {
      // every page
      for (int i = threadIdx.x; i < a.num_pages; i += NT_) {
        const int64_t at = static_cast<int64_t>(u) * a.num_pages + i;
        if (i < pages) a.table[at] = c.block_table[static_cast<int64_t>(b) * c.bt_stride + i];
        if (a.selected) a.selected[at] = i < pages ? i : -1;
      }
    }
    return;
  }
  if (chunk == c_first && threadIdx.x == 0) {
    float best = 0.f;
    for (int w = 0; w < kWarps; ++w) best = fmaxf(best, wmax[w]);
    a.qnorm[u] = sqrtf(best) * 1.001f;
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
  float norm_max = 0.f;
  const int t1 = min(t0 + a.chunk_pages, hi);
  for (int t = t0 + warp * 16; t < t1; t += kWarps * 16) {
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
    if (sub < 2) {
      const int p = t + r0 + 8 * sub;
      if (p >= lo && p < hi) out[p] = sub ? s[1] : s[0];
    }
  }
  norm_max = block_max(norm_max, sh.buf);
  // ---- the unit's last chunk selects
  if (threadIdx.x == 0)
    a.cnorm[static_cast<int64_t>(u) * a.chunks + chunk] = sqrtf(norm_max * 1.25f) + 8.7e-19f;  // 2^-60
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int all = (hi - 1) / a.chunk_pages - c_first + 1;
    sh.bin = atomicAdd(a.done + u, 1) == all - 1;
    if (sh.bin) a.done[u] = 0;
  }
  __syncthreads();
  const bool last = sh.bin != 0;
  __syncthreads();
  if (!last) return;
  __threadfence();
  select_unit<D>(a, u, b, h, n, pages, dyn, sh);
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
// to fp16, with Q and P as two fp16 terms (22 bits). Terms are MMAs into the
// same accumulator.
// Few selected keys a unit: what counts is the chain of dependent steps, so
// there is no ring to fill, and q is rotated and split while the selection is
// still running.
template <int D, bool F8>
struct AttendGeo {
  static constexpr int TERMS = F8 ? 2 : 3;
  static constexpr int J = F8 ? D / 64 : D / 32;      // 16-byte loads of a row and lane
  static constexpr int DPJ = F8 ? 64 : 32;            // dims of a quad's load
  static constexpr int PITCH = D + 8;                 // 16-bit elements of a query row in shared memory
  static constexpr int QB = TERMS * 8 * PITCH * 2;    // bytes
  static constexpr int TILES = D / 16;                // M tiles of O^T
};

template <int D, bool F8>
__global__ void __launch_bounds__(NT_) page_attend_kernel(const PageArgs a) {
  using Gm = AttendGeo<D, F8>;
  constexpr int TERMS = Gm::TERMS, J = Gm::J;
  extern __shared__ __align__(16) uint8_t dyn[];
  uint16_t* qb = reinterpret_cast<uint16_t*>(dyn);       // [TERMS][8][PITCH]
  float* qf = reinterpret_cast<float*>(dyn + Gm::QB);    // [8][D], then the warps' outputs [kWarps + 1][G][D]
  __shared__ double inv_s[9];
  __shared__ float ms[kWarps + 1][8], ls[kWarps + 1][8];
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
  rotate_queries<D, 8>(a, b, h, a.q_scale, qf, inv_s);
  float q_up = 1.f;  // E4M3: a power of two that brings the query into the fp16 range, and back
  if constexpr (F8) {
    float mx = 0.f;
    for (int e = t; e < G * D; e += NT_) mx = fmaxf(mx, fabsf(qf[e]));
    mx = block_max(mx, reinterpret_cast<int*>(&ms[0][0]));
    if (mx > 0.f && mx < 3e38f) {
      const int ex = ((__float_as_int(mx) >> 23) & 255) - 127;  // 2^ex <= mx
      q_up = ex > 126 ? 1.7014118e38f : (ex < -126 ? 1.1754944e-38f : __int_as_float((ex + 127) << 23));
    }
  }
  for (int e = t; e < 8 * D; e += NT_) {
    const int g = e / D, d = e - g * D;
    float x = qf[e];
    if constexpr (F8) {
      x /= q_up;
      const __half hi = __float2half_rn(x);
      qb[g * Gm::PITCH + d] = __half_as_ushort(hi);
      qb[(8 + g) * Gm::PITCH + d] = __half_as_ushort(__float2half_rn(x - __half2float(hi)));
    } else {
#pragma unroll
      for (int y = 0; y < TERMS; ++y) {
        const uint16_t w = f32_to_bf16(x);
        qb[(y * 8 + g) * Gm::PITCH + d] = w;
        x -= bf16_to_f32(w);
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
    for (int p = t; p < D / 2; p += NT_) {
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
    for (int d = t; d < D; d += NT_) {
      float v = bf16_to_f32(vn[d]);
      if constexpr (F8) {
        // the stored bytes, and the values they stand for
        const uint8_t k8 = e4m3_from_f64(static_cast<double>(bf16_to_f32(kn_s[d])) / static_cast<double>(a.k_scale));
        const uint8_t v8 = e4m3_from_f64(static_cast<double>(v) / static_cast<double>(a.v_scale));
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
  float o[Gm::TILES][4];
#pragma unroll
  for (int i = 0; i < Gm::TILES; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float mrun[2] = {-INFINITY, -INFINITY}, lrun[2] = {0.f, 0.f};  // columns (heads) 2 sub, 2 sub + 1
  for (int it0 = 0; gi0 + it0 * stride < groups; it0 += 32) {
    // the pages of this warp's next 32 groups, one per lane
    int my_pg = 0;
    {
      const int gi = gi0 + (it0 + lane) * stride;
      if (gi < groups) {
        my_pg = __ldcg(table + gi / gpp);
        if (my_pg < 0 || my_pg >= c.n_rows) {
          raise_error(a.err, ERR_INDEX);
          my_pg = 0;
        }
      }
    }
    for (int it = it0; it < it0 + 32; ++it) {
      const int gi = gi0 + it * stride;
      if (gi >= groups) break;
      const int pg = __shfl_sync(kFull, my_pg, it - it0);
      const int pi = gi / gpp, gr = gi - pi * gpp;
      const int valid = min(16, (pi == m - 1 ? last_rows : c.P) - gr * 16);
      if (valid <= 0) continue;
      const int64_t row = (static_cast<int64_t>(pg) * a.Hkv + h) * c.P + gr * 16;
      uint4 kw[2][J], vw[2][J];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bool in = r0 + 8 * x < valid;
        const int64_t off = ((row + r0 + 8 * x) * D + sub * (16 / (F8 ? 1 : 2))) * (F8 ? 1 : 2);
        const uint8_t* kp = reinterpret_cast<const uint8_t*>(c.k) + off;
        const uint8_t* vp = reinterpret_cast<const uint8_t*>(c.v) + off;
#pragma unroll
        for (int j = 0; j < J; ++j) kw[x][j] = in ? ld_stream(kp + 64 * j) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < J; ++j) vw[x][j] = in ? ld_stream(vp + 64 * j) : make_uint4(0u, 0u, 0u, 0u);
      }
      // ---- scores
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int y = 0; y < TERMS; ++y) {
          const uint16_t* qp = qb + (y * 8 + r0) * Gm::PITCH + j * Gm::DPJ + sub * (Gm::DPJ / 4);
          if constexpr (F8) {
            const uint4 q0 = *reinterpret_cast<const uint4*>(qp), q1 = *reinterpret_cast<const uint4*>(qp + 8);
            const uint32_t k0[4] = {kw[0][j].x, kw[0][j].y, kw[0][j].z, kw[0][j].w};
            const uint32_t k1[4] = {kw[1][j].x, kw[1][j].y, kw[1][j].z, kw[1][j].w};
            const uint32_t qq[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const uint32_t af[4] = {e4m3x2_lo(k0[z]), e4m3x2_lo(k1[z]), e4m3x2_hi(k0[z]), e4m3x2_hi(k1[z])};
              mma_f16(s, af, qq[2 * z], qq[2 * z + 1]);
            }
          } else {
            const uint4 q0 = *reinterpret_cast<const uint4*>(qp);
            const uint32_t a0[4] = {kw[0][j].x, kw[1][j].x, kw[0][j].y, kw[1][j].y};
            const uint32_t a1[4] = {kw[0][j].z, kw[1][j].z, kw[0][j].w, kw[1][j].w};
            mma_bf16(s, a0, q0.x, q0.y);
            mma_bf16(s, a1, q0.z, q0.w);
          }
        }
      }
      if constexpr (F8) {
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x] *= q_up;
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
      // ---- P^T, in terms
      uint32_t pt[TERMS][2];
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
      if (g < G) qf[(warp * G + g) * D + d] = o[i][x];
    }
  __syncthreads();
  const int parts = kWarps + (sp == 0 ? 1 : 0);
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * G * (D + 2);
  const bool single = a.splits == 1;
  auto store_out = [&](int g, int d, float x, float l) {
    x /= l;
    if constexpr (F8) x *= a.v_scale;
    const int64_t head = static_cast<int64_t>(u) * G + g;
    if (a.gate) x *= 1.f / (1.f + expf(-bf16_to_f32(a.gate[head])));
    a.out[head * D + d] = x;
  };
  for (int e = t; e < G * D; e += NT_) {
    const int g = e / D, d = e - g * D;
    float mm = -INFINITY;
    for (int w = 0; w < parts; ++w) mm = fmaxf(mm, ms[w][g]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float x = 0.f, l = 0.f;
    for (int w = 0; w < parts; ++w) {
      const float f = exp2_fast(ms[w][g] - ref);
      x = fmaf(w == kWarps ? vn_s[d] : qf[(w * G + g) * D + d], f, x);
      l = fmaf(ls[w][g], f, l);
    }
    if (single) {
      store_out(g, d, x, l);
    } else {
      part[g * D + d] = x;
      if (d == 0) {
        part[G * D + g] = mm;
        part[G * D + G + g] = l;
      }
    }
  }
  // ---- the new entry into its slot: no key of it is read as valid by this
  // call, and masked rows' values are replaced by zeros
  if (sp == 0 && a.write_back) {
    const int pi = n / c.P;
    const int pg = pi < c.bt_stride ? c.block_table[static_cast<int64_t>(b) * c.bt_stride + pi] : -1;
    if (pg < 0 || pg >= c.n_rows) {
      if (t == 0) raise_error(a.err, ERR_INDEX);
    } else {
      const int64_t at = ((static_cast<int64_t>(pg) * a.Hkv + h) * c.P + n % c.P) * D;
      for (int d = t; d < D; d += NT_) {
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
  __threadfence();
  __syncthreads();
  if (t == 0) {
    flag = atomicAdd(a.counters + u, 1) == a.splits - 1;
    if (flag) a.counters[u] = 0;
  }
  __syncthreads();
  if (!flag) return;
  __threadfence();
  const int64_t ps = static_cast<int64_t>(G) * (D + 2);
  const float* p0 = a.part + static_cast<int64_t>(u) * a.splits * ps;
  for (int e = t; e < G * D; e += NT_) {
    const int g = e / D, d = e - g * D;
    float mm = -INFINITY;
#pragma unroll 8
    for (int w = 0; w < a.splits; ++w) mm = fmaxf(mm, __ldcg(p0 + w * ps + G * D + g));
    float x = 0.f, l = 0.f;
#pragma unroll 8
    for (int w = 0; w < a.splits; ++w) {
      const float f = exp2_fast(__ldcg(p0 + w * ps + G * D + g) - mm);
      x = fmaf(__ldcg(p0 + w * ps + g * D + d), f, x);
      l = fmaf(__ldcg(p0 + w * ps + G * D + G + g), f, l);
    }
    store_out(g, d, x, l);
  }
}

}  // namespace

cudaError_t launch_summarize(const SummarizeArgs& a, int D, cudaStream_t s) {
  const int64_t jobs = (static_cast<int64_t>(a.max_tokens) + a.c.P - 1) / a.c.P * a.Hkv;
  const dim3 grid(static_cast<unsigned>((jobs + 7) / 8), a.B);
  auto k = D == 128 ? (a.f8 ? summarize_kernel<128, true> : summarize_kernel<128, false>)
                    : (a.f8 ? summarize_kernel<256, true> : summarize_kernel<256, false>);
  return launch_pdl(k, grid, dim3(256), 0, s, a);
}

int page_chunk_pages(int units, int pages, int num_sms) {
  // Every CTA first rotates the group's queries, so: as many 16-page tiles a
  // warp as leave the grid within the two CTAs an SM that run at once.
  const int tile = kWarps * 16;
  int64_t tiles = (pages + tile - 1) / tile;
  const int64_t ctas = std::max<int64_t>(1, 2ll * num_sms / units);
  return tile * static_cast<int>((tiles + ctas - 1) / ctas);
}

int page_splits(int units, int groups, int num_sms) {
  // a group a warp where there are few of them; no more CTAs than SMs
  int s = num_sms / units;
  s = std::min(s, (groups + kWarps - 1) / kWarps);
  return std::max(s, 1);
}

cudaError_t launch_page_select(PageArgs a, int D, cudaStream_t s) {
  const int pages = (a.max_len + a.c.P - 1) / a.c.P;
  size_t off = (static_cast<size_t>(pages) + 31) / 32 * 4;
  a.q64_off = static_cast<int>((off + 15) / 16 * 16);
  off = a.q64_off + static_cast<size_t>(std::max(a.G * 8, (a.G <= 4 ? 4 : 8) * 4)) * D;
  a.staged_off = static_cast<int>((off + 15) / 16 * 16);
  off = a.staged_off + static_cast<size_t>(std::min(pages, kStaged)) * 4;
  if (pages <= a.num_pages) off = 0;  // no stream has more pages than it may read
  if (off > static_cast<size_t>(kSelectSmemMax)) return cudaErrorNotSupported;
  auto k = D == 128 ? (a.G <= 4 ? page_select_kernel<128, 1> : page_select_kernel<128, 2>)
                    : (a.G <= 4 ? page_select_kernel<256, 1> : page_select_kernel<256, 2>);
  static std::atomic<uint64_t> opted[4];
  const cudaError_t e = opt_in_smem(k, kSelectSmemMax, opted[(D == 128 ? 0 : 2) + (a.G <= 4 ? 0 : 1)]);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(a.chunks, a.B * a.Hkv), dim3(NT_), off, s, a);
}

template <int D, bool F8>
static cudaError_t attend_launch(const PageArgs& a, cudaStream_t s) {
  auto k = page_attend_kernel<D, F8>;
  // the query's terms, then its fp32 values or the warps' outputs
  const auto bytes = [](int G) { return AttendGeo<D, F8>::QB + std::max(8, kWarps * G) * D * 4; };
  static std::atomic<uint64_t> opted{0};
  const cudaError_t e = opt_in_smem(k, bytes(8), opted);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(a.B * a.Hkv * a.splits), dim3(NT_), bytes(a.G), s, a);
}

cudaError_t launch_page_attend(const PageArgs& a, int D, bool f8, cudaStream_t s) {
  if (D == 128) return f8 ? attend_launch<128, true>(a, s) : attend_launch<128, false>(a, s);
  return f8 ? attend_launch<256, true>(a, s) : attend_launch<256, false>(a, s);
}

}  // namespace dattn
