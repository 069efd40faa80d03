// Decode over selected pages: the page summaries, their scores against the new
// token's query and the selection. The attention over the selected pages is
// the decode kernel's, which reads a page table of its own for each (stream,
// KV head) unit.
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

#include "common.cuh"
#include "mma.cuh"
#include "qk_norm.cuh"

namespace dattn {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kSelectThreads = 1024;
constexpr int kList = 1024;   // pages near the border ranked in shared memory
constexpr int kBins = 1024;   // histogram bins of the threshold search

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

// ---------------------------------------------------------------- scores

// Screened scores. A warp takes 16 pages at a time as the rows of an
// m16n8k16 A operand. The sum over the dims may run in any order, so a lane's
// 16-byte load of a summary (8 dims) is its k-elements of two MMAs, without a
// trip through shared memory; the query's B operand uses the same order and
// stays in registers. Columns: the group's heads as bf16 hi and, 4 (or one
// 8-column tile) further, what is left as bf16 lo.
// Bound by reading the candidates' summaries once (D * 2 bytes a page and
// head); the squared norm that the error bound needs is one bf16x2 FMA a
// loaded word.
template <int D, int NT>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const PageScoreArgs a) {
  constexpr int GP = NT * 4;
  constexpr int J = D / 32;                 // 32-dim blocks: one 16-byte load a row and lane
  constexpr int PITCH = D + 8;              // bf16 a query row in shared memory
  __shared__ __align__(16) uint16_t qb[8 * NT * PITCH];
  __shared__ float qf[GP * D];
  __shared__ double inv_s[GP];
  __shared__ float wmax[kScoreWarps];
  const CacheView& c = a.c;
  const int u = blockIdx.y, chunk = blockIdx.x;
  const int b = u / a.Hkv, h = u - b * a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = stream_length(c, b, a.max_len, chunk == 0 && h == 0, a.err);
  const int pages = (n + c.P - 1) / c.P;
  const int lo = a.keep_first, hi = pages - a.keep_last;  // the candidates
  const int t0 = chunk * a.chunk_pages;                   // this CTA's pages
  const bool work = pages > a.num_pages && t0 < hi && t0 + a.chunk_pages > lo;
  if (work) {
    // the group's queries, normalised and rotated in fp32 (caller inputs: not
    // written by the launch before)
    const uint16_t* q = a.q + (static_cast<int64_t>(b) * a.Hkv + h) * a.G * D;
    if (a.q_norm) {
      for (int g = warp; g < a.G; g += kScoreWarps) {
        const double inv = qk_norm_inv(q + g * D, D, a.norm_eps, lane);
        if (lane == 0) inv_s[g] = inv;
      }
      __syncthreads();
    }
    const int half = a.r / 2;
    const int64_t pos = a.pos[b];
    for (int p = threadIdx.x; p < D / 2; p += kScoreThreads) {
      const int d0 = p < half ? p : a.r + 2 * (p - half);
      const int d1 = p < half ? p + half : d0 + 1;
      float cf = 1.f, sf = 0.f;
      if (p < half) rope_cos_sin(pos, a.rope_step[p], cf, sf);
      for (int g = 0; g < GP; ++g) {
        float v0 = 0.f, v1 = 0.f;
        if (g < a.G) {
          uint16_t x = q[g * D + d0], y = q[g * D + d1];
          if (a.q_norm) {
            x = qk_norm_apply(x, a.q_norm[d0], inv_s[g]);
            y = qk_norm_apply(y, a.q_norm[d1], inv_s[g]);
          }
          const float xf = bf16_to_f32(x), yf = bf16_to_f32(y);
          v0 = p < half ? fmaf(xf, cf, -yf * sf) : xf;
          v1 = p < half ? fmaf(yf, cf, xf * sf) : yf;
        }
        qf[g * D + d0] = v0;
        qf[g * D + d1] = v1;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < GP * D; e += kScoreThreads) {
      const int g = e / D, d = e - g * D;
      const float x = qf[e];
      const uint16_t hb = f32_to_bf16(x);
      qb[g * PITCH + d] = hb;
      qb[(GP + g) * PITCH + d] = f32_to_bf16(x - bf16_to_f32(hb));
    }
    // the largest query norm of the group, for the error bound
    if (chunk == max(lo, 0) / a.chunk_pages) {
      float best = 0.f;
      for (int g = warp; g < a.G; g += kScoreWarps) {
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
  if (!work) return;
  if (chunk == max(lo, 0) / a.chunk_pages && threadIdx.x == 0) {
    float best = 0.f;
    for (int w = 0; w < kScoreWarps; ++w) best = fmaxf(best, wmax[w]);
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
  for (int t = t0 + warp * 16; t < t1; t += kScoreWarps * 16) {
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
      v0 = v0 != v0 ? INFINITY : v0;
      v1 = v1 != v1 ? INFINITY : v1;
      s[x] = fmaxf(g < a.G ? v0 : -INFINITY, g + 1 < a.G ? v1 : -INFINITY);
      s[x] = fmaxf(s[x], __shfl_xor_sync(kFull, s[x], 1));
      if constexpr (NT == 2) s[x] = fmaxf(s[x], __shfl_xor_sync(kFull, s[x], 2));
    }
    if (sub < 2) {
      const int p = t + r0 + 8 * sub;
      if (p >= lo && p < hi) out[p] = sub ? s[1] : s[0];
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) norm_max = fmaxf(norm_max, __shfl_xor_sync(kFull, norm_max, o));
  __syncthreads();
  if (lane == 0) wmax[warp] = norm_max;
  __syncthreads();
  if (threadIdx.x == 0) {
    float best = 0.f;
    for (int w = 0; w < kScoreWarps; ++w) best = fmaxf(best, wmax[w]);
    a.cnorm[static_cast<int64_t>(u) * a.chunks + chunk] = sqrtf(best * 1.25f) + 8.7e-19f;  // 2^-60
  }
}

// ---------------------------------------------------------------- selection

// fp64 to an unsigned key of the same order (NaN above everything).
__device__ __forceinline__ uint64_t order_key(double x) {
  if (x != x) x = INFINITY;
  const uint64_t v = static_cast<uint64_t>(__double_as_longlong(x + 0.0));  // -0 as +0
  return (v >> 63) ? ~v : (v | 0x8000000000000000ull);
}

// Sum over the block, known to every thread (kSelectThreads threads; `buf`:
// 33 ints of shared memory).
__device__ __forceinline__ int block_sum(int x, int* buf) {
  x = __reduce_add_sync(kFull, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  return __reduce_add_sync(kFull, buf[threadIdx.x & 31]);
}

// One CTA per unit.
template <int D>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const PageSelectArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int hist[kBins];
  __shared__ int list[kList];
  __shared__ uint64_t list_key[kList];
  __shared__ int buf[33];
  __shared__ float fbuf[2][32];
  __shared__ int n_in, n_list, bin_s, above_s, inside_s;
  __shared__ double inv_s[8];
  const CacheView& c = a.c;
  const int u = blockIdx.x, t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int b = u / a.Hkv, h = u - b * a.Hkv;
  const int n = stream_length(c, b, a.max_len, false, a.err);
  const int pages = (n + c.P - 1) / c.P;
  const int W = a.num_pages + 1;
  int32_t* table = a.table + static_cast<int64_t>(u) * W;
  int32_t* sel = a.selected ? a.selected + static_cast<int64_t>(u) * a.num_pages : nullptr;
  const int words = (pages + 31) / 32;
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem);
  double* q64 = reinterpret_cast<double*>(smem + (static_cast<size_t>(a.max_words) * 4 + 15) / 16 * 16);

  pdl_wait();
  pdl_trigger();
  const int chosen = min(pages, a.num_pages);
  if (t == 0) {
    if (h == 0) a.seq_out[b] = n - (pages - chosen) * c.P;
    // the page that the new entry goes to when the cached ones are full
    if (n == pages * c.P)
      table[chosen] = pages < c.bt_stride ? c.block_table[static_cast<int64_t>(b) * c.bt_stride + pages] : -1;
  }
  if (pages <= a.num_pages) {
    for (int i = t; i < a.num_pages; i += kSelectThreads) {
      if (i < pages) table[i] = c.block_table[static_cast<int64_t>(b) * c.bt_stride + i];
      if (sel) sel[i] = i < pages ? i : -1;
    }
    return;
  }

  const int lo = a.keep_first, hi = pages - a.keep_last;
  const int k = a.num_pages - a.keep_first - a.keep_last;  // 0 <= k < hi - lo
  const float* sc = a.scores + static_cast<int64_t>(u) * a.pitch;
  for (int w = t; w < words; w += kSelectThreads) {
    uint32_t m = 0;
    for (int x = 0; x < 32; ++x) {
      const int p = w * 32 + x;
      if (p < pages && (p < lo || p >= hi)) m |= 1u << x;
    }
    bits[w] = m;
  }
  if (t == 0) n_in = n_list = 0;
  __syncthreads();

  if (k > 0) {
    // ---- the screened scores' range and error bound
    float mn = INFINITY, mx = -INFINITY, cn = 0.f;
    for (int p = lo + t; p < hi; p += kSelectThreads) {
      const float s = sc[p];
      mn = fminf(mn, s);
      mx = fmaxf(mx, s);
    }
    for (int x = lo / a.chunk_pages + t; x < a.chunks && x * a.chunk_pages < hi; x += kSelectThreads) {
      cn = fmaxf(cn, a.cnorm[static_cast<int64_t>(u) * a.chunks + x]);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      mn = fminf(mn, __shfl_xor_sync(kFull, mn, o));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      cn = fmaxf(cn, __shfl_xor_sync(kFull, cn, o));
    }
    if (lane == 0) {
      fbuf[0][warp] = mn;
      fbuf[1][warp] = mx;
      buf[warp] = __float_as_int(cn);
    }
    __syncthreads();
    mn = fbuf[0][lane];
    mx = fbuf[1][lane];
    cn = __int_as_float(buf[lane]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      mn = fminf(mn, __shfl_xor_sync(kFull, mn, o));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      cn = fmaxf(cn, __shfl_xor_sync(kFull, cn, o));
    }
    // Error of a screened score, relative to |q| |summary|: the tensor cores'
    // fp32 sums, D / 16 steps of 17 addends that may each lose 2^-23 of the
    // largest (D 2^-23 1.07 in all; what the lo terms add is 2^-9 of that), q
    // as two bf16 terms (2^-17) and the fp32 rotation (2^-20): below D 2^-22
    // for D >= 128. Sums below the fp32 range add 2^-100.
    const float e = fmaf(static_cast<float>(D) * 2.3841858e-7f * cn, a.qnorm[u], 7.9e-31f);
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
        auto bin_of = [&](float s) { return min(kBins - 1, static_cast<int>((s - a0) * inv)); };
        hist[t] = 0;
        __syncthreads();
        for (int p = lo + t; p < hi; p += kSelectThreads) {
          const float s = sc[p];
          if (s >= a0 && s <= a1) atomicAdd(&hist[bin_of(s)], 1);
        }
        __syncthreads();
        // counts above each bin: thread t holds bin kBins - 1 - t
        const int mine = hist[kBins - 1 - t];
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kFull, incl, o);
          if (lane >= o) incl += y;
        }
        if (lane == 31) buf[warp] = incl;
        __syncthreads();
        int before = lane < warp ? buf[lane] : 0;
        before = __reduce_add_sync(kFull, before);
        const int above = before + incl - mine;
        if (above < want && want <= above + mine) {
          bin_s = kBins - 1 - t;
          above_s = above;
          inside_s = mine;
        }
        if (t == 0) n_list = 0;
        __syncthreads();
        const int bin = bin_s, inside = inside_s;
        want -= above_s;
        float b0 = INFINITY, b1 = -INFINITY;  // the bin's own range
        for (int p = lo + t; p < hi; p += kSelectThreads) {
          const float s = sc[p];
          if (s >= a0 && s <= a1 && bin_of(s) == bin) {
            b0 = fminf(b0, s);
            b1 = fmaxf(b1, s);
            if (inside <= kList) list[atomicAdd(&n_list, 1)] = __float_as_int(s);
          }
        }
        __syncthreads();
        if (inside <= kList) {
          // the score with `want - 1` larger ones before it
          if (t < inside) {
            const float s = __int_as_float(list[t]);
            int more = 0, same = 0;
            for (int x = 0; x < inside; ++x) {
              const float y = __int_as_float(list[x]);
              more += y > s;
              same += y == s;
            }
            if (more < want && want <= more + same) fbuf[0][0] = s;  // equal scores write the same
          }
          __syncthreads();
          a0 = a1 = fbuf[0][0];
          __syncthreads();
          break;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
          b0 = fminf(b0, __shfl_xor_sync(kFull, b0, o));
          b1 = fmaxf(b1, __shfl_xor_sync(kFull, b1, o));
        }
        if (lane == 0) {
          fbuf[0][warp] = b0;
          fbuf[1][warp] = b1;
        }
        __syncthreads();
        b0 = fbuf[0][lane];
        b1 = fbuf[1][lane];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
          b0 = fminf(b0, __shfl_xor_sync(kFull, b0, o));
          b1 = fmaxf(b1, __shfl_xor_sync(kFull, b1, o));
        }
        a0 = b0;
        a1 = b1;
        __syncthreads();
      }
      up = __fadd_ru(a1, 2.f * e);
      dn = __fsub_rd(a0, 2.f * e);
      __syncthreads();
      if (t == 0) n_list = 0;
      __syncthreads();
    }
    // ---- in, out, or near the border
    for (int p = lo + t; p < hi; p += kSelectThreads) {
      const float s = sc[p];
      if (screened && s > up) {
        atomicOr(&bits[p >> 5], 1u << (p & 31));
        atomicAdd(&n_in, 1);
      } else if (!screened || s >= dn) {
        const int x = atomicAdd(&n_list, 1);
        if (x < kList) list[x] = p;
      }
    }
    __syncthreads();
    const int m = n_list, want = k - n_in;  // 1 <= want <= m
    auto near = [&](int p) {
      const float s = sc[p];
      return !screened || (s <= up && s >= dn);
    };
    if (want == m) {
      for (int p = lo + t; p < hi; p += kSelectThreads)
        if (near(p)) atomicOr(&bits[p >> 5], 1u << (p & 31));
    } else {
      // ---- exact scores of the pages near the border: q rotated in fp64
      const uint16_t* q = a.q + (static_cast<int64_t>(b) * a.Hkv + h) * a.G * D;
      if (a.q_norm) {
        if (warp < a.G) {
          const double inv = qk_norm_inv(q + warp * D, D, a.norm_eps, lane);
          if (lane == 0) inv_s[warp] = inv;
        }
        __syncthreads();
      }
      const int half = a.r / 2;
      const int64_t pos = a.pos[b];
      for (int i = t; i < a.G * (D / 2); i += kSelectThreads) {
        const int g = i / (D / 2), p = i - g * (D / 2);
        const int d0 = p < half ? p : a.r + 2 * (p - half);
        const int d1 = p < half ? p + half : d0 + 1;
        uint16_t x = q[g * D + d0], y = q[g * D + d1];
        if (a.q_norm) {
          x = qk_norm_apply(x, a.q_norm[d0], inv_s[g]);
          y = qk_norm_apply(y, a.q_norm[d1], inv_s[g]);
        }
        const double xd = bf16_to_f32(x), yd = bf16_to_f32(y);
        double cd = 1.0, sd = 0.0;
        // the phase in turns is an exact 64-bit fraction; signed, times 2 for
        // half turns: int64 -> 2^-63 of a half turn
        if (p < half)
          sincospi(static_cast<double>(static_cast<int64_t>(static_cast<uint64_t>(pos) * a.rope_step[p])) *
                       1.0842021724855044e-19,
                   &sd, &cd);
        q64[g * D + d0] = xd * cd - yd * sd;
        q64[g * D + d1] = yd * cd + xd * sd;
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
          double s = 0.0;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) s = fma(q64[g * D + lane + 32 * x], mv[x], s);
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
          if (s != s) s = INFINITY;
          best = s > best ? s : best;
        }
        return order_key(best);
      };
      if (m <= kList) {
        for (int x = warp; x < m; x += kSelectThreads / 32) {
          const uint64_t key = exact_key(list[x]);
          if (lane == 0) list_key[x] = key;
        }
        __syncthreads();
        if (t < m) {
          const uint64_t key = list_key[t];
          const int p = list[t];
          int before = 0;
          for (int x = 0; x < m; ++x) before += list_key[x] > key || (list_key[x] == key && list[x] < p);
          if (before < want) atomicOr(&bits[p >> 5], 1u << (p & 31));
        }
      } else {
        // many pages near the border (equal summaries, or values beyond the
        // fp32 range): their keys go to memory and the border is found bit by
        // bit, first of the keys, then of the page among equal keys
        uint64_t* keys = a.keys + static_cast<int64_t>(u) * a.pitch;
        for (int p = lo + warp; p < hi; p += kSelectThreads / 32) {
          if (!near(p)) continue;
          const uint64_t key = exact_key(p);
          if (lane == 0) keys[p] = key;
        }
        __syncthreads();
        uint64_t T = 0;
        for (int bit = 63; bit >= 0; --bit) {
          const uint64_t cand = T | (1ull << bit);
          int x = 0;
          for (int p = lo + t; p < hi; p += kSelectThreads) x += near(p) && keys[p] >= cand;
          if (block_sum(x, buf) >= want) T = cand;
        }
        int x = 0;
        for (int p = lo + t; p < hi; p += kSelectThreads) x += near(p) && keys[p] > T;
        const int ties = want - block_sum(x, buf);  // of the pages with key T, the lowest
        int step = 1;
        while (step < hi - lo) step <<= 1;
        int last = lo - 1;  // the largest page up to which fewer than `ties` of them lie
        for (; step >= 1; step >>= 1) {
          const int cand = last + step;
          if (cand >= hi) continue;
          int y = 0;
          for (int p = lo + t; p <= cand; p += kSelectThreads) y += near(p) && keys[p] == T;
          if (block_sum(y, buf) < ties) last = cand;
        }
        for (int p = lo + t; p < hi; p += kSelectThreads)
          if (near(p) && (keys[p] > T || (keys[p] == T && p <= last + 1))) atomicOr(&bits[p >> 5], 1u << (p & 31));
      }
    }
    __syncthreads();
  }

  // ---- the selected pages in ascending order
  int done = 0;
  for (int w0 = 0; w0 < words; w0 += kSelectThreads) {
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
    if (lane == 31) buf[warp] = incl;
    __syncthreads();
    const int all = __reduce_add_sync(kFull, buf[lane]);
    int at = done + __reduce_add_sync(kFull, lane < warp ? buf[lane] : 0) + incl - mine;
    while (m) {
      const int p = w * 32 + __ffs(m) - 1;
      m &= m - 1;
      if (at < a.num_pages) {
        table[at] = c.block_table[static_cast<int64_t>(b) * c.bt_stride + p];
        if (sel) sel[at] = p;
      }
      ++at;
    }
    done += all;
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

int score_chunk_pages(int units, int pages, int num_sms) {
  // One 16-page tile a warp; more where the grid then has over eight CTAs an
  // SM, for every CTA first rotates the group's queries.
  const int tile = kScoreWarps * 16;
  int per = 1;
  while (per < 8 && static_cast<int64_t>(units) * ((pages + tile * per - 1) / (tile * per)) > 8ll * num_sms) per *= 2;
  return tile * per;
}

cudaError_t launch_page_scores(const PageScoreArgs& a, int D, cudaStream_t s) {
  const dim3 grid(a.chunks, a.B * a.Hkv);
  auto k = D == 128 ? (a.G <= 4 ? score_kernel<128, 1> : score_kernel<128, 2>)
                    : (a.G <= 4 ? score_kernel<256, 1> : score_kernel<256, 2>);
  return launch_pdl(k, grid, dim3(kScoreThreads), 0, s, a);
}

cudaError_t launch_page_select(const PageSelectArgs& a, int D, cudaStream_t s) {
  const size_t smem = (static_cast<size_t>(a.max_words) * 4 + 15) / 16 * 16 + static_cast<size_t>(a.G) * D * 8;
  static std::atomic<uint64_t> opted[2];
  auto k = D == 128 ? select_kernel<128> : select_kernel<256>;
  const cudaError_t e = opt_in_smem(k, kSelectSmemMax, opted[D == 128 ? 0 : 1]);
  if (e != cudaSuccess) return e;
  if (smem > static_cast<size_t>(kSelectSmemMax)) return cudaErrorNotSupported;
  return launch_pdl(k, dim3(a.B * a.Hkv), dim3(kSelectThreads), smem, s, a);
}

}  // namespace dattn
