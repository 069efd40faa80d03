// Linear attention over prompts: the chunked form, on the 5th-generation tensor
// cores.
//
// A chunk of C = 64 tokens of one KV head, with S the state before it, n <= C
// its valid tokens and lam the head's decay (i, j: tokens of the chunk):
//   o_i = lam^(i+1) q_i S + sum_{j <= i} lam^(i-j) (q_i . k_j) v_j
//   S'  = lam^n S + sum_j lam^(n-1-j) k_j v_j^T
// as four products, each an fp32 sum in tensor memory:
//   A  = Q K^T          rows: 64 tokens x 2 query heads (or 1), columns: tokens
//   O1 = Q S            S as three bf16 terms (24 significant bits)
//   O2 = P V            P = A masked and decayed, as three bf16 terms, from tensor
//                       memory
//   dS = K^T W          W = lam^(n-1-j) v_j as three bf16 terms
// q, k and v are bf16 and enter exactly; the state itself stays in fp32, in
// registers. Three terms keep the operands' 24 bits, so that the error is that of
// fp32 sums: 2.7e-7 of the outputs' size (root mean squares; 5.4e-7 over 1 x 32,768
// tokens). With two (2^-17 of each operand) it was 2.8e-6, 11 to 14 times what the
// same products in fp32 leave, in 137 us for 1 x 32,768 tokens (161 now) and 177
// for 16 ragged prompts (216): a third more MMAs and terms, and S's third term in
// the place of a second Q tile and a second K, whose copies are now waited for.
//
// Work split. A unit is one (stream, KV head, slice): EB of the state's columns
// (all 128 at D = 128, 64 of 256 at D = 256: what S's terms leave room for in
// shared memory beside Q, K, V and W). Where units are many, or their streams
// short or alike, a CTA has one unit. Otherwise the heads' chunks are laid end to
// end and one CTA an SM takes an equal range of them, worked out on the device
// from the counts: a range begins and ends inside a unit, so a first kernel sums
// what each CTA's last unit contributes to the state (for the CTA after it), a
// second carries the states along, and the main kernel starts each range from
// its state. At D = 256 four CTAs have the same range, a slice each: they read
// the same Q and K at the same time (16 ragged prompts: 214 MB from memory; 671
// MB when each had a range of its own).
//
// Roles: 16 state warps (W, P, and the state: dS in, S's terms out), 8 row warps
// (the epilogue), one warp that copies (TMA, 128-byte swizzle) and one that
// issues the MMAs. The state warps' chain and the row warps' run beside one
// another; both end in tensor memory, which is full, so that the next chunk's Q S
// waits until the outputs are read. 832 threads leave 72 registers each, and the
// roles' loops are kept small: when they missed the instruction cache, that was
// 43% of the stalls. The MMA warp walks its loops as a whole: descriptors worked
// out by one thread took it 60 - 120 ns an MMA.
//
// Bound by a chunk's chain of dependent steps, not by a unit: 4.5 us a chunk at D =
// 128 and two query heads a KV head, 6.0 at D = 256 and four (two Q tiles). The
// state warps make W, P and S's terms one after another, and a Q tile is copied
// once Q S has read the one before; beside them the row warps' outputs. Tensor
// pipe 40% and 45% of the main pass; at the memory's rate the chunk's copies take
// 2.9 us at D = 128. 1 x 32,768 tokens, 16 / 8 heads of 128: 161 us, under ncu sums
// 36, scan 11, main 124 (503 MB of it from and to memory, 4.1 TB/s), partly beside
// one another. 16 streams of 512 - 4,096 tokens, 8 / 2 heads of 256: 216 us, 41,
// 10, 178.
//
// An infinity or no number in v would reach earlier tokens of its chunk (its
// weight in P is 0, and 0 times it is no number): the state warps replace it by
// 0 for P V, and the row warps give its column no number from its token on -
// what the recurrence makes of it, whose state column then holds infinities of
// either sign.
#include "linear.cuh"
#include "mma.cuh"
#include "tc.cuh"

namespace dattn {

namespace {

constexpr int C = kLinearChunk;
constexpr int kStateWarps = 16, kRowWarps = 8;
constexpr int kTmaWarp = 24, kMmaWarp = 25;
constexpr int kThreads = 832;
constexpr int kTerms = 3;      // bf16 terms of an fp32 operand
constexpr int kPieceCost = 1;  // a unit's share of a CTA's range, in chunks, besides its own

enum : int {
  B_KFULL,              // a chunk's K has landed
  B_KFREE,              // every MMA that reads it has completed
  B_VFULL,              // [2] the same for V
  B_VFREE = B_VFULL + 2,
  B_WREADY = B_VFREE + 2,  // W (and the zeroed rows of a short chunk) written
  B_SREADY,             // the state's terms written
  B_SFREE,              // every Q S of a chunk complete
  B_ADONE,              // Q K^T complete
  B_PREADY,             // P written
  B_ODONE,              // Q S and P V complete
  B_OFREE,              // ... and read
  B_DSDONE,             // K^T W complete
  B_FINAL,
  B_QFULL,              // [2] a Q tile has landed (an arrival for each two regions)
  B_QFREE = B_QFULL + 2,  // [2] the MMAs that read two regions of Q completed
  B_COUNT = B_QFREE + 2
};

template <int D>
struct Geo {
  static constexpr int EB = D == 128 ? 128 : 64;   // state columns of a CTA
  static constexpr int SLICES = D / EB;
  static constexpr int ER = EB / 64, DR = D / 64;  // 64-element regions
  static constexpr int DP = DR / 2;                // pairs of Q's regions: one tile, each pair handed back by itself
  static constexpr int VS = D == 128 ? 2 : 1;      // chunks of V
  static constexpr int Q_REGION = 16384;           // [128 rows][128 bytes]
  static constexpr int Q_PAIR = 2 * Q_REGION;
  static constexpr int K_TILE = DR * 8192;         // [region][64 rows][128 bytes]
  static constexpr int V_TILE = ER * 8192;
  static constexpr int S_PLANE = ER * D * 128;     // [region][D rows][128 bytes]
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + DP * Q_PAIR;
  static constexpr int V_OFF = K_OFF + K_TILE;
  static constexpr int W_OFF = V_OFF + VS * V_TILE;      // the terms, the largest first
  static constexpr int S_OFF = W_OFF + kTerms * V_TILE;  // the same
  static constexpr int BAR_OFF = S_OFF + kTerms * S_PLANE;
  static constexpr int MISC_OFF = BAR_OFF + 8 * B_COUNT;
  static constexpr int BAD_OFF = (MISC_OFF + 16 + 15) / 16 * 16;  // [2][EB]: 64 chunk + 63 - token of the first
                                                                  // token without a number in a column
  static constexpr int FLAG_OFF = BAD_OFF + 2 * EB * 4;           // [2] latest chunk with such a token
  static constexpr int SMEM = FLAG_OFF + 16 + 1024;               // (1024: alignment)
  // tensor memory columns, all 512. At D = 256 the products with S's terms have
  // their own columns: one MMA of N = 192 then does all three. P's first two terms
  // are beside A, the third is in A's place, each warp's 16 columns over what it
  // has read of A.
  static constexpr int T_A = 0, T_P = 64, T_O1 = 128, T_O2 = T_O1 + (D == 128 ? 128 : 192), T_DS = T_O2 + EB;
  static constexpr int T_COLS = 512;
  static_assert(T_DS + D / 128 * EB == T_COLS);
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

// A bounded wait that did not succeed at once (out of line: the roles' loops have
// to stay in the instruction cache).
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort, int* err, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > limit_ns) {
      *abort = 1;
      raise_error(err, ERR_TIMEOUT);
      return false;
    }
  }
}

struct Waiter {
  uint32_t bars;
  volatile int* abort;
  const LinearArgs& a;
  // Bounded wait by a whole warp or one thread; after a timeout (or when
  // another role gave up) every role leaves its loop.
  __device__ __forceinline__ bool wait(int b, uint32_t parity) const {
    return mbar_try_wait(bars + 8 * b, parity) || wait_on(bars + 8 * b, parity, abort, a.err, a.wait_ns);
  }
};

// 8 consecutive floats: one 32-byte store (a whole sector) where the array is
// aligned for it, two of 16 bytes otherwise.
__device__ __forceinline__ void st_8(float* p, const float (&x)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// Brings the box at element coordinates (x, y, z) of the tensor map to the L2 cache.
__device__ __forceinline__ void tma_prefetch_3d(const void* tmap, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(tmap), "r"(x), "r"(y),
               "r"(z)
               : "memory");
}

// Limit of the wait for copies that may or may not be in flight.
constexpr uint64_t kDrainNs = 1000000;

// Two floats in one instruction: a b + c and a b.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Two floats as three packed bf16 terms, each what the ones before it leave
// (differences are exact): 24 bits together.
__device__ __forceinline__ void split3(float2 x, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
  t0 = pack_bf16x2(x.x, x.y);
  x = fma2(make_float2(bf16_lo(t0), bf16_hi(t0)), make_float2(-1.f, -1.f), x);
  t1 = pack_bf16x2(x.x, x.y);
  x = fma2(make_float2(bf16_lo(t1), bf16_hi(t1)), make_float2(-1.f, -1.f), x);
  t2 = pack_bf16x2(x.x, x.y);
}
// Eight floats as 16 bytes of each term.
__device__ __forceinline__ void split3(const float (&x)[8], uint4 (&t)[kTerms]) {
  split3(make_float2(x[0], x[1]), t[0].x, t[1].x, t[2].x);
  split3(make_float2(x[2], x[3]), t[0].y, t[1].y, t[2].y);
  split3(make_float2(x[4], x[5]), t[0].z, t[1].z, t[2].z);
  split3(make_float2(x[6], x[7]), t[0].w, t[1].w, t[2].w);
}
// The same of eight bf16 values times w.
__device__ __forceinline__ void split3(uint4 y, float w, uint4 (&t)[kTerms]) {
  const float2 w2 = make_float2(w, w);
  split3(mul2(make_float2(bf16_lo(y.x), bf16_hi(y.x)), w2), t[0].x, t[1].x, t[2].x);
  split3(mul2(make_float2(bf16_lo(y.y), bf16_hi(y.y)), w2), t[0].y, t[1].y, t[2].y);
  split3(mul2(make_float2(bf16_lo(y.z), bf16_hi(y.z)), w2), t[0].z, t[1].z, t[2].z);
  split3(mul2(make_float2(bf16_lo(y.w), bf16_hi(y.w)), w2), t[0].w, t[1].w, t[2].w);
}

// The chunks of stream b (0, reported, for a row without a state or a count out
// of range).
__device__ __forceinline__ int stream_chunks(const LinearArgs& a, int b, bool report) {
  int n = a.count[b];
  if (n < 0 || n > a.T) {
    if (report) raise_error(a.err, ERR_INDEX);
    n = 0;
  }
  if (state_row(a, b, report) < 0) n = 0;
  return (n + C - 1) / C;
}

// A place in the (stream, KV head)s laid end to end: which of them, and chunk.
struct Place {
  int u, k;
};

// Where the i-th of NC groups of CTAs (one a slice) begins. `cum`: [B] inclusive
// sums over the streams of their heads' weights (chunks + kPieceCost each), in
// shared memory.
__device__ __forceinline__ Place range_start(const LinearArgs& a, const int* cum, int i, int NC) {
  const int HS = a.Hkv;
  const int64_t total = cum[a.B - 1];
  const int64_t t = total * i / NC;
  if (t >= total) return Place{a.B * HS, 0};
  int lo = 0, hi = a.B - 1;  // the stream that holds t: the first with cum > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] > t) hi = mid; else lo = mid + 1;
  }
  const int before = lo ? cum[lo - 1] : 0;
  const int w = (cum[lo] - before) / HS;
  const int off = static_cast<int>(t - before);
  const int r = off / w, k = off - r * w - kPieceCost;
  return Place{lo * HS + r, max(k, 0)};
}

// The streams' weights summed (see range_start), by a whole block of NT threads;
// returns whether the units are worth cutting. In chunks' times: uncut, the
// longest unit's chunks; cut, everything spread evenly, with 40% more for the
// sums and 2.5 chunks' time for what is launched between. Measured, cut / uncut:
// 16 streams of 512 - 4,096 tokens (128 units of 256) 216 / 350 us, 16 x 4,096
// 416 / 391, 4 x 512 (32 units of 128) 32.2 / 39.0, 1 x 32,768 (8) 160 / 1,973.
template <int NT>
__device__ __forceinline__ bool sum_weights(const LinearArgs& a, int* cum, int groups, bool report) {
  __shared__ int longest;
  if (threadIdx.x == 0) longest = 0;
  __syncthreads();
  for (int b = threadIdx.x; b < a.B; b += NT) {
    const int n = stream_chunks(a, b, report);
    cum[b] = n > 0 ? (n + kPieceCost) * a.Hkv : 0;
    atomicMax(&longest, n);
  }
  __syncthreads();
  block_scan_inclusive<NT>(cum, a.B);
  return static_cast<int64_t>(14) * cum[a.B - 1] / groups + 25 < static_cast<int64_t>(10) * longest;
}

// The pieces of a CTA's range: chunks [k0, k1) of a (stream, KV head); every
// role walks them.
struct Pieces {
  const LinearArgs& a;
  Place at, end;
  int slice;
  int b, h, k0, k1, count;
  bool last;  // the unit's last piece
  __device__ __forceinline__ bool next() {
    while (at.u < end.u || (at.u == end.u && at.k < end.k)) {
      const int u = at.u;
      b = u / a.Hkv;
      h = u - b * a.Hkv;
      const int n = stream_chunks(a, b, false);
      count = a.count[b];
      k0 = at.k;
      k1 = u == end.u ? min(n, end.k) : n;
      last = k1 == n;
      at = Place{u + 1, 0};
      if (k1 > k0) return true;
    }
    return false;
  }
};

// What the scan knows of a CTA's slot: the unit that goes on in the next CTA (-1:
// none), whether the slot holds a sum (1; 2 when it is from the unit's beginning)
// and the decay over its tokens as hi + lo. Behind the slots and their copies.
struct alignas(16) SlotNote {
  int unit, kind;
  float lam, lam_lo;
};
template <int D>
__device__ __forceinline__ SlotNote* slot_notes(const LinearArgs& a) {
  return reinterpret_cast<SlotNote*>(a.sums + static_cast<int64_t>(2) * a.ctas * D * Geo<D>::EB);
}
// Whether the sums gave up waiting: set by them, then moved on to the main pass by
// the scan.
template <int D>
__device__ __forceinline__ int* gave_up(const LinearArgs& a) {
  return reinterpret_cast<int*>(slot_notes<D>(a) + a.ctas);
}

// The main pass over a CTA's pieces.
template <int D>
__global__ void __launch_bounds__(kThreads, 1) linear_prompt_kernel(const __grid_constant__ LinearArgs a) {
  using Gm = Geo<D>;
  constexpr int EB = Gm::EB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bars = sbase + Gm::BAR_OFF;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Gm::MISC_OFF + 8);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = a.G, hpt = G > 1 ? 2 : 1;  // query heads of an M tile
  const int tiles = (G + hpt - 1) / hpt;

  // ---- the CTA's range (the counts and rows are the caller's)
  const int group = blockIdx.x / Gm::SLICES, slice = blockIdx.x - group * Gm::SLICES;
  Place begin{group, 0}, end{group + 1, 0};
  if (a.split) {
    int* cum = reinterpret_cast<int*>(smem);  // (before the copies)
    const int groups = a.ctas / Gm::SLICES, heads = a.B * a.Hkv;
    if (sum_weights<kThreads>(a, cum, groups, blockIdx.x == 0)) {
      begin = range_start(a, cum, min(group, groups), groups);
      end = range_start(a, cum, min(group + 1, groups), groups);
    } else {
      begin = Place{min(group, heads), 0};
      end = Place{min(group + 1, heads), 0};
    }
    __syncthreads();
  } else {
    stream_chunks(a, group / a.Hkv, group % a.Hkv == 0 && slice == 0 && threadIdx.x == 0);
  }
  const Pieces all{a, begin, end, slice};
  {
    Pieces p = all;
    if (!p.next()) {  // (the whole CTA)
      pdl_wait();
      return;
    }
  }

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < B_COUNT; ++i)
      mbar_init(bars + 8 * i, i == B_WREADY || i == B_SREADY || i == B_PREADY ? kStateWarps
                              : i == B_OFREE                                  ? kRowWarps
                              : i == B_QFULL || i == B_QFULL + 1              ? Gm::DP
                                                                              : 1);
    reinterpret_cast<int*>(smem + Gm::FLAG_OFF)[0] = reinterpret_cast<int*>(smem + Gm::FLAG_OFF)[1] = -1;
    for (int i = 0; i < 2 * EB; ++i) reinterpret_cast<int*>(smem + Gm::BAD_OFF)[i] = -1;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tc::alloc(sbase + Gm::MISC_OFF, Gm::T_COLS);
  fence_proxy_async_smem();  // (the sums lay where copies go)
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_wait();
  pdl_trigger();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Gm::MISC_OFF);
  const Waiter W{bars, abort_flag, a};
  auto warp_wait = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, W.wait(bar, parity)); };
  auto arrive = [&](int bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * bar);
  };

  if (warp == kTmaWarp) {
    // ================= copies =================
    if (lane == 0) {
      // (not evict-first: the other slices' CTAs read the same Q and K)
      uint64_t policy;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
      bool ok = true;
      int cc = 0, qp = 0;  // chunks and pairs of Q's regions so far
      Pieces p = all;
      while (ok && p.next()) {
        for (int k = p.k0; k < p.k1 && ok; ++k, ++cc) {
          const int tok = p.b * a.T + k * C;
          // Q has one place, so a tile's copy waits until the tile before is done with
          // it: its data come to the L2 cache meanwhile (8 prompts of 1,000 tokens, 24 /
          // 4 heads of 256, 148 us, 162 without; 16 ragged ones 217, 229; at D = 128,
          // where a copy is half as long, 163, 162)
          if constexpr (D == 256)
            if (cc > 0)
              for (int mt = 0; mt < tiles; ++mt)
                for (int r = 0; r < Gm::DR; ++r) tma_prefetch_3d(&a.tmap_q, 64 * r, p.h * G + mt * hpt, tok);
          {
            const int st = cc % Gm::VS;
            if (cc >= Gm::VS) ok = W.wait(B_VFREE + st, (cc / Gm::VS - 1) & 1);
            if (!ok) break;
            const uint32_t bar = bars + 8 * (B_VFULL + st);
            mbar_arrive_expect_tx(bar, Gm::V_TILE);
            for (int r = 0; r < Gm::ER; ++r)
              tma_load_3d(sbase + Gm::V_OFF + st * Gm::V_TILE + r * 8192, &a.tmap_v, p.slice * EB + 64 * r, p.h, tok,
                          bar, policy);
          }
          {
            if (cc > 0) ok = W.wait(B_KFREE, (cc - 1) & 1);
            if (!ok) break;
            const uint32_t bar = bars + 8 * B_KFULL;
            mbar_arrive_expect_tx(bar, Gm::K_TILE);
            for (int r = 0; r < Gm::DR; ++r)
              tma_load_3d(sbase + Gm::K_OFF + r * 8192, &a.tmap_k, 64 * r, p.h, tok, bar, policy);
          }
          for (int mt = 0; mt < tiles && ok; ++mt)
            for (int i = 0; i < Gm::DP; ++i, ++qp) {
              const int t = qp / Gm::DP;
              if (t > 0) ok = W.wait(B_QFREE + i, (t - 1) & 1);
              if (!ok) break;
              if (t == 0 && (a.debug_flags & kDebugWithholdQ)) continue;
              const uint32_t bar = bars + 8 * (B_QFULL + (t & 1)), dst = sbase + Gm::Q_OFF + i * Gm::Q_PAIR;
              mbar_arrive_expect_tx(bar, 2 * static_cast<uint32_t>(hpt) * 8192u);
              for (int r = 0; r < 2; ++r)
                tma_load_3d(dst + r * Gm::Q_REGION, &a.tmap_q, 64 * (2 * i + r), p.h * G + mt * hpt, tok, bar, policy);
            }
        }
      }
      // Copies still in flight exist only when a role gave up: they land
      // before the CTA exits. They are those of the chunks and the tile behind the
      // one that was not requested any more, or in part: a wait for a place's
      // release that ran out says nothing of the copy into it.
      if (*abort_flag) {
        for (int i = max(0, cc - Gm::VS); i <= cc; ++i)
          mbar_wait_bounded(bars + 8 * (B_VFULL + i % Gm::VS), (i / Gm::VS) & 1, kDrainNs);
        for (int i = max(0, cc - 1); i <= cc; ++i) mbar_wait_bounded(bars + 8 * B_KFULL, i & 1, kDrainNs);
        for (int t = max(0, qp / Gm::DP - 1); t <= qp / Gm::DP; ++t)
          mbar_wait_bounded(bars + 8 * (B_QFULL + (t & 1)), (t >> 1) & 1, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ================= MMA issue =================
    // (the whole warp walks the loops, so that descriptors stay in uniform
    // registers; one thread issues)
    {
      const bool lead = tc::elect();
      constexpr uint32_t id_a = tc::f16_idesc_ab(128, C, 1, false, false);
      constexpr uint32_t id_q = tc::f16_idesc_ab(128, D == 128 ? 128 : 192, 1, false, true);
      constexpr uint32_t id_o = tc::f16_idesc_ab(128, EB, 1, false, true);
      constexpr uint32_t id_s = tc::f16_idesc_ab(128, EB, 1, true, true);
      // A descriptor is a constant and the start address in 16-byte units.
      const uint64_t k_major = tc::sw128_desc(0, 16, 1024);
      const uint64_t mn_major = tc::sw128_desc(0, 8192, 1024);
      // S as an operand: at D = 128 one term's two regions of 64 value dims (N =
      // 128), at D = 256 the three terms' one region (N = 192). Sums take the small
      // terms first: they round as often as there are MMAs, by what is there then.
      const uint64_t s_major = tc::sw128_desc(0, D == 128 ? D * 128 : Gm::S_PLANE, 1024);
      auto at = [&](uint64_t desc, uint32_t addr) { return desc + (addr >> 4); };
      // dS = K^T W
      auto issue_ds = [&](uint32_t kt) {
#pragma unroll 1
        for (int m = 0; m < D / 128; ++m) {
          const uint64_t kd = at(mn_major, kt + m * 16384), wd = at(mn_major, sbase + Gm::W_OFF);
          const uint32_t d = tmem + Gm::T_DS + m * EB;
          if (lead)
#pragma unroll
            for (int x = kTerms - 1; x >= 0; --x)
#pragma unroll
              for (int kk = 0; kk < C / 16; ++kk)
                tc::mma(d, kd + 128 * kk, wd + 128 * kk + x * (Gm::V_TILE / 16), id_s, x < kTerms - 1 || kk > 0);
        }
        if (lead) tc::commit(bars + 8 * B_DSDONE);
        if (tiles == 1 && lead) tc::commit(bars + 8 * B_KFREE);
      };
      bool ok = true;
      int cc = 0, t = 0;  // chunks and Q tiles so far
      Pieces p = all;
      while (ok && p.next()) {
        for (int k = p.k0; k < p.k1 && ok; ++k, ++cc) {
          const int st = cc % Gm::VS;
          const uint32_t vt = sbase + Gm::V_OFF + st * Gm::V_TILE, kt = sbase + Gm::K_OFF;
          ok = warp_wait(B_KFULL, cc & 1);
          if (!ok) break;
          for (int mt = 0; mt < tiles && ok; ++mt, ++t) {
            // A = Q K^T (over the last tile's third term of P, so behind its P V)
            ok = (t == 0 || warp_wait(B_ODONE, (t - 1) & 1)) && warp_wait(B_QFULL + (t & 1), (t >> 1) & 1);
            if (!ok) break;
            tc::fence_after();
#pragma unroll 1
            for (int i = 0; i < Gm::DP; ++i) {
              const uint64_t qd = at(k_major, sbase + Gm::Q_OFF + i * Gm::Q_PAIR);
              const uint64_t kd = at(k_major, kt + i * 16384);
              if (lead)
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                  tc::mma(tmem + Gm::T_A, qd + (kk >> 2) * (Gm::Q_REGION / 16) + 2 * (kk & 3), kd + (kk >> 2) * 512 + 2 * (kk & 3),
                          id_a, i > 0 || kk > 0);
            }
            if (lead) tc::commit(bars + 8 * B_ADONE);
            // (dS went before)
            if (tiles > 1 && mt == tiles - 1 && lead) tc::commit(bars + 8 * B_KFREE);
            // At D = 128, where the outputs of the tile before are still being read,
            // dS goes first; at D = 256 last (16 ragged prompts 230 us, 246 first).
            // W comes with the chunk's zeroed rows, which P V wants too.
            if constexpr (D == 128)
              if (mt == 0) {
                ok = warp_wait(B_WREADY, cc & 1);
                if (!ok) break;
                tc::fence_after();
                issue_ds(kt);
              }
            // O1 = Q S
            ok = (mt > 0 || warp_wait(B_SREADY, cc & 1)) && (t == 0 || warp_wait(B_OFREE, (t - 1) & 1));
            if (!ok) break;
            tc::fence_after();
#pragma unroll 1
            for (int i = 0; i < Gm::DP; ++i) {
              const uint64_t qd = at(k_major, sbase + Gm::Q_OFF + i * Gm::Q_PAIR);
              const uint64_t sd = at(s_major, sbase + Gm::S_OFF + i * 16384);
              if (lead) {
#pragma unroll
                for (int x = D == 128 ? kTerms - 1 : 0; x >= 0; --x)
#pragma unroll
                  for (int kk = 0; kk < 8; ++kk)
                    tc::mma(tmem + Gm::T_O1, qd + (kk >> 2) * (Gm::Q_REGION / 16) + 2 * (kk & 3),
                            sd + 128 * kk + x * (Gm::S_PLANE / 16), id_q, i > 0 || kk > 0 || (D == 128 && x < kTerms - 1));
                tc::commit(bars + 8 * (B_QFREE + i));
              }
            }
            if (mt == tiles - 1 && lead) tc::commit(bars + 8 * B_SFREE);
            if constexpr (D == 256)
              if (mt == 0) {
                ok = warp_wait(B_WREADY, cc & 1);
                if (!ok) break;
                tc::fence_after();
              }
            // O2 = P V
            ok = warp_wait(B_PREADY, t & 1);
            if (!ok) break;
            tc::fence_after();
            const uint64_t vd = at(mn_major, vt);
            if (lead)
#pragma unroll
              for (int x = kTerms - 1; x >= 0; --x)
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk)
                  tc::mma_ts(tmem + Gm::T_O2, tmem + (x == 2 ? Gm::T_A + 16 * kk : Gm::T_P + 32 * x + 8 * kk),
                             vd + 128 * kk, id_o, x < kTerms - 1 || kk > 0);
            if (lead) tc::commit(bars + 8 * B_ODONE);
            if (mt == tiles - 1 && lead) tc::commit(bars + 8 * (B_VFREE + st));
            if constexpr (D == 256)
              if (mt == 0) issue_ds(kt);
          }
        }
      }
      // every MMA issued has completed before the tensor memory is freed
      if (lead) tc::commit(bars + 8 * B_FINAL);
      if (!mbar_wait_bounded(bars + 8 * B_FINAL, 0) && lead) raise_error(a.err, ERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp < kStateWarps) {
    // ================= state warps =================
    const int q4 = warp & 3, w4 = warp >> 2;  // lane quarter of tensor memory, column quarter
    const int r = 32 * q4 + lane;             // tensor memory lane
    // this thread's key dim (row of the state) and 32 value dims. (Its code is
    // unrolled over them; with 64, the roles' loops missed the instruction cache
    // on 43% of the stalled cycles.)
    const int sd = D == 128 ? r : 128 * (w4 >> 1) + r;
    const int se = D == 128 ? 32 * w4 : 32 * (w4 & 1);
    const uint32_t t_ds = tmem + (static_cast<uint32_t>(32 * q4) << 16) + Gm::T_DS + 32 * w4;
    int* bad = reinterpret_cast<int*>(smem + Gm::BAD_OFF);
    volatile int* bad_chunk = reinterpret_cast<volatile int*>(smem + Gm::FLAG_OFF);
    float S[32];
    // the state's terms as the B operand of Q S (value dims contiguous)
    auto store_s = [&]() {
      uint8_t* dst = smem + Gm::S_OFF + (D == 128 ? w4 >> 1 : 0) * (D * 128) + sd * 128;
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = S[8 * ch + e];
        uint4 y[kTerms];
        split3(x, y);
        const int off = (((w4 & 1) * 4 + ch) ^ (sd & 7)) << 4;
#pragma unroll
        for (int e = 0; e < kTerms; ++e) *reinterpret_cast<uint4*>(dst + e * Gm::S_PLANE + off) = y[e];
      }
      fence_proxy_async_smem();
      arrive(B_SREADY);
    };
    // P of a tile: 16 columns of A a warp, masked and decayed (pw: lam^0 .. lam^C)
    const int pi = min(hpt == 2 ? r >> 1 : r, C - 1);         // the row's token
    const int top = min((r | 31) >> (hpt - 1), C - 1);        // the last token of the warp's rows
    auto write_p = [&](int t, const float* pw) -> bool {
      // (Q K^T waited for P V of the tile before, which has read its P)
      if (!warp_wait(B_ADONE, t & 1)) return false;
      tc::fence_after();
      const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * q4) << 16);
#pragma unroll 1
      for (int j0 = 16 * w4; j0 < 16 * w4 + 16; j0 += 8) {
        uint32_t p0[4] = {0, 0, 0, 0}, p1[4] = {0, 0, 0, 0}, p2[4] = {0, 0, 0, 0};
        if (j0 <= top) {  // (some of the warp's rows reach these columns)
          uint32_t y[8];
          tc::ld8(lanes + Gm::T_A + j0, y);
          const int m = pi - j0;  // columns up to this one count
          float w[8];
#pragma unroll
          for (int jj = 0; jj < 8; ++jj) w[jj] = __ldg(pw + max(m - jj, 0));
          tc::wait_ld();
#pragma unroll
          for (int jj = 0; jj < 8; jj += 2)
            split3(mul2(make_float2(jj <= m ? __uint_as_float(y[jj]) : 0.f, jj + 1 <= m ? __uint_as_float(y[jj + 1]) : 0.f),
                        make_float2(w[jj], w[jj + 1])),
                   p0[jj >> 1], p1[jj >> 1], p2[jj >> 1]);
        }
        tc::st4(lanes + Gm::T_P + j0 / 2, p0);
        tc::st4(lanes + Gm::T_P + 32 + j0 / 2, p1);
        // (over columns of A that this warp has read, in this pass or the one before)
        tc::st4(lanes + Gm::T_A + 16 * w4 + (j0 & 8) / 2, p2);
      }
      tc::wait_st();
      tc::fence_before();
      arrive(B_PREADY);
      return true;
    };
    bool ok = true;
    int cc = 0, t = 0;
    Pieces p = all;
    while (ok && p.next()) {
      const float* pw = a.decay + static_cast<int64_t>(p.h) * kDecayStride;
      float* state = a.state + (static_cast<int64_t>(state_row(a, p.b, false)) * a.Hkv + p.h) * D * D +
                     static_cast<int64_t>(sd) * D + p.slice * EB + se;
      // a whole unit starts from the cache's state; inside one, from what the scan
      // left in the slot of the CTA before, and the first piece of a unit that
      // goes on from the scan's copy of the state (the CTA that ends the unit may
      // have stored the new one by now)
      const float* src = state;
      if (p.k0 > 0)
        src = a.sums + (static_cast<int64_t>(blockIdx.x - Gm::SLICES) * D + sd) * EB + se;
      else if (!p.last)
        src = a.sums + (static_cast<int64_t>(a.ctas + blockIdx.x) * D + sd) * EB + se;
      // (sums that gave up waiting: the call has failed, and the cache's states
      // stay as they are)
      const bool lost = a.split && __ldcg(gave_up<D>(a) + 1);
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 y = *reinterpret_cast<const float4*>(src + e);
        S[e] = y.x;
        S[e + 1] = y.y;
        S[e + 2] = y.z;
        S[e + 3] = y.w;
      }
      if (lost) {
        *abort_flag = 1;
        break;
      }
      // (the terms of the last piece are read no more)
      if (cc > 0 && !warp_wait(B_SFREE, (cc - 1) & 1)) break;
      store_s();
      for (int k = p.k0; k < p.k1 && ok; ++k, ++cc) {
        const int st = cc & 1;                  // (of the notes)
        const int n = min(C, p.count - k * C);  // valid tokens
        ok = warp_wait(B_VFULL + cc % Gm::VS, (cc / Gm::VS) & 1);
        if (!ok) break;
        // ---- W = lam^(n-1-j) v_j in terms; the rows past n become zeros in
        // V, W and K (a zero weight would not stop a NaN there)
        uint8_t* vt = smem + Gm::V_OFF + cc % Gm::VS * Gm::V_TILE;
        uint8_t* wt = smem + Gm::W_OFF;
#pragma unroll 1
        for (int off = threadIdx.x * 16; off < Gm::V_TILE; off += kStateWarps * 512) {
          const int j = (off >> 7) & (C - 1);
          uint4 y = *reinterpret_cast<const uint4*>(vt + off);
          if (j >= n) {
            y = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(vt + off) = y;
          }
          {
            const uint32_t mag = __vmaxu2(__vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu),
                                          __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu));
            if ((mag & 0xffffu) >= 0x7f80u || (mag >> 16) >= 0x7f80u) {
              // (rare) 0 in place of infinities and no numbers, and a note of the
              // first such token of the column (a later chunk's note is larger)
              uint16_t* e16 = reinterpret_cast<uint16_t*>(vt + off);
              for (int x = 0; x < 8; ++x)
                if ((e16[x] & 0x7f80u) == 0x7f80u) {
                  const int e = (off / 8192) * 64 + ((((off >> 4) & 7) ^ (j & 7)) << 3) + x;
                  atomicMax(bad + st * EB + e, cc * C + C - 1 - j);
                  e16[x] = 0;
                }
              bad_chunk[st] = cc;
            }
          }
          const float w = j < n ? __ldg(pw + n - 1 - j) : 0.f;
          uint4 z[kTerms];
          split3(y, w, z);
#pragma unroll
          for (int e = 0; e < kTerms; ++e) *reinterpret_cast<uint4*>(wt + e * Gm::V_TILE + off) = z[e];
        }
        if (n < C) {
          ok = warp_wait(B_KFULL, cc & 1);
          if (!ok) break;
          uint8_t* kt = smem + Gm::K_OFF;
          for (int off = threadIdx.x * 16; off < Gm::K_TILE; off += kStateWarps * 512)
            if (((off >> 7) & (C - 1)) >= n) *reinterpret_cast<uint4*>(kt + off) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        arrive(B_WREADY);
        // ---- the state: S = lam^n S + dS (lam^C with what fp32 drops of it)
        const float ln = __ldg(pw + n), ln_lo = n == C ? __ldg(pw + C + 2) : 0.f;
        ok = write_p(t++, pw) && warp_wait(B_DSDONE, cc & 1);
        if (!ok) break;
        tc::fence_after();
#pragma unroll
        for (int e0 = 0; e0 < 32; e0 += 16) {
          uint32_t y[16];
          tc::ld16(t_ds + e0, y);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 x = make_float2(S[e0 + e], S[e0 + e + 1]);
            const float2 z = fma2(x, make_float2(ln, ln),
                                  fma2(x, make_float2(ln_lo, ln_lo),
                                       make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1]))));
            S[e0 + e] = z.x;
            S[e0 + e + 1] = z.y;
          }
        }
        tc::fence_before();
        for (int mt = 1; mt < tiles && ok; ++mt) ok = write_p(t++, pw);
        if (ok && k + 1 < p.k1) {
          ok = warp_wait(B_SFREE, cc & 1);
          if (ok) store_s();
        }
      }
      if (ok && p.last && !*abort_flag) {
        float* dst = state;
        const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          float z[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) z[q] = S[e + q];
          st_8(dst + e, z, wide);
        }
      }
    }
  } else {
    // ================= row warps =================
    const int r = 32 * (warp & 3) + lane;  // tensor memory lane: row of the M tile
    const int w2 = (warp - kStateWarps) >> 2;  // half of the columns
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const int i = hpt == 2 ? r >> 1 : r;  // the row's token and head
    const int hd = hpt == 2 ? r & 1 : 0;
    const int* bad = reinterpret_cast<const int*>(smem + Gm::BAD_OFF);
    const volatile int* bad_chunk = reinterpret_cast<const volatile int*>(smem + Gm::FLAG_OFF);
    bool ok = true;
    int cc = 0, t = 0;
    Pieces p = all;
    while (ok && p.next()) {
      const float* gpw = a.decay + static_cast<int64_t>(p.h) * kDecayStride;
      const float row_decay = __ldg(gpw + min(i, C - 1) + 1);
      for (int k = p.k0; k < p.k1 && ok; ++k, ++cc) {
        const int n = min(C, p.count - k * C);
        for (int mt = 0; mt < tiles && ok; ++mt, ++t) {
          const int g = mt * hpt + hd;
          const bool store = i < n && g < G;
          const int64_t head =
              (static_cast<int64_t>(p.b) * a.T + k * C + i) * a.Hkv * G + static_cast<int64_t>(p.h) * G + g;
          const float gate = store && a.gate ? bf16_to_f32(a.gate[head]) : 0.f;
          // ---- epilogue
          float f = a.scale;
          if (a.gate) f /= 1.f + expf(-gate);
          const float f1 = f * row_decay;
          // Two lanes with two rows (a token's heads, or two tokens of one head): each
          // stores half of a step's columns of both, so that a store instruction is
          // in 16 rows, 64 bytes in each. (dst: of the even row; the odd one's is `next`
          // behind it.)
          const int odd_lane = lane & 1;
          const int64_t next = hpt == 2 ? D : static_cast<int64_t>(a.Hkv) * G * D;
          float* dst = a.out + head * D - odd_lane * next + p.slice * EB + 8 * odd_lane;
          const bool store0 = __shfl_sync(0xffffffffu, store, lane & ~1), store1 = __shfl_sync(0xffffffffu, store, lane | 1);
          const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
          ok = warp_wait(B_ODONE, t & 1);
          if (!ok) break;
          tc::fence_after();
          const bool odd = bad_chunk[cc & 1] == cc;
#pragma unroll 1
          for (int e0 = EB / 2 * w2; e0 < EB / 2 * (w2 + 1); e0 += 16) {
            uint32_t o1[16], o2[16];
            tc::ld16(tmem + lane_off + Gm::T_O1 + e0, o1);
            tc::ld16(tmem + lane_off + Gm::T_O2 + e0, o2);
            if constexpr (D == 256) {
              uint32_t lo[16];
              tc::ld16(tmem + lane_off + Gm::T_O1 + 64 + e0, lo);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o1[e] = __float_as_uint(__uint_as_float(o1[e]) + __uint_as_float(lo[e]));
              tc::ld16(tmem + lane_off + Gm::T_O1 + 128 + e0, lo);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o1[e] = __float_as_uint(__uint_as_float(o1[e]) + __uint_as_float(lo[e]));
            }
            tc::wait_ld();
            float z[16];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 y = fma2(make_float2(__uint_as_float(o1[e]), __uint_as_float(o1[e + 1])), make_float2(f1, f1),
                                    mul2(make_float2(__uint_as_float(o2[e]), __uint_as_float(o2[e + 1])), make_float2(f, f)));
              z[e] = y.x;
              z[e + 1] = y.y;
            }
            if (odd) {
              uint32_t mask = 0;
#pragma unroll 1
              for (int e = 0; e < 16; ++e) {
                const int x = bad[(cc & 1) * EB + e0 + e] - cc * C;
                if (x >= 0 && i >= C - 1 - x) mask |= 1u << e;
              }
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (mask >> e & 1) z[e] = __uint_as_float(0x7fffffffu);
            }
            // (the notes too are free then: their place is written again two chunks on,
            // after the next chunk's Q S)
            if (e0 + 16 == EB / 2 * (w2 + 1)) {
              tc::fence_before();
              arrive(B_OFREE);
            }
            float z0[8], z1[8];  // this lane's columns of the even row and of the odd one
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float other = __shfl_xor_sync(0xffffffffu, odd_lane ? z[e] : z[8 + e], 1);
              z0[e] = odd_lane ? other : z[e];
              z1[e] = odd_lane ? z[8 + e] : other;
            }
            if (store0) st_8(dst + e0, z0, wide);
            if (store1) st_8(dst + next + e0, z1, wide);
          }
        }
      }
    }
  }

  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, Gm::T_COLS);
  }
}

// ---------------------------------------------------------------- the sums

// What each CTA's last piece contributes to the state, if its unit goes on in the
// next CTA: K^T W over chunks (all full), in tensor memory over groups of up to
// kSumGroup of them - W's weights reach to the group's end - and from group to
// group in registers. The state warps make W, the rest is copies and MMAs; K, V
// and W are rings. 36 us under ncu at 1 x 32,768 tokens (127 MB, 3.5 TB/s), 41 at
// 16 ragged prompts: W's three terms, about a microsecond a chunk.
constexpr int kSumGroup = 4, kSumStages = 4;
constexpr int kSumThreads = (kStateWarps + 2) * 32;
enum : int { R_FULL, R_FREE = R_FULL + kSumStages, R_WREADY = R_FREE + kSumStages, R_WFREE = R_WREADY + 2,
             R_DONE = R_WFREE + 2, R_FINAL = R_DONE + 2, R_COUNT };

template <int D>
struct SumGeo {
  using Gm = Geo<D>;
  static constexpr int STAGE = Gm::K_TILE + Gm::V_TILE;
  static constexpr int W_OFF = kSumStages * STAGE;             // [2] the terms
  static constexpr int BAR_OFF = W_OFF + 2 * kTerms * Gm::V_TILE;
  static constexpr int MISC_OFF = BAR_OFF + 8 * R_COUNT;
  static constexpr int SMEM = MISC_OFF + 16 + 1024;
  static constexpr int ACC = D / 128 * Gm::EB;  // tensor memory columns of a group's sum, of which there are two
  static constexpr int T_COLS = 2 * ACC;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

template <int D>
__global__ void __launch_bounds__(kSumThreads, 1) linear_sums_kernel(const __grid_constant__ LinearArgs a) {
  using Gm = Geo<D>;
  using Sg = SumGeo<D>;
  constexpr int EB = Gm::EB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bars = sbase + Sg::BAR_OFF;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Sg::MISC_OFF + 8);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  int* cum = reinterpret_cast<int*>(smem);  // (before the copies)
  const int groups = a.ctas / Gm::SLICES, group = blockIdx.x / Gm::SLICES, slice = blockIdx.x - group * Gm::SLICES;
  const bool cut = sum_weights<kSumThreads>(a, cum, groups, false);
  const Place begin = cut ? range_start(a, cum, min(group, groups), groups) : Place{0, 0};
  const Place end = cut ? range_start(a, cum, min(group + 1, groups), groups) : Place{0, 0};
  const int k0 = begin.u == end.u ? begin.k : 0, chunks = end.k - k0;
  const int b = end.u / a.Hkv, h = end.u - b * a.Hkv;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) {
    SlotNote n{-1, 0, 0.f, 0.f};
    if (end.k > 0) {
      const double l = exp(static_cast<double>(a.log_decay[h]) * C * chunks);
      const float lam = static_cast<float>(l);
      n = SlotNote{end.u, chunks > 0 ? (k0 == 0 ? 2 : 1) : 0, lam, static_cast<float>(l - static_cast<double>(lam))};
    }
    slot_notes<D>(a)[blockIdx.x] = n;
  }
  if (end.k == 0 || chunks <= 0) return;  // (the whole CTA)
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < R_COUNT; ++i)
      mbar_init(bars + 8 * i, i == R_WREADY || i == R_WREADY + 1 ? kStateWarps / 2 : 1);
    fence_mbar_init();
  }
  if (warp == kStateWarps + 1) tc::alloc(sbase + Sg::MISC_OFF, Sg::T_COLS);
  fence_proxy_async_smem();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Sg::MISC_OFF);
  const Waiter W{bars, abort_flag, a};
  auto warp_wait = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, W.wait(bar, parity)); };

  if (warp == kStateWarps) {
    // ================= copies =================
    if (lane == 0) {
      const uint64_t policy = l2_evict_first_policy();
      int c = 0;
      for (; c < chunks; ++c) {
        const int st = c % kSumStages;
        if (c >= kSumStages && !W.wait(R_FREE + st, (c / kSumStages - 1) & 1)) break;
        const uint32_t bar = bars + 8 * (R_FULL + st), dst = sbase + st * Sg::STAGE;
        const int tok = b * a.T + (k0 + c) * C;
        if (c == 0 && (a.debug_flags & kDebugWithholdKV)) continue;
        mbar_arrive_expect_tx(bar, Sg::STAGE);
        for (int r = 0; r < Gm::DR; ++r) tma_load_3d(dst + r * 8192, &a.tmap_k, 64 * r, h, tok, bar, policy);
        for (int r = 0; r < Gm::ER; ++r)
          tma_load_3d(dst + Gm::K_TILE + r * 8192, &a.tmap_v, slice * EB + 64 * r, h, tok, bar, policy);
      }
      // (a role gave up: copies in flight land before the CTA exits)
      if (*abort_flag)
        for (int i = max(0, c - kSumStages); i < c; ++i)
          mbar_wait_bounded(bars + 8 * (R_FULL + i % kSumStages), (i / kSumStages) & 1, kDrainNs);
    }
    __syncwarp();
  } else if (warp == kStateWarps + 1) {
    // ================= MMA issue =================
    {
      const bool lead = tc::elect();
      constexpr uint32_t id_s = tc::f16_idesc_ab(128, EB, 1, true, true);
      const uint64_t mn_major = tc::sw128_desc(0, 8192, 1024);
      for (int c = 0; c < chunks; ++c) {
        const int st = c % kSumStages;
        if (!warp_wait(R_FULL + st, (c / kSumStages) & 1) || !warp_wait(R_WREADY + (c & 1), (c >> 1) & 1)) break;
        tc::fence_after();
        const uint32_t kt = sbase + st * Sg::STAGE, wt = sbase + Sg::W_OFF + (c & 1) * kTerms * Gm::V_TILE;
        const uint32_t d0 = tmem + ((c / kSumGroup) & 1) * Sg::ACC;
#pragma unroll 1
        for (int m = 0; m < D / 128; ++m) {
          const uint64_t kd = mn_major + ((kt + m * 16384) >> 4), wd = mn_major + (wt >> 4);
          const uint32_t d = d0 + m * EB;
          if (lead)
#pragma unroll
            for (int x = kTerms - 1; x >= 0; --x)
#pragma unroll
              for (int kk = 0; kk < C / 16; ++kk)
                tc::mma(d, kd + 128 * kk, wd + 128 * kk + x * (Gm::V_TILE / 16), id_s,
                        x < kTerms - 1 || kk > 0 || c % kSumGroup > 0);
        }
        if (lead) tc::commit(bars + 8 * (R_FREE + st));
        if (lead) tc::commit(bars + 8 * (R_WFREE + (c & 1)));
        if (lead && (c % kSumGroup == kSumGroup - 1 || c == chunks - 1))
          tc::commit(bars + 8 * (R_DONE + ((c / kSumGroup) & 1)));
      }
      if (lead) tc::commit(bars + 8 * R_FINAL);
      if (!mbar_wait_bounded(bars + 8 * R_FINAL, 0) && lead) {
        *abort_flag = 1;
        raise_error(a.err, ERR_TIMEOUT);
      }
    }
    __syncwarp();
  } else {
    // ================= state warps =================
    const int q4 = warp & 3, w4 = warp >> 2, r = 32 * q4 + lane;
    const int sd = D == 128 ? r : 128 * (w4 >> 1) + r;
    const int se = D == 128 ? 32 * w4 : 32 * (w4 & 1);
    const float* pw = a.decay + static_cast<int64_t>(h) * kDecayStride;
    const float lam = __ldg(pw + C), lam_lo = __ldg(pw + C + 2);
    float S[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) S[e] = 0.f;
    // S = lam^(its tokens) S + sum, for group g
    auto add = [&](int g) -> bool {
      if (!warp_wait(R_DONE + (g & 1), (g >> 1) & 1)) return false;
      tc::fence_after();
      for (int i = min(kSumGroup, chunks - g * kSumGroup); i > 0; --i)
#pragma unroll
        for (int e = 0; e < 32; ++e) S[e] = fmaf(S[e], lam, S[e] * lam_lo);
#pragma unroll
      for (int e0 = 0; e0 < 32; e0 += 16) {
        uint32_t y[16];
        tc::ld16(tmem + (static_cast<uint32_t>(32 * q4) << 16) + (g & 1) * Sg::ACC + 32 * w4 + e0, y);
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) S[e0 + e] += __uint_as_float(y[e]);
      }
      tc::fence_before();
      return true;
    };
    bool ok = true;
    int added = 0;  // groups
    for (int c = 0; c < chunks && ok; ++c) {
      const int st = c % kSumStages;
      // W: even chunks by one half of the warps, odd ones by the other, so that two
      // are on their way
      if ((c & 1) == warp >> 3) {
        const int after = min(kSumGroup - 1 - c % kSumGroup, chunks - 1 - c);  // chunks of the group behind this one
        float g = 1.f;
        for (int i = 0; i < after; ++i) g *= lam;
        ok = warp_wait(R_FULL + st, (c / kSumStages) & 1) && (c < 2 || warp_wait(R_WFREE + (c & 1), ((c >> 1) - 1) & 1));
        if (!ok) break;
        const uint8_t* vt = smem + st * Sg::STAGE + Gm::K_TILE;
        uint8_t* wt = smem + Sg::W_OFF + (c & 1) * kTerms * Gm::V_TILE;
#pragma unroll 2
        for (int off = (threadIdx.x & 255) * 16; off < Gm::V_TILE; off += kStateWarps / 2 * 512) {
          const uint4 y = *reinterpret_cast<const uint4*>(vt + off);
          const float w = __ldg(pw + C - 1 - ((off >> 7) & (C - 1))) * g;
          uint4 z[kTerms];
          split3(y, w, z);
#pragma unroll
          for (int e = 0; e < kTerms; ++e) *reinterpret_cast<uint4*>(wt + e * Gm::V_TILE + off) = z[e];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * (R_WREADY + (c & 1)));
      }
      // a group's sum once the next group is under way (its accumulator is written
      // again from the group after that, whose first MMA waits for W of a chunk
      // that either half makes after this)
      if (c % kSumGroup == 1 && c > kSumGroup) ok = add(added++);
    }
    for (; ok && added * kSumGroup < chunks; ++added) ok = add(added);
    float* dst = a.sums + (static_cast<int64_t>(blockIdx.x) * D + sd) * EB + se;
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
      float z[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) z[q] = S[e + q];
      st_8(dst + e, z, true);
    }
  }

  tc::fence_before();
  __syncthreads();
  if (warp == kStateWarps + 1) {
    tc::fence_after();
    tc::dealloc(tmem, Sg::T_COLS);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicOr(gave_up<D>(a), 1);
}

// The states at the CTAs' starts from their sums (and a copy of the state that
// a split unit starts from): the slot of a CTA whose last
// unit goes on holds its piece's own contribution, and then the state after it.
// The block row of the CTA that holds a unit's beginning carries the unit's state
// through the slots; one thread per 4 elements. Every chunk of these pieces is
// full.
template <int D>
__global__ void __launch_bounds__(256) linear_scan_kernel(const LinearArgs a) {
  using Gm = Geo<D>;
  constexpr int EB = Gm::EB;
  constexpr int64_t SLOT = static_cast<int64_t>(D) * EB;
  constexpr int SLOTS = 8;  // in flight
  extern __shared__ SlotNote note[];  // [NC]
  constexpr int SL = Gm::SLICES;
  const int c = blockIdx.y, NC = a.ctas, slice = c % SL;  // the CTA, and those after it on its slice
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && c == 0 && threadIdx.x == 0) {
    // what the sums say of this call, for its main pass; the next call's begin anew
    int* f = gave_up<D>(a);
    f[1] = f[0];
    f[0] = 0;
  }
  const SlotNote* notes = slot_notes<D>(a) + c;
  const SlotNote first = notes[0];
  if (first.kind != 2) return;
  const int u = first.unit, b = u / a.Hkv, h = u - b * a.Hkv;
  const int at = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int d = at / EB, e = at - d * EB;
  float4 s = *reinterpret_cast<const float4*>(
      a.state + ((static_cast<int64_t>(state_row(a, b, false)) * a.Hkv + h) * D + d) * D + slice * EB + e);
  for (int x = threadIdx.x; c + x * SL < NC; x += 256) note[x] = notes[x * SL];
  __syncthreads();
  *reinterpret_cast<float4*>(a.sums + (NC + c) * SLOT + at) = s;
  for (int x0 = 0; c + x0 * SL < NC && note[x0].unit == u; x0 += SLOTS) {
    float4 y[SLOTS];
#pragma unroll
    for (int x = 0; x < SLOTS; ++x)
      y[x] = c + (x0 + x) * SL < NC && note[x0 + x].unit == u && note[x0 + x].kind > 0
                 ? *reinterpret_cast<const float4*>(a.sums + (c + (x0 + x) * SL) * SLOT + at)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < SLOTS; ++x) {
      if (c + (x0 + x) * SL >= NC || note[x0 + x].unit != u) return;
      // (the decay of a slot without a sum is 1)
      const float lam = note[x0 + x].lam, lo = note[x0 + x].lam_lo;
      s.x = fmaf(s.x, lam, fmaf(s.x, lo, y[x].x));
      s.y = fmaf(s.y, lam, fmaf(s.y, lo, y[x].y));
      s.z = fmaf(s.z, lam, fmaf(s.z, lo, y[x].z));
      s.w = fmaf(s.w, lam, fmaf(s.w, lo, y[x].w));
      *reinterpret_cast<float4*>(a.sums + (c + (x0 + x) * SL) * SLOT + at) = s;
    }
  }
}

template <int D>
cudaError_t prompt_launches(const LinearArgs& a, int ctas, cudaStream_t s) {
  using Gm = Geo<D>;
  static std::atomic<uint64_t> opted[2];
  cudaError_t e = opt_in_smem(linear_prompt_kernel<D>, Gm::SMEM, opted[0]);
  if (e == cudaSuccess) e = opt_in_smem(linear_sums_kernel<D>, SumGeo<D>::SMEM, opted[1]);
  if (e != cudaSuccess) return e;
  if (a.split) {
    e = launch_pdl(linear_sums_kernel<D>, dim3(a.ctas), dim3(kSumThreads), SumGeo<D>::SMEM, s, a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(linear_scan_kernel<D>, dim3(D * Gm::EB / 1024, a.ctas), dim3(256), a.ctas * sizeof(SlotNote), s, a);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(linear_prompt_kernel<D>, dim3(ctas), dim3(kThreads), Gm::SMEM, s, a);
}

}  // namespace

cudaError_t launch_linear_prompt(const LinearArgs& args, int D, int num_sms, cudaStream_t s) {
  LinearArgs a = args;
  const int units = a.B * a.Hkv * (D == 128 ? Geo<128>::SLICES : Geo<256>::SLICES);
  const int chunks = (a.T + C - 1) / C;
  // Whether units are cut is decided on the device, from the counts (10 us where it
  // comes out against it); not even considered for short prompts (cut / uncut: 4 x
  // 330 tokens of 8 heads of 128 31.8 / 31.1 us, 4 x 256 30.9 / 23.6) nor with more
  // units than SMs, where it depends on how they even each other out (20 x 512 -
  // 2,048, 160 units: 139 / 146 us, 32 x 1,024: 162 / 146, 48 x 512 - 2,048: 276 /
  // 288, 64 x 16 - 4,096: 588 / 635).
  a.split = chunks > 6 && units <= num_sms;
  a.ctas = num_sms;
  const int ctas = a.split ? num_sms : units;
  return D == 128 ? prompt_launches<128>(a, ctas, s) : prompt_launches<256>(a, ctas, s);
}

}  // namespace dattn
