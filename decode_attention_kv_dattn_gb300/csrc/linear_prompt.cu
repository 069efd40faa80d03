// Linear attention over prompts: the chunked form, on the 5th-generation tensor
// cores.
//
// A chunk of C = 64 tokens of one KV head, with S the state before it, n <= C
// its valid tokens and lam the head's decay (i, j: tokens of the chunk):
//   o_i = lam^(i+1) q_i S + sum_{j <= i} lam^(i-j) (q_i . k_j) v_j
//   S'  = lam^n S + sum_j lam^(n-1-j) k_j v_j^T
// as four products, each an fp32 sum in tensor memory:
//   A  = Q K^T          rows: 64 tokens x 2 query heads (or 1), columns: tokens
//   O1 = Q S            S as two bf16 terms (hi + lo: 16 significant bits)
//   O2 = P V            P = A masked and decayed, as two bf16 terms, from tensor
//                       memory
//   dS = K^T W          W = lam^(n-1-j) v_j as two bf16 terms
// q, k and v are bf16 and enter exactly; the state itself stays in fp32, in
// registers.
//
// Work split. A CTA has one (stream, KV head), EB of the state's columns (all
// 128 at D = 128, 64 of 256 at D = 256: what S's two terms leave room for in
// shared memory beside Q, two chunks of K and V, and W) and a segment of the
// stream's chunks. Streams are cut into segments where there are few of them:
// a first pass sums each segment's own contribution to the state, a scan
// carries the states across segments, and the main pass starts each segment
// from its state.
//
// Roles: 8 compute warps (W, P, the epilogue, the state), one warp that copies
// (TMA, 128-byte swizzle) and one that issues the MMAs.
#include "linear.cuh"
#include "mma.cuh"
#include "tc.cuh"

namespace dattn {

namespace {

constexpr int C = kLinearChunk;
constexpr int kComputeWarps = 8;
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 320;

enum : int {
  B_KVFULL = 0,   // [2] K and V of a chunk have landed
  B_KVFREE = 2,   // [2] every MMA that reads them has completed
  B_QFULL = 4,    // [2]
  B_QFREE = 6,    // [2]
  B_WREADY = 8,   // W (and the zeroed rows of a short chunk) written
  B_SREADY = 9,   // the state's two terms written
  B_ADONE = 10,   // Q K^T complete
  B_AFREE = 11,   // ... and read
  B_PREADY = 12,  // P written
  B_ODONE = 13,   // Q S and P V complete
  B_OFREE = 14,   // ... and read
  B_DSDONE = 15,  // K^T W complete
  B_FINAL = 16,
  B_COUNT = 17
};

template <int D>
struct Geo {
  static constexpr int EB = D == 128 ? 128 : 64;   // state columns of a CTA
  static constexpr int SLICES = D / EB;
  static constexpr int QS = D == 128 ? 2 : 1;      // Q tiles in shared memory
  static constexpr int ER = EB / 64, DR = D / 64;  // 64-element regions
  static constexpr int Q_TILE = DR * 16384;        // [region][128 rows][128 bytes]
  static constexpr int K_TILE = DR * 8192;         // [region][64 rows][128 bytes]
  static constexpr int V_TILE = ER * 8192;
  static constexpr int S_PLANE = ER * D * 128;     // [region][D rows][128 bytes]
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + QS * Q_TILE;
  static constexpr int V_OFF = K_OFF + 2 * K_TILE;
  static constexpr int W_OFF = V_OFF + 2 * V_TILE;  // hi, lo
  static constexpr int S_OFF = W_OFF + 2 * V_TILE;  // hi, lo
  static constexpr int BAR_OFF = S_OFF + 2 * S_PLANE;
  static constexpr int MISC_OFF = BAR_OFF + 8 * B_COUNT;
  static constexpr int PW_OFF = (MISC_OFF + 16 + 15) / 16 * 16;
  static constexpr int SMEM = PW_OFF + (C + 3) * 4 + 1024;  // (1024: alignment)
  // tensor memory columns
  static constexpr int T_A = 0, T_P = 64, T_O1 = 128, T_O2 = T_O1 + EB, T_DS = T_O2 + EB;
  static constexpr int T_COLS = 512;
};

struct Waiter {
  uint32_t bars;
  volatile int* abort;
  int* err;
  // Bounded wait by a whole warp or one thread; after a timeout (or when
  // another role gave up) every role leaves its loop.
  __device__ __forceinline__ bool wait(int b, uint32_t parity) const {
    const uint32_t bar = bars + 8 * b;
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
      for (int i = 0; i < 32; ++i)
        if (mbar_try_wait(bar, parity)) return true;
      if (*abort) return false;
      if (global_timer_ns() - t0 > kDefaultWaitNs) {
        *abort = 1;
        raise_error(err, ERR_TIMEOUT);
        return false;
      }
    }
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

// Two floats as packed bf16 hi terms and what is left as lo terms.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  lo = pack_bf16x2(x - bf16_lo(hi), y - bf16_hi(hi));
}

// One pass over a segment. SUMS: the segment's own contribution to the state
// (from zero), nothing else.
template <int D, bool SUMS>
__global__ void __launch_bounds__(kThreads, 1) linear_prompt_kernel(const __grid_constant__ LinearArgs a) {
  using Gm = Geo<D>;
  constexpr int EB = Gm::EB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bars = sbase + Gm::BAR_OFF;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Gm::MISC_OFF + 8);
  float* pw = reinterpret_cast<float*>(smem + Gm::PW_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- the CTA's work: (unit, slice, segment)
  int x = blockIdx.x;
  const int slice = x % Gm::SLICES;
  x /= Gm::SLICES;
  const int seg = x % a.segments, u = x / a.segments;
  const int b = u / a.Hkv, h = u - b * a.Hkv;
  const int G = a.G, hpt = G > 1 ? 2 : 1;  // query heads of an M tile
  const int tiles = SUMS ? 0 : (G + hpt - 1) / hpt;

  pdl_wait();
  pdl_trigger();
  const bool report = !SUMS && h == 0 && slice == 0 && seg == 0 && threadIdx.x == 0;
  const int row = state_row(a, b, report);
  int count = a.count[b];
  if (count < 0 || count > a.T) {
    if (report) raise_error(a.err, ERR_INDEX);
    count = 0;
  }
  const int chunks_all = (count + C - 1) / C;
  const int c0 = seg * a.seg_chunks, c1 = min(chunks_all, c0 + a.seg_chunks);
  const bool last_seg = c1 == chunks_all;
  const int nc = row < 0 ? 0 : c1 - c0;
  if (nc <= 0 || (SUMS && last_seg)) return;  // (the whole CTA)

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + 8 * (B_KVFULL + i), 1);
      mbar_init(bars + 8 * (B_KVFREE + i), 1);
      mbar_init(bars + 8 * (B_QFULL + i), 1);
      mbar_init(bars + 8 * (B_QFREE + i), 1);
    }
    mbar_init(bars + 8 * B_WREADY, kComputeWarps);
    mbar_init(bars + 8 * B_SREADY, kComputeWarps);
    mbar_init(bars + 8 * B_ADONE, 1);
    mbar_init(bars + 8 * B_AFREE, kComputeWarps);
    mbar_init(bars + 8 * B_PREADY, kComputeWarps);
    mbar_init(bars + 8 * B_ODONE, 1);
    mbar_init(bars + 8 * B_OFREE, kComputeWarps);
    mbar_init(bars + 8 * B_DSDONE, 1);
    mbar_init(bars + 8 * B_FINAL, 1);
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < C + 3; i += kThreads) pw[i] = a.decay[h * kDecayStride + i];
  if (warp == kMmaWarp) tc::alloc(sbase + Gm::MISC_OFF, Gm::T_COLS);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Gm::MISC_OFF);
  const Waiter W{bars, abort_flag, a.err};

  if (warp == kTmaWarp) {
    // ================= copies =================
    if (lane == 0) {
      const uint64_t policy = l2_evict_first_policy();
      bool ok = true;
      int kv = 0, qt = 0;  // copies issued
      for (int c = 0; c < nc && ok; ++c) {
        const int st = c & 1;
        const int tok = b * a.T + (c0 + c) * C;
        if (c >= 2) ok = W.wait(B_KVFREE + st, ((c >> 1) - 1) & 1);
        if (!ok) break;
        {
          const uint32_t bar = bars + 8 * (B_KVFULL + st);
          mbar_arrive_expect_tx(bar, Gm::K_TILE + Gm::V_TILE);
          for (int r = 0; r < Gm::DR; ++r)
            tma_load_3d(sbase + Gm::K_OFF + st * Gm::K_TILE + r * 8192, &a.tmap_k, 64 * r, h, tok, bar, policy);
          for (int r = 0; r < Gm::ER; ++r)
            tma_load_3d(sbase + Gm::V_OFF + st * Gm::V_TILE + r * 8192, &a.tmap_v, slice * EB + 64 * r, h, tok, bar,
                        policy);
          ++kv;
        }
        for (int mt = 0; mt < tiles && ok; ++mt, ++qt) {
          const int qs = qt % Gm::QS;
          if (qt >= Gm::QS) ok = W.wait(B_QFREE + qs, (qt / Gm::QS - 1) & 1);
          if (!ok) break;
          const uint32_t bar = bars + 8 * (B_QFULL + qs);
          mbar_arrive_expect_tx(bar, Gm::DR * static_cast<uint32_t>(hpt) * 8192u);
          for (int r = 0; r < Gm::DR; ++r)
            tma_load_3d(sbase + Gm::Q_OFF + qs * Gm::Q_TILE + r * 16384, &a.tmap_q, 64 * r, h * G + mt * hpt, tok, bar,
                        policy);
        }
      }
      // Copies still in flight exist only when a role gave up: they land
      // before the CTA exits.
      if (*abort_flag) {
        for (int i = max(0, kv - 2); i < kv; ++i) mbar_wait_bounded(bars + 8 * (B_KVFULL + (i & 1)), (i >> 1) & 1);
        for (int i = max(0, qt - Gm::QS); i < qt; ++i)
          mbar_wait_bounded(bars + 8 * (B_QFULL + i % Gm::QS), (i / Gm::QS) & 1);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ================= MMA issue =================
    if (lane == 0) {
      constexpr uint32_t id_a = tc::f16_idesc_ab(128, C, 1, false, false);
      constexpr uint32_t id_o = tc::f16_idesc_ab(128, EB, 1, false, true);
      constexpr uint32_t id_s = tc::f16_idesc_ab(128, EB, 1, true, true);
      auto issue_ds = [&](int c) -> bool {
        const int st = c & 1;
        if (!W.wait(B_WREADY, c & 1)) return false;
        tc::fence_after();
        const uint32_t kt = sbase + Gm::K_OFF + st * Gm::K_TILE, wt = sbase + Gm::W_OFF;
#pragma unroll
        for (int m = 0; m < D / 128; ++m)
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk) {
            const uint64_t kd = tc::sw128_desc(kt + m * 16384 + kk * 2048, 8192, 1024);
#pragma unroll
            for (int p = 0; p < 2; ++p)
              tc::mma(tmem + Gm::T_DS + m * EB, kd, tc::sw128_desc(wt + p * Gm::V_TILE + kk * 2048, 8192, 1024), id_s,
                      kk > 0 || p > 0);
          }
        tc::commit(bars + 8 * B_DSDONE);
        return true;
      };
      bool ok = true;
      int t = 0;  // tiles so far
      for (int c = 0; c < nc && ok; ++c) {
        const int st = c & 1;
        ok = W.wait(B_KVFULL + st, (c >> 1) & 1);
        if (!ok) break;
        if constexpr (SUMS) {
          ok = issue_ds(c);
          if (ok) tc::commit(bars + 8 * (B_KVFREE + st));
        }
        const uint32_t kt = sbase + Gm::K_OFF + st * Gm::K_TILE, vt = sbase + Gm::V_OFF + st * Gm::V_TILE;
        for (int mt = 0; mt < tiles && ok; ++mt, ++t) {
          const int qs = t % Gm::QS;
          const uint32_t qt = sbase + Gm::Q_OFF + qs * Gm::Q_TILE;
          // A = Q K^T
          ok = W.wait(B_QFULL + qs, (t / Gm::QS) & 1) && (t == 0 || W.wait(B_AFREE, (t - 1) & 1));
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma(tmem + Gm::T_A, tc::sw128_desc(qt + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024),
                    tc::sw128_desc(kt + (kk >> 2) * 8192 + (kk & 3) * 32, 16, 1024), id_a, kk > 0);
          tc::commit(bars + 8 * B_ADONE);
          // O1 = Q S
          ok = (mt > 0 || W.wait(B_SREADY, c & 1)) && (t == 0 || W.wait(B_OFREE, (t - 1) & 1));
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t qd = tc::sw128_desc(qt + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024);
#pragma unroll
            for (int p = 0; p < 2; ++p)
              tc::mma(tmem + Gm::T_O1, qd,
                      tc::sw128_desc(sbase + Gm::S_OFF + p * Gm::S_PLANE + kk * 2048, D * 128, 1024), id_o,
                      kk > 0 || p > 0);
          }
          tc::commit(bars + 8 * (B_QFREE + qs));
          if (mt == 0) {
            ok = issue_ds(c);
            if (!ok) break;
          }
          // O2 = P V
          ok = W.wait(B_PREADY, t & 1);
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk) {
            const uint64_t vd = tc::sw128_desc(vt + kk * 2048, 8192, 1024);
#pragma unroll
            for (int p = 0; p < 2; ++p)
              tc::mma_ts(tmem + Gm::T_O2, tmem + Gm::T_P + p * 32 + kk * 8, vd, id_o, kk > 0 || p > 0);
          }
          tc::commit(bars + 8 * B_ODONE);
          if (mt == tiles - 1) tc::commit(bars + 8 * (B_KVFREE + st));
        }
      }
      // every MMA issued has completed before the tensor memory is freed
      tc::commit(bars + 8 * B_FINAL);
      if (!mbar_wait_bounded(bars + 8 * B_FINAL, 0)) raise_error(a.err, ERR_TIMEOUT);
    }
    __syncwarp();
  } else {
    // ================= compute warps =================
    const int q4 = warp & 3, w2 = warp >> 2;  // lane quarter of tensor memory, column half
    const int r = 32 * q4 + lane;             // tensor memory lane
    const uint32_t lane_off = static_cast<uint32_t>(32 * q4) << 16;
    // the state: this thread's key dim (row) and 64 value dims
    const int sd = D == 128 ? r : 128 * w2 + r;
    const int se = D == 128 ? 64 * w2 : 0;
    const uint32_t t_ds = tmem + lane_off + Gm::T_DS + 64 * w2;
    float* state = a.state + (static_cast<int64_t>(row) * a.Hkv + h) * D * D + static_cast<int64_t>(sd) * D + slice * EB + se;
    float* seg_state = a.sums + ((static_cast<int64_t>(u) * a.segments + seg) * D + sd) * D + slice * EB + se;
    float S[64];
    if constexpr (SUMS) {
#pragma unroll
      for (int e = 0; e < 64; ++e) S[e] = 0.f;
    } else {
      const float* src = a.segments > 1 ? seg_state : state;
#pragma unroll
      for (int e = 0; e < 64; e += 4) {
        const float4 y = *reinterpret_cast<const float4*>(src + e);
        S[e] = y.x;
        S[e + 1] = y.y;
        S[e + 2] = y.z;
        S[e + 3] = y.w;
      }
    }
    auto arrive = [&](int bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * bar);
    };
    // the state's two terms as the B operand of Q S (value dims contiguous)
    auto store_s = [&]() {
      uint8_t* dst = smem + Gm::S_OFF + (D == 128 ? w2 : 0) * (D * 128) + sd * 128;
#pragma unroll
      for (int ch = 0; ch < 8; ++ch) {
        uint4 hi, lo;
        split2(S[8 * ch], S[8 * ch + 1], hi.x, lo.x);
        split2(S[8 * ch + 2], S[8 * ch + 3], hi.y, lo.y);
        split2(S[8 * ch + 4], S[8 * ch + 5], hi.z, lo.z);
        split2(S[8 * ch + 6], S[8 * ch + 7], hi.w, lo.w);
        const int off = (ch ^ (sd & 7)) << 4;
        *reinterpret_cast<uint4*>(dst + off) = hi;
        *reinterpret_cast<uint4*>(dst + Gm::S_PLANE + off) = lo;
      }
      fence_proxy_async_smem();
      arrive(B_SREADY);
    };
    if constexpr (!SUMS) store_s();
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    bool ok = true;
    int t = 0;
    for (int c = 0; c < nc && ok; ++c) {
      const int st = c & 1;
      const int tok0 = (c0 + c) * C;
      const int n = min(C, count - tok0);  // valid tokens
      ok = __all_sync(0xffffffffu, W.wait(B_KVFULL + st, (c >> 1) & 1));
      if (!ok) break;
      // ---- W = lam^(n-1-j) v_j as two terms; the rows past n become zeros in
      // V, W and K (a zero weight would not stop a NaN there)
      {
        uint8_t* vt = smem + Gm::V_OFF + st * Gm::V_TILE;
        uint8_t* wt = smem + Gm::W_OFF;
#pragma unroll
        for (int i = 0; i < Gm::V_TILE / 16 / 256; ++i) {
          const int off = (threadIdx.x + i * 256) * 16;
          const int j = (off >> 7) & (C - 1);
          uint4 y = *reinterpret_cast<const uint4*>(vt + off);
          if (j >= n) {
            y = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(vt + off) = y;
          }
          const float w = j < n ? pw[n - 1 - j] : 0.f;
          uint4 hi, lo;
          split2(bf16_lo(y.x) * w, bf16_hi(y.x) * w, hi.x, lo.x);
          split2(bf16_lo(y.y) * w, bf16_hi(y.y) * w, hi.y, lo.y);
          split2(bf16_lo(y.z) * w, bf16_hi(y.z) * w, hi.z, lo.z);
          split2(bf16_lo(y.w) * w, bf16_hi(y.w) * w, hi.w, lo.w);
          *reinterpret_cast<uint4*>(wt + off) = hi;
          *reinterpret_cast<uint4*>(wt + Gm::V_TILE + off) = lo;
        }
        if (n < C) {
          uint8_t* kt = smem + Gm::K_OFF + st * Gm::K_TILE;
          for (int off = threadIdx.x * 16; off < Gm::K_TILE; off += 256 * 16)
            if (((off >> 7) & (C - 1)) >= n) *reinterpret_cast<uint4*>(kt + off) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        arrive(B_WREADY);
      }
      if constexpr (!SUMS) {
        const int i = hpt == 2 ? r >> 1 : r;      // the row's token and head
        const int hd = hpt == 2 ? r & 1 : 0;
        for (int mt = 0; mt < tiles && ok; ++mt, ++t) {
          // ---- P: columns 32 w2 .. of A, masked and decayed
          ok = __all_sync(0xffffffffu, W.wait(B_ADONE, t & 1));
          if (!ok) break;
          tc::fence_after();
          uint32_t y[32];
          tc::ld32(tmem + lane_off + Gm::T_A + 32 * w2, y);
          tc::wait_ld();
          tc::fence_before();
          arrive(B_AFREE);
          uint32_t hi[16], lo[16];
          const int lim = min(i, C - 1) - 32 * w2;  // columns up to this one count
          const float* pi = pw + (i & (C - 1)) - 32 * w2;
#pragma unroll
          for (int jj = 0; jj < 32; jj += 2) {
            const float p0 = jj <= lim ? __uint_as_float(y[jj]) * pi[-jj] : 0.f;
            const float p1 = jj + 1 <= lim ? __uint_as_float(y[jj + 1]) * pi[-jj - 1] : 0.f;
            split2(p0, p1, hi[jj >> 1], lo[jj >> 1]);
          }
          tc::st16(tmem + lane_off + Gm::T_P + 16 * w2, hi);
          tc::st16(tmem + lane_off + Gm::T_P + 32 + 16 * w2, lo);
          tc::wait_st();
          fence_proxy_async_smem();  // (a short chunk's zeroed V rows)
          tc::fence_before();
          arrive(B_PREADY);
          // ---- epilogue: this thread's row, half of the columns
          const int g = mt * hpt + hd, tok = tok0 + i;
          const bool store = i < n && g < G;
          const int64_t head = (static_cast<int64_t>(b) * a.T + tok) * a.Hkv * G + static_cast<int64_t>(h) * G + g;
          float f = a.scale;
          if (store && a.gate) f /= 1.f + expf(-bf16_to_f32(a.gate[head]));
          const float f1 = f * pw[min(i, C - 1) + 1];
          ok = __all_sync(0xffffffffu, W.wait(B_ODONE, t & 1));
          if (!ok) break;
          tc::fence_after();
          float* dst = a.out + head * D + slice * EB + (EB / 2) * w2;
#pragma unroll
          for (int e0 = 0; e0 < EB / 2; e0 += 32) {
            uint32_t o1[32], o2[32];
            tc::ld32(tmem + lane_off + Gm::T_O1 + (EB / 2) * w2 + e0, o1);
            tc::ld32(tmem + lane_off + Gm::T_O2 + (EB / 2) * w2 + e0, o2);
            tc::wait_ld();
            if (e0 + 32 == EB / 2) {
              tc::fence_before();
              arrive(B_OFREE);
            }
            if (store) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                float z[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  z[q] = fmaf(__uint_as_float(o1[e + q]), f1, __uint_as_float(o2[e + q]) * f);
                st_8(dst + e0 + e, z, wide);
              }
            }
          }
        }
        if (!ok) break;
      }
      // ---- the state: S = lam^n S + dS (lam^C with what fp32 drops of it)
      ok = __all_sync(0xffffffffu, W.wait(B_DSDONE, c & 1));
      if (!ok) break;
      tc::fence_after();
      const float ln = pw[n], ln_lo = n == C ? pw[C + 2] : 0.f;
#pragma unroll
      for (int e0 = 0; e0 < 64; e0 += 32) {
        uint32_t y[32];
        tc::ld32(t_ds + e0, y);
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e)
          S[e0 + e] = fmaf(S[e0 + e], ln, fmaf(S[e0 + e], ln_lo, __uint_as_float(y[e])));
      }
      tc::fence_before();
      if constexpr (!SUMS) {
        if (c + 1 < nc) store_s();
      }
    }
    if (ok && (SUMS || last_seg)) {
      float* dst = SUMS ? seg_state : state;
#pragma unroll
      for (int e = 0; e < 64; e += 8) {
        float z[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) z[q] = S[e + q];
        st_8(dst + e, z, (reinterpret_cast<uintptr_t>(dst) & 31u) == 0);
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

// The states at the segments' starts from the segments' own sums: start 0 is
// the cache's state, start s + 1 = lam^(tokens of a segment) start s + sum s.
// One thread per 4 elements of a unit's state; every segment but a stream's
// last is full.
__global__ void __launch_bounds__(256) linear_scan_kernel(const LinearArgs a, int DD) {
  pdl_wait();
  pdl_trigger();
  const int64_t e = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  const int u = static_cast<int>(e / DD), at = static_cast<int>(e - static_cast<int64_t>(u) * DD);
  const int b = u / a.Hkv, h = u - b * a.Hkv;
  if (b >= a.B) return;
  const int row = state_row(a, b, false);
  const int count = a.count[b];
  if (row < 0 || count <= 0 || count > a.T) return;
  const int segs = ((count + C - 1) / C + a.seg_chunks - 1) / a.seg_chunks;
  const double l = exp(static_cast<double>(a.log_decay[h]) * a.seg_chunks * C);
  const float lam = static_cast<float>(l), lam_lo = static_cast<float>(l - static_cast<double>(lam));
  float4 s = *reinterpret_cast<const float4*>(a.state + (static_cast<int64_t>(row) * a.Hkv + h) * DD + at);
  float* p = a.sums + static_cast<int64_t>(u) * a.segments * DD + at;
  float4 next = make_float4(0.f, 0.f, 0.f, 0.f);
  if (segs > 1) next = *reinterpret_cast<const float4*>(p);
  for (int i = 0; i < segs; ++i) {
    const float4 y = next;
    if (i + 2 < segs) next = *reinterpret_cast<const float4*>(p + static_cast<int64_t>(i + 1) * DD);
    *reinterpret_cast<float4*>(p + static_cast<int64_t>(i) * DD) = s;
    s.x = fmaf(s.x, lam, fmaf(s.x, lam_lo, y.x));
    s.y = fmaf(s.y, lam, fmaf(s.y, lam_lo, y.y));
    s.z = fmaf(s.z, lam, fmaf(s.z, lam_lo, y.z));
    s.w = fmaf(s.w, lam, fmaf(s.w, lam_lo, y.w));
  }
}

template <int D, bool SUMS>
cudaError_t prompt_launch(const LinearArgs& a, cudaStream_t s) {
  using Gm = Geo<D>;
  auto k = linear_prompt_kernel<D, SUMS>;
  static std::atomic<uint64_t> opted{0};
  const cudaError_t e = opt_in_smem(k, Gm::SMEM, opted);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.B) * a.Hkv * a.segments * Gm::SLICES);
  return launch_pdl(k, grid, dim3(kThreads), Gm::SMEM, s, a);
}

}  // namespace

int linear_prompt_segments(int units, int T, int D, int num_sms, int* seg_chunks) {
  const int chunks = (T + C - 1) / C;
  const int ctas = units * (D == 128 ? Geo<128>::SLICES : Geo<256>::SLICES);
  int segs = num_sms / ctas;
  if (segs > chunks / 4) segs = chunks / 4;
  if (segs < 1) segs = 1;
  *seg_chunks = (chunks + segs - 1) / segs;
  return (chunks + *seg_chunks - 1) / *seg_chunks;
}

cudaError_t launch_linear_prompt(const LinearArgs& a, int D, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.segments > 1) {
    e = D == 128 ? prompt_launch<128, true>(a, s) : prompt_launch<256, true>(a, s);
    if (e != cudaSuccess) return e;
    const int64_t elems = static_cast<int64_t>(a.B) * a.Hkv * D * D / 4;
    e = launch_pdl(linear_scan_kernel, dim3(static_cast<unsigned>((elems + 255) / 256)), dim3(256), 0, s, a, D * D);
    if (e != cudaSuccess) return e;
  }
  return D == 128 ? prompt_launch<128, false>(a, s) : prompt_launch<256, false>(a, s);
}

}  // namespace dattn
