// Decode attention over 4-bit caches (int4_format.h) in one launch per call: RoPE of the
// new token, the pass over the cached blocks, the join of the new token in score space,
// the gate, the fp32 store and the write-back of the new entry.
//
// A unit is one (stream, KV head); its cache is a row of blocks of 16 tokens. What
// bounds the pass is its arithmetic, more than its memory traffic (4.5 bits a value): with
// operands as they come out of the codes it took 0.93 of the copies' time on 256-wide heads
// of 4 queries and 1.5 times that time on groups of 5 to 8, whose scores and outputs are two
// column tiles of the MMAs, and precision (decode_int4.cuh) cost a quarter more. So every
// sub-partition of every SM has to work all the time:
//  * The split is made for warps, not CTAs. All units' blocks are laid end to end, each
//    unit charged a fixed cost in blocks before them (Split), and every warp of the grid
//    takes an equal contiguous range: it turns its own query, streams its own blocks
//    through its own ring of stage buffers and meets no other warp until its CTA is done.
//    A unit that lies within one warp's range is finished by that warp on the way. The
//    warps are a multiple of 4, as the sub-partition with the most sets the pace. (The
//    other formats' layout, 10 or 11 streaming warps that share a CTA's units beside a
//    helper warp, took 244 us for 8 x 262,144 tokens, where this one took 193 with the
//    same operands, 53 for 64 ragged streams, 42 here, and 193 for 32 x 16,384 tokens of
//    24 / 4 heads, 144 here; one stream of 5,003 tokens 19.3, and 20 here.)
//  * At the end of a CTA the warps' states of each unit are merged by a team of its warps,
//    the teams of several units side by side; states of units that cross CTAs go to global
//    memory and the team that counts last for a unit joins them, in two levels where they
//    are many.
//  * The new token of a unit is quantised, scored and gated by the warp that starts the
//    unit, and lies ready in global memory when the unit is finished.
// Copies are whole blocks (9 D bytes of K and of V, one bulk copy each; neighbouring
// blocks of a page go as one), issued by one lane NS stages ahead; the page table is
// read 32 blocks ahead, a block a lane, and handed on by shuffles.
//
// Measured (GB300, a call among others): 8 x 262,144 tokens of 8 / 2 heads of 256 248 us,
// 4.9 TB/s; 1 x 1,048,576 134 us; 64 ragged streams 48 us; 32 x 16,384 of 24 / 4 heads 176.
// Of the first ~8 us pass before the first copies land and ~10 between the last block and
// the last output.
#include "decode_int4.cuh"
#include "int4.cuh"
#include "bf16_exact.h"
#include "qk_norm.cuh"
#include "round_f64.h"

namespace dattn {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxUnits = 512;
constexpr int kMergeBatch = 8;  // CTAs of a group of the two-level merge
constexpr int kFoldBatch = 12;  // states read per round trip
constexpr int64_t kPrefetchLines = 1 << 15;  // largest page table (128-byte lines) put in L2 at start
// Cost of a unit's start (its query and new token) in blocks of a warp: 2 / 4 / 6 / 9
// blocks, 64 ragged streams of 8 heads of 128 52.1 / 48.1 / 49.5 / 48.5 us, 32 x 16,384 tokens of
// 24 / 4 heads of 256 176.3 / 173.8 / 173.9 / 173.9.
constexpr int kUnitCost = 4;
// Blocks that are worth another warp where a call has few: 2 / 3 / 4 / 5, in a graph of such
// calls, one stream of 5,003 tokens of 8 / 2 heads of 256 9.9 / 11.2 / 11.4 / 13.1 us, 20,000
// tokens 18.2 / 12.6 / 12.3 / 13.2 us, 4 streams of 2,000 - 4,000 tokens of 24 / 4 heads 26.1 /
// 26.4 / 18.5 / 18.0 us (more CTAs are more partial states to join; with the operands as
// they are now, 5,003 tokens with write-back and read back, 2 / 4 / 6 blocks, 23.5 / 23.4 / 25.6).
constexpr int kMinBlocks = 4;

template <int HEAD_DIM, int NT>
struct Geo4 {
  static constexpr int D = HEAD_DIM, GP = 4 * NT;
  // Warps, blocks of a stage, stages of a warp's ring. Two blocks are taken at once: their
  // chains of dependent steps overlap (one at a time, 8 x 262,144 tokens 193 -> 208 us
  // before the operands were made precise). 256-wide heads then need up to 255 registers,
  // which leaves 8 warps (12 with one block a stage: 220 us then). 128-wide ones of up to 4
  // queries fit 168 and 12 warps (8: 48.1 -> 51.8 us on 64 ragged); with a second column tile
  // 168 spill, and 8 warps are faster (12 -> 8: 64 / 8 heads, 64 ragged streams 91 -> 86 us and
  // 16 x 16,384 tokens 109.7 -> 107.8; 8 / 1, 8 x 262,144 109.6 -> 107.3, 64 ragged 23.0 -> 21.4;
  // 6 / 1, 32 x 16,384 39.6 -> 36.3; one stream of 5,003 13.9 -> 12.9).
  static constexpr int W = D == 256 || NT == 2 ? 8 : 12;
  static constexpr int KG = 2;
  static constexpr int NS = D == 256 ? 2 : 3;
  static constexpr int THREADS = W * 32;
  static constexpr int BLK = int4_block_bytes(D);
  static constexpr int HALF = KG * BLK;                   // K part of a stage; V follows
  static constexpr int RING = NS * 2 * HALF;
  using Warp = Int4Warp<D, NT>;
  // a warp's inputs as they come, then its query in fp32, then the fragments where they
  // stay in shared memory; at a unit's end within the warp's range, its state
  static constexpr int STATE = GP * (D + 2);  // floats of a state: o [GP][D], m [GP], l [GP]
  static constexpr int SCRATCH = Warp::kSharedQ && Warp::kQBytes > STATE * 4 ? Warp::kQBytes : STATE * 4;
  static constexpr int SCRATCH_OFF = W * RING;
  static constexpr int BAR_OFF = SCRATCH_OFF + W * SCRATCH;   // [W][NS] stages, [W] inputs
  static constexpr int LIST_OFF = BAR_OFF + W * (NS + 1) * 8; // pointer [W][32]: a team's states
  static constexpr int SEG_OFF = LIST_OFF + W * 32 * 8;       // int [2 W]: units of the CTA's states
  static constexpr int SPAN_OFF = SEG_OFF + 2 * W * 4;        // Span [2 W]: where those units' other states are
  // the call's arguments and the CTAs' split, where functions that are not inlined read
  // them (through a pointer to the parameters every field would be a trip to global memory)
  static constexpr int ARG_OFF = SPAN_OFF + 2 * W * 16;
  static constexpr int SPLIT_OFF = ARG_OFF + (sizeof(Int4DecodeArgs) + 15) / 16 * 16;
  static constexpr int FLAG_OFF = SPLIT_OFF + (sizeof(Split) + 15) / 16 * 16;
  static constexpr int TAB_OFF = FLAG_OFF + W * 4;             // int [U + 1], [U]
  static constexpr int SMEM_MAX = 128 + TAB_OFF + (2 * kMaxUnits + 1) * 4;
  static_assert(STATE * 4 <= RING && SCRATCH % 16 == 0, "a state fits where a warp leaves it");
  static_assert(SMEM_MAX <= 232448 - 256, "shared memory per CTA");
  static_assert(2 * W <= 32, "the states of a CTA, a lane each");
  static_assert(KG == 2, "issue() and the tail of a unit know two blocks a stage");
};

// Some warps of a CTA, one beside the other, that work on a unit's states together.
struct Team {
  int t, nth;  // the thread's index in it, its threads
  int bar;     // its barrier (1 .. 15)
  __device__ __forceinline__ void sync() const {
    if (nth == 32) __syncwarp(); else asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(nth) : "memory");
  }
};

// Running merge of softmax states over 4 dims of a head.
struct Merge4 {
  float M, L;
  float4 o;
  __device__ __forceinline__ void add(float m, float l, const float4& x) {
    const float Mn = fmaxf(M, m);
    const float base = Mn == -INFINITY ? 0.f : Mn;
    const float al = exp2_fast(M - base), be = exp2_fast(m - base);
    L = fmaf(L, al, l * be);
    o = make_float4(fmaf(o.x, al, x.x * be), fmaf(o.y, al, x.y * be), fmaf(o.z, al, x.z * be), fmaf(o.w, al, x.w * be));
    M = Mn;
  }
};

// A state's floats, in shared memory or written by another CTA before it counted.
__device__ __forceinline__ float4 ld_state4(const float* p) {
  float4 x;
  asm volatile("ld.relaxed.gpu.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(p) : "memory");
  return x;
}
__device__ __forceinline__ float ld_state(const float* p) {
  float x;
  asm volatile("ld.relaxed.gpu.f32 %0, [%1];" : "=f"(x) : "l"(p) : "memory");
  return x;
}

// Dims d .. d + 3 of head g of the n listed states (null: none), merged; the loads of
// kFoldBatch states at once.
template <int D, int GP>
__device__ __forceinline__ Merge4 fold(const float* const* list, int n, int g, int d) {
  Merge4 mg{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 1
  for (int k = 0; k < n; k += kFoldBatch) {
    float4 x[kFoldBatch];
    float m[kFoldBatch], l[kFoldBatch];
#pragma unroll
    for (int i = 0; i < kFoldBatch; ++i) {
      const float* p = k + i < n ? list[k + i] : nullptr;
      m[i] = -INFINITY;
      l[i] = 0.f;
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p) {
        x[i] = ld_state4(p + g * D + d);
        m[i] = ld_state(p + GP * D + g);
        l[i] = ld_state(p + GP * D + GP + g);
      }
    }
#pragma unroll
    for (int i = 0; i < kFoldBatch; ++i)
      if (k + i < n) mg.add(m[i], l[i], x[i]);
  }
  return mg;
}

// The listed states merged into the state dst (none of them), by a team.
template <int D, int GP>
__device__ __forceinline__ void store_state(float* dst, const float* const* list, int n, const Team& tm) {
#pragma unroll 1
  for (int e = tm.t * 4; e < GP * D; e += tm.nth * 4) {
    const int g = e / D, d = e - g * D;
    const Merge4 mg = fold<D, GP>(list, n, g, d);
    *reinterpret_cast<float4*>(dst + e) = mg.o;
    if (d == 0) {
      dst[GP * D + g] = mg.M;
      dst[GP * D + GP + g] = mg.L;
    }
  }
}

// Cached tokens of call row b; bad metadata is reported and clamped.
__device__ __forceinline__ int stream_length(const Int4DecodeArgs& a, int b, bool report) {
  const int cap = min(a.max_len, a.c.bt_stride * a.c.P);
  const int n = a.c.seq_len[b];
  if (n >= 0 && n <= cap) return n;
  if (report) raise_error(a.err, ERR_LENGTH);
  return n < 0 ? 0 : cap;
}

// Dim d of a new key row (global): the entry, normalised and turned (as key_exact says).
__device__ __forceinline__ uint32_t key_entry(const Int4DecodeArgs& a, const uint16_t* row, double inv, int pos, int d) {
  const uint16_t* kn = a.k_norm;
  auto at = [&](int x) { return kn ? qk_norm_apply(row[x], kn[x], inv) : row[x]; };
  const uint16_t x = at(d);
  if (d >= a.r) return x;
  const int half = a.r / 2;
  const bool first = d < half;
  float c, s;
  rope_cos_sin_near(pos, a.rope_step[first ? d : d - half], c, s);
  const float xc = bf16_to_f32(x) * c, y = bf16_to_f32(at(first ? d + half : d - half));
  const float v = fmaf(y, first ? -s : s, xc), e = fmaf(fabsf(xc) + fabsf(v), kTurnError, 0x1p-110f);
  const uint32_t w = pack_bf16x2(v - e, v + e);
  if ((w >> 16) == (w & 0xffffu)) return w & 0xffffu;
  return key_exact(row, kn, inv, pos, a.rope_step, a.r, d);
}

// One lane: the inputs of unit u into a warp's scratch, counted on bar: its query rows in
// the upper half, and for the warp that starts the unit its new key and value in the lower.
template <int D, int GP>
__device__ __forceinline__ void stage_inputs(const Int4DecodeArgs& a, int u, bool token, uint32_t scratch, uint32_t bar) {
  const uint64_t policy = l2_evict_first_policy();
  const uint32_t qbytes = static_cast<uint32_t>(a.G) * D * 2;
  mbar_arrive_expect_tx(bar, qbytes + (token ? 4u * D : 0u));
  bulk_copy_g2s(scratch + GP * D * 2, a.q + static_cast<int64_t>(u) * a.G * D, qbytes, bar, policy);
  if (token) {
    bulk_copy_g2s(scratch, a.k_new + static_cast<int64_t>(u) * D, 2u * D, bar, policy);
    bulk_copy_g2s(scratch + 2 * D, a.v_new + static_cast<int64_t>(u) * D, 2u * D, bar, policy);
  }
}

// One warp, its inputs staged: the G query heads of unit u, normalised, turned and scaled,
// into qs [GP][D] fp32 (heads >= G are zero), over the inputs. For the warp that starts the
// unit: the new token as the cache will hold it, its scores against that query and the
// heads' gates, into the unit's record: float [GP] scores, float [GP] gates, codes of key and
// value in the dims' order, their pairs. Ends with a warp barrier.
template <int D, int GP>
__device__ __forceinline__ void prepare(const Int4DecodeArgs& a, int u, bool token, float* qs, int lane) {
  constexpr int CH = D / 32, LPG = kInt4Group / CH;  // dims of a lane, lanes of a group
  constexpr int STEPS = GP * D / 256;
  const int half = a.r / 2;
  const int pos = a.r > 0 ? a.pos[u / a.Hkv] : 0;
  const uint16_t gate = token && a.gate && lane < a.G ? a.gate[static_cast<int64_t>(u) * a.G + lane] : 0;
  uint32_t kv[2][CH / 2];
#pragma unroll
  for (int i = 0; i < CH / 2; ++i) {
    kv[0][i] = reinterpret_cast<const uint32_t*>(qs)[lane * (CH / 2) + i];
    kv[1][i] = reinterpret_cast<const uint32_t*>(qs)[D / 2 + lane * (CH / 2) + i];
  }
  {
    uint4 q[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int e = (i * 32 + lane) * 8;
      q[i] = e < a.G * D ? *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(qs) + GP * D + e) : make_uint4(0u, 0u, 0u, 0u);
    }
    __syncwarp();
    const float scale = a.r == 0 && !a.q_norm ? a.q_scale : 1.f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const uint4 x = q[i];
      float4* dst = reinterpret_cast<float4*>(qs + (i * 32 + lane) * 8);
      dst[0] = make_float4(bf16_lo(x.x) * scale, bf16_hi(x.x) * scale, bf16_lo(x.y) * scale, bf16_hi(x.y) * scale);
      dst[1] = make_float4(bf16_lo(x.z) * scale, bf16_hi(x.z) * scale, bf16_lo(x.w) * scale, bf16_hi(x.w) * scale);
    }
    __syncwarp();
  }
  if (a.q_norm) {
    const uint16_t* src = a.q + static_cast<int64_t>(u) * a.G * D;
    for (int g = 0; g < a.G; ++g) {
      const double inv = qk_norm_inv(src + g * D, D, a.norm_eps, lane);
      for (int d = lane; d < D; d += 32) qs[g * D + d] = bf16_to_f32(qk_norm_apply(src[g * D + d], a.q_norm[d], inv));
    }
    __syncwarp();
  }
  if (a.r > 0 || a.q_norm) {
#pragma unroll 1
    for (int p = lane; p < D / 2; p += 32) {
      const int d0 = p < half ? p : a.r + 2 * (p - half), d1 = p < half ? p + half : d0 + 1;
      float c = 1.f, s = 0.f;
      if (p < half) rope_cos_sin(pos, a.rope_step[p], c, s);
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        const float x = qs[g * D + d0], y = qs[g * D + d1];
        qs[g * D + d0] = (p < half ? fmaf(x, c, -y * s) : x) * a.q_scale;
        qs[g * D + d1] = (p < half ? fmaf(y, c, x * s) : y) * a.q_scale;
      }
    }
    __syncwarp();
  }
  if (!token) return;
  uint8_t* rec = a.token + u * int4_token_bytes(D, GP);
  if (a.r > 0 || a.k_norm) {
    const uint16_t* row = a.k_new + static_cast<int64_t>(u) * D;
    const double inv = a.k_norm ? qk_norm_inv(row, D, a.norm_eps, lane) : 0.0;
#pragma unroll 1
    for (int i = 0; i < CH; ++i) {
      const uint32_t v = key_entry(a, row, inv, pos, lane * CH + i);
#pragma unroll
      for (int j = 0; j < CH / 2; ++j)  // (no indexing of registers)
        if (i >> 1 == j) kv[0][j] = i & 1 ? (kv[0][j] & 0xffffu) | (v << 16) : (kv[0][j] & 0xffff0000u) | v;
    }
    __syncwarp();
  }
  float* sn = reinterpret_cast<float*>(rec);
  uint8_t* packed = rec + 8 * GP;
  float k[CH];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    uint32_t e = extent(kv[side]);
#pragma unroll
    for (int o = 1; o < LPG; o <<= 1) e = max2_nan(e, __shfl_xor_sync(kFull, e, o));
    const Int4Grid q = grid_of(e);
    const uint32_t c = codes<CH>(kv[side], q);
    if constexpr (CH == 8) reinterpret_cast<uint32_t*>(packed + side * (D / 2))[lane] = c;
    else reinterpret_cast<uint16_t*>(packed + side * (D / 2))[lane] = static_cast<uint16_t>(c);
    if (lane % LPG == 0) reinterpret_cast<uint32_t*>(packed + D)[side * (D / kInt4Group) + lane / LPG] = q.pair;
    if (side == 0)
#pragma unroll
      for (int i = 0; i < CH; ++i)
        k[i] = fmaf(static_cast<float>((c >> (4 * i)) & 15u), bf16_hi(q.pair), bf16_lo(q.pair));
  }
  float dot[GP];
#pragma unroll
  for (int g = 0; g < GP; ++g) {
    dot[g] = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) dot[g] = fmaf(qs[g * D + lane * CH + i], k[i], dot[g]);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
    for (int g = 0; g < GP; ++g) dot[g] += __shfl_xor_sync(kFull, dot[g], o);
#pragma unroll
  for (int g = 0; g < GP; ++g)
    if (lane == g) sn[g] = dot[g];
  if (lane < GP) sn[GP + lane] = a.gate ? 1.f / (1.f + expf(-bf16_to_f32(gate))) : 1.f;
  __syncwarp();
}

// Output and write-back of unit u by a team, once all of its blocks have been read: its
// n listed states joined with the new token.
template <int D, int GP>
__device__ __forceinline__ void finish_unit(const Int4DecodeArgs& a, int u, const float* const* list, int n_states, const Team& tm) {
  const uint8_t* rec = a.token + u * int4_token_bytes(D, GP);
  const float* sn = reinterpret_cast<const float*>(rec);
  const uint8_t* packed = rec + 8 * GP;
  // the slot of the new entry: its loads beside those of the states. (A length outside the
  // bound has none: the one after the bound holds a token of the longer stream.)
  const CacheView& c = a.c;
  const int b = u / a.Hkv;
  int n = -1, pi = 0, pg = -1;
  if (a.write_back) {
    n = c.seq_len[b];
    if (n > min(a.max_len, c.bt_stride * c.P)) n = -1;
    pi = max(n, 0) / c.P;
    if (n >= 0 && pi < c.bt_stride) pg = c.block_table[static_cast<int64_t>(b) * c.bt_stride + pi];
  }
#pragma unroll 1
  for (int e = tm.t * 4; e < a.G * D; e += tm.nth * 4) {
    const int g = e / D, d = e - g * D;
    const float score = ld_state(sn + g), sig = ld_state(sn + GP + g);
    const uint32_t code = __ldcg(reinterpret_cast<const uint16_t*>(packed + D / 2 + d / 2));
    const uint32_t pair = __ldcg(reinterpret_cast<const uint32_t*>(packed + D) + D / kInt4Group + d / kInt4Group);
    Merge4 mg = fold<D, GP>(list, n_states, g, d);
    const float step = bf16_hi(pair), least = bf16_lo(pair);
    mg.add(score, 1.f, make_float4(fmaf(static_cast<float>(code & 15u), step, least), fmaf(static_cast<float>((code >> 4) & 15u), step, least),
                                   fmaf(static_cast<float>((code >> 8) & 15u), step, least), fmaf(static_cast<float>(code >> 12), step, least)));
    const float scale = sig / mg.L;
    *reinterpret_cast<float4*>(a.out + (static_cast<int64_t>(u) * a.G + g) * D + d) =
        make_float4(mg.o.x * scale, mg.o.y * scale, mg.o.z * scale, mg.o.w * scale);
  }
  if (!a.write_back || n < 0) return;
  if (pg < 0 || pg >= c.n_rows) {
    if (tm.t == 0) raise_error(a.err, ERR_INDEX);
    return;
  }
  const int at = n - pi * c.P, r = at % kInt4Block;
  const int64_t base = ((static_cast<int64_t>(pg) * a.Hkv + (u - b * a.Hkv)) * (c.P / kInt4Block) + at / kInt4Block) * int4_block_bytes(D);
  uint8_t* kd = reinterpret_cast<uint8_t*>(c.k) + base;
  uint8_t* vd = reinterpret_cast<uint8_t*>(c.v) + base;
  for (int w = tm.t; w < D / 8; w += tm.nth)
    *reinterpret_cast<uint32_t*>(kd + int4_key_word(r, w)) = __ldcg(reinterpret_cast<const uint32_t*>(packed) + w);
  for (int w = tm.t; w < D / 4; w += tm.nth)
    *reinterpret_cast<uint16_t*>(vd + int4_value_half(r, w)) = __ldcg(reinterpret_cast<const uint16_t*>(packed + D / 2) + w);
  for (int x = tm.t; x < D / 32; x += tm.nth)
    *reinterpret_cast<uint32_t*>((x < D / 64 ? kd : vd) + int4_pair(D, r, x % (D / 64))) =
        __ldcg(reinterpret_cast<const uint32_t*>(packed + D) + x);
}

// The last unit u in [0, U) with P[u] + C u <= t (0 <= t), by a whole warp: 32 units a step.
__device__ __forceinline__ int unit_at(const int* P, int U, int C, int t, int lane) {
  const int step = (U + 31) / 32;  // (at most 16)
  int u = lane * step;
  const int at = (__popc(__ballot_sync(kFull, u < U && P[u] + C * u <= t)) - 1) * step;
  u = at + lane;
  return at + __popc(__ballot_sync(kFull, lane < step && u < U && P[u] + C * u <= t)) - 1;
}

// Split::tile_at(bound(w)) by a whole warp: the first block of worker w of n. In 32 bits
// (w W / n = w (W / n) + w (W mod n) / n; the weight of all blocks is below 2^31, n^2 as well).
__device__ __forceinline__ int first_block(const int* P, int U, int C, int weight, int w, int n, int lane) {
  const unsigned q = static_cast<unsigned>(weight) / n, r = static_cast<unsigned>(weight) - q * n;
  const int t = static_cast<int>(w * q + w * r / n);
  if (t >= weight) return P[U];
  const int u = unit_at(P, U, C, t, lane);
  const int off = t - (P[u] + C * u) - C;
  return P[u] + max(off, 0);
}

// The CTAs that hold blocks of a unit: the first and the last, and the partial slot of the
// first one (its own unless another unit ends there).
struct Span {
  int lo, hi, slot;
};
__device__ __forceinline__ Span span_of(const Split& cs, int u) {
  Span s;
  s.lo = cs.cta_of(cs.P[u], u);
  s.hi = cs.cta_of(cs.P[u + 1] - 1, u);
  s.slot = cs.tile_at(cs.bound(s.lo)) == cs.P[u] ? s.lo : cs.NC + u;
  return s;
}

// A unit's n listed states in this CTA, merged by a team: straight into the output when
// the unit lies wholly in the CTA, otherwise into the CTA's partial slot; the team of the CTA
// that counts last for the unit joins the partials. Where they are many it joins what the
// last to count of each group of kMergeBatch CTAs has merged.
template <int D, int GP>
__device__ __forceinline__ void merge_unit(const Int4DecodeArgs& a, const Split& cs, int u, const Span span, int cta,
                                           const float** list, int n, int* flag, const Team& tm) {
  constexpr int stride = GP * (D + 2);
  const int c_lo = span.lo, S = span.hi - c_lo + 1;
  // a CTA strictly inside the unit's span holds blocks of it unless it got none at all
  const bool full = cs.W >= cs.NC;
  auto holds = [&](int k) { return full || k == 0 || k == S - 1 || cs.has_tiles_inside(c_lo + k); };
  auto slot = [&](int k) { return a.part + static_cast<int64_t>(k == 0 ? span.slot : c_lo + k) * stride; };
  auto count = [&](int k0, int k1) {
    int m = k1 - k0;
    if (!full)
      for (int k = k0; k < k1; ++k) m -= !holds(k);
    return m;
  };
  const int groups = (S + kMergeBatch - 1) / kMergeBatch;
  const int k0 = (cta - c_lo) / kMergeBatch * kMergeBatch, k1 = min(S, k0 + kMergeBatch);
  // 0: the CTA's states, 1: a group's partials, 2: the unit's partials or groups
  int level = S == 1 ? 2 : 0;
#pragma unroll 1
  while (level < 2) {
    const bool grouped = S > 2 * kMergeBatch;
    // (a group's counter and its merged state are named by its last CTA: no other unit's group ends there)
    store_state<D, GP>(level == 0 ? slot(cta - c_lo) : a.gpart + static_cast<int64_t>(c_lo + k1 - 1) * stride, list, n, tm);
    const bool to_group = level == 0 && grouped;
    int m;
    if (to_group) {
      m = count(k0, k1);
    } else if (!grouped) {
      m = count(0, S);
    } else {
      m = groups;
      if (!full)
        for (int q = 0; q < groups; ++q) m -= count(q * kMergeBatch, min(S, (q + 1) * kMergeBatch)) == 0;
    }
    // count the team in, of m in all; the last sees what the others wrote
    tm.sync();
    if (tm.t == 0) {
      int* counter = to_group ? a.counters + cs.U + c_lo + k1 - 1 : a.counters + u;
      int before;
      asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
      *flag = before == m - 1;
      if (before == m - 1) *counter = 0;
    }
    tm.sync();
    if (*flag == 0) return;
    level = to_group ? 1 : 2;
    n = to_group ? k1 - k0 : grouped ? groups : S;
    for (int k = tm.t; k < n; k += tm.nth) {
      const float* p;
      if (to_group || !grouped) {
        const int x = to_group ? k0 + k : k;
        p = holds(x) ? slot(x) : nullptr;
      } else {
        const int e = min(S, (k + 1) * kMergeBatch);
        p = count(k * kMergeBatch, e) > 0 ? a.gpart + static_cast<int64_t>(c_lo + e - 1) * stride : nullptr;
      }
      list[k] = p;
    }
    tm.sync();
  }
  finish_unit<D, GP>(a, u, list, n, tm);
}

template <int D, int NT>
__global__ void __launch_bounds__(Geo4<D, NT>::THREADS, 1) int4_decode_kernel(const __grid_constant__ Int4DecodeArgs args) {
  using Gm = Geo4<D, NT>;
  using Warp = typename Gm::Warp;
  constexpr int GP = Gm::GP, W = Gm::W, KG = Gm::KG, NS = Gm::NS, BLK = Gm::BLK;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Int4DecodeArgs& a = *reinterpret_cast<Int4DecodeArgs*>(smem + Gm::ARG_OFF);
  Split& cs = *reinterpret_cast<Split*>(smem + Gm::SPLIT_OFF);
  const CacheView& c = args.c;
  const int Hkv = args.Hkv, U = args.B * Hkv, NC = gridDim.x, cta = blockIdx.x;
  const float** list = reinterpret_cast<const float**>(smem + Gm::LIST_OFF) + warp * 32;
  int* SEG = reinterpret_cast<int*>(smem + Gm::SEG_OFF);
  int* flag = reinterpret_cast<int*>(smem + Gm::FLAG_OFF);
  int* P = reinterpret_cast<int*>(smem + Gm::TAB_OFF);  // [U + 1] block prefix over units
  int* N = P + U + 1;                                    // [U] cached tokens
  float* scratch = reinterpret_cast<float*>(smem + Gm::SCRATCH_OFF + warp * Gm::SCRATCH);
  uint8_t* ring = smem + warp * Gm::RING;
  const uint32_t ring_a = smem_addr(ring), bar0 = smem_addr(smem + Gm::BAR_OFF) + warp * (NS + 1) * 8, inbar = bar0 + NS * 8;

  {
    // the page table into L2 (each CTA a share of its lines)
    const int64_t lines = (static_cast<int64_t>(args.B) * c.bt_stride + 31) / 32;
    if (lines <= kPrefetchLines)
      for (int64_t i = static_cast<int64_t>(cta) * Gm::THREADS + threadIdx.x; i < lines; i += static_cast<int64_t>(NC) * Gm::THREADS)
        prefetch_l2(c.block_table + i * 32);
  }
  if (lane == 0) {
    for (int i = 0; i <= NS; ++i) mbar_init(bar0 + 8 * i, 1);
    fence_mbar_init();
  }
  for (int u = threadIdx.x; u < U; u += Gm::THREADS) {
    const int b = u / Hkv;
    const int n = stream_length(args, b, cta == 0 && u == b * Hkv);
    N[u] = n;
    P[u + 1] = (n + kInt4Block - 1) / kInt4Block;
  }
  if (threadIdx.x == 0) {
    P[0] = 0;
    a = args;
  }
  if (lane < 2) SEG[2 * warp + lane] = -1;
  __syncthreads();
  block_scan_inclusive<Gm::THREADS>(P + 1, U);
  const int weight = P[U] + kUnitCost * U;
  if (threadIdx.x == 0) cs = Split{P, U, kUnitCost, NC, weight};  // (read after the next barrier)
  const int worker = cta * W + warp;
  const int b0 = first_block(P, U, kUnitCost, weight, worker, NC * W, lane);
  const int nb = first_block(P, U, kUnitCost, weight, worker + 1, NC * W, lane) - b0;
  const int u_first = nb > 0 ? unit_at(P, U, 0, b0, lane) : U;
  // Ordering with the preceding launch on the stream: as decode_kernel. Inputs, metadata
  // and this call's half of the workspace are not written by it (but for inputs that it
  // reads back: then they wait); the cache may be read early where it does not write that;
  // outputs and the write-back come after the wait.
  bool waited = false;
  auto wait_prev = [&]() {
    if (!waited) {
      pdl_wait();
      pdl_trigger();
      waited = true;
    }
  };
  if (args.late) wait_prev();
  // the inputs first: every warp's, ahead of any warp's blocks
  if (nb > 0 && lane == 0) stage_inputs<D, GP>(args, u_first, b0 == P[u_first], smem_addr(scratch), inbar);

  if (!args.early) wait_prev();

  // ---- copies: the pool blocks of the range 32 at a time, a block a lane (the current
  // window and the next); stage by stage, never across a unit's end
  const int bpp = c.P / kInt4Block;
  auto window = [&](int w) {
    const int x = w * 32 + lane;
    if (w * 32 >= nb) return 0;
    // the units of the window's first and last block, and the lane's between them
    const int u0 = unit_at(P, U, 0, b0 + w * 32, lane), u1 = unit_at(P, U, 0, b0 + min(w * 32 + 31, nb - 1), lane);
    if (x >= nb) return 0;
    const int u = u0 + unit_of(P + u0, u1 - u0 + 1, b0 + x), b = u / Hkv, bi = b0 + x - P[u], pi = bi / bpp;
    int pg = c.block_table[static_cast<int64_t>(b) * c.bt_stride + pi];
    if (pg < 0 || pg >= c.n_rows) {
      raise_error(args.err, ERR_INDEX);
      pg = 0;
    }
    return (pg * Hkv + (u - b * Hkv)) * bpp + bi - pi * bpp;
  };
  const uint64_t policy = l2_evict_first_policy();
  uint32_t copies = 0;  // stages with copies in flight; bit 8 + stage: parity of its next wait
  bool failed = false;
  int win = window(0), win_next = window(1), win_at = 0;
  int ix = 0, iu = u_first, iend = nb > 0 ? min(P[iu + 1] - b0, nb) : 0, is = 0;
  bool withhold = (args.debug_flags & kDebugWithholdQ) != 0;
  auto issue = [&]() {
    if (ix >= nb) return;
    const int n = min(KG, iend - ix);
    if ((ix >> 5) != win_at) {
      win = win_next;
      ++win_at;
      win_next = window(win_at + 1);
    }
    const int r0 = __shfl_sync(kFull, win, ix & 31);
    const int r1 = __shfl_sync(kFull, ((ix + 1) >> 5) == win_at ? win : win_next, (ix + 1) & 31);
    if (lane == 0 && !withhold) {
      const uint32_t bar = bar0 + 8 * is, dst = ring_a + is * 2 * Gm::HALF;
      const uint8_t* k = reinterpret_cast<const uint8_t*>(c.k) + static_cast<int64_t>(r0) * BLK;
      const uint8_t* v = reinterpret_cast<const uint8_t*>(c.v) + static_cast<int64_t>(r0) * BLK;
      const bool joined = n == 2 && r1 == r0 + 1;
      const uint32_t bytes = joined ? 2 * BLK : BLK;
      mbar_arrive_expect_tx(bar, 2u * n * BLK);
      bulk_copy_g2s(dst, k, bytes, bar, policy);
      bulk_copy_g2s(dst + Gm::HALF, v, bytes, bar, policy);
      if (n == 2 && !joined) {
        const int64_t at = static_cast<int64_t>(r1) * BLK;
        bulk_copy_g2s(dst + BLK, reinterpret_cast<const uint8_t*>(c.k) + at, BLK, bar, policy);
        bulk_copy_g2s(dst + Gm::HALF + BLK, reinterpret_cast<const uint8_t*>(c.v) + at, BLK, bar, policy);
      }
    }
    if (!withhold) copies |= 1u << is;
    withhold = false;
    ix += n;
    if (ix == iend && ix < nb) {
      do ++iu;
      while (P[iu + 1] == P[iu]);
      iend = min(P[iu + 1] - b0, nb);
    }
    is = is + 1 == NS ? 0 : is + 1;
  };
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < NS; ++i) issue();

  // (while they are on their way)
  Span* spans = reinterpret_cast<Span*>(smem + Gm::SPAN_OFF);
  if (nb > 0 && lane < 2) spans[2 * warp + lane] = span_of(cs, lane == 0 ? u_first : unit_of(P, U, b0 + nb - 1));

  // ---- the warp's units
  int x = 0, st = 0, u = u_first, staged = 0;
  bool lost_inputs = false;
  auto wait_inputs = [&]() {
    if (!failed) {
      const bool ok = mbar_wait_bounded(inbar, staged & 1, args.wait_ns);
      if (__all_sync(kFull, ok)) {
        ++staged;
      } else {
        failed = lost_inputs = true;
        if (lane == 0) raise_error(args.err, ERR_TIMEOUT);
      }
    }
  };
  auto restage = [&](int unit, bool token) {  // (the scratch was read and written by loads and stores)
    if (failed) return;
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) stage_inputs<D, GP>(args, unit, token, smem_addr(scratch), inbar);
  };
  // Jobs: the units of the range, then the warp's share of the units without cached tokens.
  int bare = worker - NC * W;
  bool first_job = true;
  for (;;) {
    const bool cached = x < nb;
    if (!cached) {
      do bare += NC * W;
      while (bare < U && P[bare + 1] != P[bare]);
      if (bare >= U) break;
      u = bare;
    }
    const int end = cached ? min(P[u + 1] - b0, nb) : x;
    const bool from_start = !cached || b0 + x == P[u], to_end = !cached || b0 + end == P[u + 1];
    if (!first_job || !cached) restage(u, from_start);
    first_job = false;
    wait_inputs();
    prepare<D, GP>(a, u, from_start, scratch, lane);
    if (cached) {
      Warp q4;
      if constexpr (Warp::kSharedQ) Warp::put_query(scratch, reinterpret_cast<uint8_t*>(scratch), lane);
      q4.get_query(scratch, reinterpret_cast<const uint8_t*>(scratch), lane);
      q4.clear();
      __syncwarp();
      int left = N[u] - (b0 + x - P[u]) * kInt4Block;  // tokens from block x on
#pragma unroll 1
      while (x < end) {
        if (!failed) {
          const bool ok = mbar_wait_bounded(bar0 + 8 * st, (copies >> (8 + st)) & 1u, args.wait_ns);
          if (__all_sync(kFull, ok)) {
            copies = (copies & ~(1u << st)) ^ (0x100u << st);
          } else {
            failed = true;
            if (lane == 0) raise_error(args.err, ERR_TIMEOUT);
          }
        }
        if (!failed) {
          uint8_t* kb = ring + st * 2 * Gm::HALF;
          uint32_t masks[KG];
#pragma unroll
          for (int i = 0; i < KG; ++i) {
            const int n = x + i < end ? left - i * kInt4Block : 0;
            masks[i] = n >= kInt4Block ? 0xffffu : (1u << max(n, 0)) - 1u;
            if (masks[i] != 0xffffu) Warp::clear_rows(kb + Gm::HALF + i * BLK, masks[i], lane);
          }
          q4.template blocks<KG>(kb, kb + Gm::HALF, masks, reinterpret_cast<const uint8_t*>(scratch), lane);
          __syncwarp();
          issue();
        }
        x = min(x + KG, end);
        left -= KG * kInt4Block;
        st = st + 1 == NS ? 0 : st + 1;
      }
      // its state: a whole unit's in the scratch; at a unit's end with others behind it in
      // global memory; the last one's in the ring, which is idle now (unless a wait gave up)
      __syncwarp();
      const bool whole = from_start && to_end, last = x == nb;
      float* state = whole || (last && failed) ? scratch
                     : last                    ? reinterpret_cast<float*>(ring)
                                               : args.wpart + static_cast<int64_t>(worker) * Gm::STATE;
      q4.finish(state, state + GP * D, GP, lane);
      if (!whole && lane == 0) SEG[2 * warp + (last ? 1 : 0)] = u;
    }
    if (from_start && to_end) {
      if (lane == 0) list[0] = scratch;
      __syncwarp();
      wait_prev();
      finish_unit<D, GP>(a, u, list, cached ? 1 : 0, Team{lane, 32, 0});
      __syncwarp();
    }
    if (x < nb) {
      do ++u;
      while (P[u + 1] == P[u]);
    }
  }
  // copies in flight exist only after a wait gave up: let them land
  if (lane == 0) {
    for (int i = 0; i < NS; ++i)
      if ((copies >> i) & 1u) mbar_wait_bounded(bar0 + 8 * i, (copies >> (8 + i)) & 1u, args.wait_ns);
    if (lost_inputs) mbar_wait_bounded(inbar, staged & 1, args.wait_ns);
  }
  wait_prev();
  __syncthreads();

  // ---- the CTA's states: entry 2 w is what warp w left in global memory, 2 w + 1 what lies
  // in its ring; a unit's entries follow one another
  const int mine = lane < 2 * W ? SEG[lane] : -1;
  const unsigned some = __ballot_sync(kFull, mine >= 0), below = some & ((1u << lane) - 1u);
  const int before = __shfl_sync(kFull, mine, below ? 31 - __clz(below) : lane);
  unsigned starts = __ballot_sync(kFull, mine >= 0 && (!below || before != mine));
  // a team for each unit: all warps for one, shares of them for several, a warp each for
  // more units than warps
  const int runs = __popc(starts), width = runs > 0 ? max(W / runs, 1) : 1;
  for (int r = 0; starts; ++r) {
    const int first = __ffs(starts) - 1;
    starts &= starts - 1;
    const int last = starts ? __ffs(starts) - 1 : 2 * W, w0 = r * width % W;
    if (warp < w0 || warp >= w0 + width) continue;
    const float** lst = reinterpret_cast<const float**>(smem + Gm::LIST_OFF) + w0 * 32;
    const unsigned have = __ballot_sync(kFull, lane >= first && lane < last && mine >= 0);
    if (warp == w0 && ((have >> lane) & 1u))
      lst[__popc(have & ((1u << lane) - 1u))] = lane & 1 ? reinterpret_cast<const float*>(smem + (lane >> 1) * Gm::RING)
                                                        : args.wpart + static_cast<int64_t>(cta * W + (lane >> 1)) * Gm::STATE;
    const Team tm{static_cast<int>(threadIdx.x) - w0 * 32, width * 32, 1 + w0 / width};
    tm.sync();
    merge_unit<D, GP>(a, cs, SEG[first], spans[first], cta, lst, __popc(have), flag + w0, tm);
  }
}

template <int D, int NT>
cudaError_t launch(const Int4DecodeArgs& a, int ctas, cudaStream_t s) {
  using Gm = Geo4<D, NT>;
  auto k = int4_decode_kernel<D, NT>;
  static std::atomic<uint64_t> opted{0};
  const cudaError_t e = opt_in_smem(k, Gm::SMEM_MAX, opted);
  if (e != cudaSuccess) return e;
  const size_t smem = 128 + Gm::TAB_OFF + (2 * a.B * a.Hkv + 1) * sizeof(int);
  return a.late ? launch_pdl_waiting(k, dim3(ctas), dim3(Gm::THREADS), smem, s, a)
                : launch_pdl(k, dim3(ctas), dim3(Gm::THREADS), smem, s, a);
}

}  // namespace

int int4_decode_ctas(int units, int n_max, int D, int GP, int num_sms) {
  const int W = D == 256 ? Geo4<256, 1>::W : GP == 4 ? Geo4<128, 1>::W : Geo4<128, 2>::W;
  const int64_t blocks = static_cast<int64_t>(units) * ((static_cast<int64_t>(n_max) + kInt4Block - 1) / kInt4Block + kUnitCost);
  const int64_t ctas = (blocks + kMinBlocks * W - 1) / (kMinBlocks * W);
  return static_cast<int>(ctas < 1 ? 1 : ctas > num_sms ? num_sms : ctas);
}

cudaError_t launch_decode_int4(const Int4DecodeArgs& args, int D, int ctas, cudaStream_t s) {
  static_assert(Geo4<128, 1>::W <= kInt4Warps && Geo4<128, 2>::W <= kInt4Warps && Geo4<256, 1>::W <= kInt4Warps &&
                    Geo4<256, 2>::W == Geo4<256, 1>::W, "the workspace's warps");
  Int4DecodeArgs a = args;
  if (a.wait_ns == 0) a.wait_ns = kDefaultWaitNs;
  const int GP = decode_group_pad(a.G);
  if (a.B * a.Hkv > kMaxUnits || a.r > D || a.r % 2 != 0) return cudaErrorNotSupported;
  if (D == 128) return GP == 4 ? launch<128, 1>(a, ctas, s) : launch<128, 2>(a, ctas, s);
  if (D == 256) return GP == 4 ? launch<256, 1>(a, ctas, s) : launch<256, 2>(a, ctas, s);
  return cudaErrorNotSupported;
}

}  // namespace dattn
