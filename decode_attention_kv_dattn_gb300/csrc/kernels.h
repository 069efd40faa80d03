// Internal interface between the host planner (dattn.cu) and the kernel
// translation units. Not part of the public C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cmath>
#include <utility>

namespace dattn {

// RoPE angle step of pair i of an r-dim rotation with base theta, in 64-bit
// fixed-point turns per position: rint(2^64 * theta^(-2i/r) / 2pi), the
// frequency and the division by 2pi each rounded to fp64.
inline uint64_t rope_phase_step(double theta, int r, int i) {
  const double inv_freq = std::pow(theta, -static_cast<double>(2 * i) / static_cast<double>(r));
  return static_cast<uint64_t>(std::llrint(std::ldexp(inv_freq / 6.283185307179586, 64)));
}

// Sticky device error bits (see dattn_get_error).
enum : int { ERR_INDEX = 1, ERR_TIMEOUT = 2, ERR_LENGTH = 4, ERR_RANGE = 8 };

// Limit of a bounded device wait unless the handle sets another (2 s).
constexpr uint64_t kDefaultWaitNs = 2000000000ull;
// Testing aid (dattn_debug_config): the decode kernel's helper warp withholds
// the first unit's rotated query, so the streaming warps' waits run out. Prompts of
// state layers: a CTA's first Q tile is not copied, or, in the pass that sums what
// the ranges contribute, its first K and V.
constexpr int kDebugWithholdQ = 1;
constexpr int kDebugWithholdKV = 2;

// One layer's cache as the kernels see it.
struct CacheView {
  uint16_t* k;                 // ring [n_rows, Hkv, R, D] / paged [pages, Hkv, P, D]
  uint16_t* v;
  int paged;                   // 0 = ring, 1 = paged
  int n_rows;                  // ring rows or pages in the pool
  int R;                       // ring slots
  int P;                       // page size
  const int32_t* ring_head;    // [B]
  const int32_t* ring_count;   // [B]
  const int32_t* stream_rows;  // [B] or null
  const int32_t* block_table;  // [B, bt_stride]
  int bt_stride;
  const int32_t* seq_len;      // [B]
};

// RoPE prologue: rotates q (fp32 out, pre-scaled) and k (bf16 entry out) of
// `rows` token rows. Decode: row = stream, position pos[row]. Verify: row =
// s * T + i, position prefix_len[s] + depth(i) from the parent array.
struct RopeArgs {
  int rows;
  int Hq, Hkv, D, r;
  const uint16_t* q;           // [rows, Hq, D]
  const uint16_t* k;           // [rows, Hkv, D]
  const int32_t* pos;          // [rows] (decode) or null
  const int32_t* prefix_len;   // [rows / T] (verify) or null
  const int32_t* parent;       // [rows] (verify) or null
  int T;
  const uint64_t* rope_step;   // [r / 2] phase steps (rope_phase_step)
  float q_scale;               // log2(e) / sqrt(D)
  float* qhat;                 // [rows, Hq, D]
  uint16_t* qhl;               // [2][qhl_rows, Hq, D]: the same values as bf16 hi, then the
                               // bf16 rounding of what is left (lo), or null
  int qhl_rows;                // rows of one plane of qhl (its capacity)
  uint16_t* khat;              // [rows, Hkv, D]
  int* err;
  const uint16_t* q_norm;      // [D] QK-norm weights, or null
  const uint16_t* k_norm;
  double norm_eps;
  // Row r = s * T + i reads the caller's q/k row s * in_T + row0 + i (a
  // prefill chunk of a longer array; rows past in_T read as zero). Verify:
  // in_T = T, row0 = 0.
  int in_T, row0;
};

// Query heads of a KV group as the decode kernel lays them out: 4 (G <= 4)
// or 8 (G <= 8); 0 for a group size with no compiled kernel.
inline int decode_group_pad(int G) { return G <= 0 ? 0 : (G <= 4 ? 4 : (G <= 8 ? 8 : 0)); }

// One decode call (RoPE of the new token, the pass over the cached keys, the
// join in score space, gate, store, write-back) as one launch. Stream-K: the
// grid cuts the concatenated tiles of all (stream, KV head) units into equal
// ranges. Partial slot of a segment: the CTA index for the first segment of a
// CTA's range, gridDim + unit for any later one; the CTA that finishes a
// unit's last segment (per-unit counter) combines the unit.
struct DecodeArgs {
  CUtensorMap tmap_k;          // the layer's K cache as a 2D [rows, D] bf16 tensor
  CUtensorMap tmap_v;          // (encode_cache_maps)
  CacheView c;
  int B, Hkv, G;
  int max_len;                 // host bound on cached length (paged)
  const uint16_t* q;           // [B, Hq, D]
  const uint16_t* k_new;       // [B, Hkv, D]
  const uint16_t* v_new;       // [B, Hkv, D]
  const uint16_t* gate;        // [B, Hq] or null
  const int32_t* pos;          // [B]
  const uint64_t* rope_step;   // [r / 2] phase steps (rope_phase_step)
  int r;
  float q_scale;               // log2(e) / sqrt(D)
  float* out;                  // [B, Hq, D]
  int write_back;
  float* part;                 // [ctas + B*Hkv][GP*(D+2)]: o[GP][D], m[GP], l[GP]
                               // (GP = decode_group_pad(G))
  int* counters;               // [B*Hkv] finished segments, then [ctas] group counters; zero between calls
  int* err;
  int early;                   // nonzero: the preceding launch on the stream writes
                               // no part of this cache, so the first cache loads may
                               // start before it completes
  int unit_cost;               // fixed cost of one segment of a unit, in stage tiles
                               // (set by launch_decode)
  uint64_t wait_ns;            // limit of every bounded wait (0 = kDefaultWaitNs)
  int debug_flags;             // kDebugWithholdQ: see dattn_debug_config
  const uint16_t* q_norm;      // [D] QK-norm weights of the queries, or null
  const uint16_t* k_norm;      // [D] of the new key, or null
  double norm_eps;
  // E4M3 cache (the pools hold bytes; k, v of CacheView are byte arrays):
  // cached value = e4m3 * scale. q_scale then includes k_scale.
  int f8;
  float k_scale, v_scale;
};

// The same over a 4-bit cache (int4_format.h; the pools are byte arrays). A unit's blocks
// of 16 tokens are split over the warps of all CTAs.
struct Int4DecodeArgs {
  CacheView c;
  int B, Hkv, G;
  int max_len;                 // host bound on cached length
  const uint16_t* q;           // [B, Hq, D]
  const uint16_t* k_new;       // [B, Hkv, D]
  const uint16_t* v_new;       // [B, Hkv, D]
  const uint16_t* gate;        // [B, Hq] or null
  const int32_t* pos;          // [B]
  const uint64_t* rope_step;   // [r / 2]
  int r;
  float q_scale;               // log2(e) / sqrt(D)
  float* out;                  // [B, Hq, D]
  int write_back;
  float* part;                 // [ctas + B*Hkv][GP*(D+2)]: as DecodeArgs::part
  float* wpart;                // [ctas * warps][GP*(D+2)]: a warp's state of a unit that it leaves for another
  float* gpart;                // [ctas][GP*(D+2)]: the states of groups of CTAs
  uint8_t* token;              // [B*Hkv][int4_token_bytes]: the new token of a unit, quantised and scored
  int* counters;               // [B*Hkv] CTAs done with a unit, then [ctas] of groups; zero between calls
  int* err;
  int early;                   // as DecodeArgs::early
  int late;                    // the launch before may be writing the inputs: they are fetched after the wait
  uint64_t wait_ns;
  int debug_flags;
  const uint16_t* q_norm;      // [D] or null
  const uint16_t* k_norm;
  double norm_eps;
};

// Page summaries: the bf16 mean of a page's stored keys (times k_scale), for
// every page whose last token is among a row's `count` new tokens.
struct SummarizeArgs {
  CacheView c;
  int B, Hkv, max_tokens;
  const int32_t* start_index;  // [B]
  const int32_t* count;        // [B]
  uint16_t* summary;           // [pages, Hkv, D]
  int f8;
  float k_scale;
  int* err;
};

// Decode over selected pages: one launch scores the candidate pages [keep_first,
// pages - keep_last) of every (stream, KV head) unit with more than num_pages
// pages and selects, a second one attends to the selected pages.
struct PageArgs {
  CacheView c;
  int B, Hkv, G;
  int max_len;                 // host bound on cached length
  int num_pages, keep_first, keep_last;
  const uint16_t* q;           // [B, Hq, D]
  const uint16_t* k_new;       // [B, Hkv, D]
  const uint16_t* v_new;       // [B, Hkv, D]
  const uint16_t* gate;        // [B, Hq] or null
  const int32_t* pos;          // [B]
  const uint64_t* rope_step;
  int r;
  const uint16_t* q_norm;      // [D] or null
  const uint16_t* k_norm;
  double norm_eps;
  float* out;                  // [B, Hq, D]
  int write_back;
  const uint16_t* summary;     // [pages, Hkv, D]
  int32_t* selected;           // [units, num_pages] logical pages, or null
  // scores and selection
  int chunk_pages, chunks;     // pages of a CTA, CTAs of a unit
  int pitch;                   // entries between units' scores
  float* scores;               // [units, pitch]
  float* tile_max;             // [units, tile_pitch]: largest score of each 16 pages
  int tile_pitch;
  float* cinfo;                // [units, chunks][3]: least and largest score, bound of the summaries' norms
  float* qnorm;                // [units] bound of the group's query norms
  uint64_t* keys;              // [units, pitch] scratch of a border with many pages
  int* done;                   // [units] finished chunks; zero between calls
  int32_t* table;              // [units, num_pages] physical pages selected
  int q64_off, qf_off, staged_off;  // shared-memory layout, and the scores that have room in it (set by
  int staged;                  // launch_page_select; a multiple of 128)
  // attention
  int splits;                  // CTAs of a unit
  float q_scale;               // log2(e) / sqrt(D), with k_scale for E4M3
  float k_scale, v_scale;      // E4M3
  float* part;                 // [units * splits][G * (D + 2)]
  int* counters;               // [units] finished splits; zero between calls
  int* err;
};

// Linear attention over a state S [D, D] for each (row, KV head), with the
// head's decay lam: S = lam S + k v^T, out = q^T S / sqrt(D).
constexpr int kLinearChunk = 64;  // tokens of a chunk of the prompt form
constexpr int kDecayStride = kLinearChunk + 3;
struct LinearArgs {
  CUtensorMap tmap_q;          // prompt: q, k, v as (D, heads, B * T) bf16, boxes of (64 dims, 2 heads for q
  CUtensorMap tmap_k;          // (1 where G is 1) or 1, 64 tokens), 128-byte swizzled
  CUtensorMap tmap_v;
  float* state;                // [n_rows, Hkv, D, D], row = key dim
  int n_rows;
  const int32_t* stream_rows;  // [B] or null
  int B, Hkv, G;
  const uint16_t* q;           // [B, (T,) Hq, D]
  const uint16_t* k;           // [B, (T,) Hkv, D]
  const uint16_t* v;
  const uint16_t* gate;        // [B, (T,) Hq] or null
  float* out;                  // [B, (T,) Hq, D]
  const float* decay;          // [Hkv][kDecayStride]: lam^0 .. lam^C in fp32, then what that drops of lam
                               // (C + 1) and of lam^C (C + 2)
  const float* log_decay;      // [Hkv] log lam
  float scale;                 // 1 / sqrt(D)
  int write_back;              // step: store the new state
  int T;                       // prompt: tokens of a row's arrays
  const int32_t* count;        // prompt: [B]
  float* sums;                 // prompt: [2][num_sms][D, EB] a CTA's slot: its last piece's contribution to the
                               // state, then the state that the next CTA starts from; and the state that its
                               // last unit starts from. Behind them a note a CTA, and two words: whether this
                               // call's sums gave up waiting, and the same for the main pass (zero between calls)
  int split;                   // prompt: units may be cut into ranges of chunks, by `ctas` CTAs (else one each)
  int ctas;
  int* err;
  uint64_t wait_ns;            // prompt: limit of the bounded waits
  int debug_flags;             // prompt: kDebugWithholdQ, kDebugWithholdKV
};

struct AppendArgs {
  CacheView c;
  int B, Tmax, Hkv, D, r;
  const int32_t* start_index;
  const int32_t* start_pos;
  const int32_t* count;
  const uint16_t* k;           // [B, Tmax, Hkv, D]
  const uint16_t* v;
  int rotate;
  const uint64_t* rope_step;   // [r / 2]
  int* err;
  const uint16_t* k_norm;      // [D] QK-norm weights of the keys (with rotate), or null
  double norm_eps;
  // source rows: b * in_T + row0 + t of k/v (in_T = Tmax, row0 = 0 but for
  // prefill chunks)
  int in_T, row0;
  // E4M3 pools: entries stored as the E4M3 bytes nearest entry / k_scale
  // (K) and v / v_scale (V)
  int f8;
  float k_scale, v_scale;
  // commit of verify paths: token t of row b is source row gather[b * Tmax + t]
  // of k/v ([B, Tmax, Hkv, D]), and the row's first count[b] entries of gather
  // must form a path from a root under parent [B, Tmax]; null for a plain append
  const int32_t* gather;
  const int32_t* parent;
};

// Cached entries [start_index, start_index + count) of each row back as bf16.
struct ReadArgs {
  CacheView c;
  int B, Tmax, Hkv, D;
  const int32_t* start_index;  // [B]
  const int32_t* count;        // [B]
  uint16_t* k;                 // out [B, Tmax, Hkv, D]
  uint16_t* v;
  float k_scale, v_scale;      // E4M3
  int* err;
};

// Tensor-core pass of tree verify over each stream's paged prefix (stream-K
// over (stream, KV head) units and their 128-key tiles; the G*T rows of a
// unit are one 128-row MMA tile).
// Partial slot layout: [ctas + S*Hkv][G*T rows][D + 4] fp32 (o[D], m, l, pad),
// row g * T + i for query head g of the group and tree node i.
struct VerifySplitArgs {
  CUtensorMap tmap_k;          // the layer's K pool as [rows, D] bf16, boxes of 16 rows x 64 dims
  CUtensorMap tmap_v;          // its V pool as (64 dims, rows, D/64 regions), boxes of (64, 16, D/64)
  CUtensorMap tmap_q;          // q hi/lo as (D, Hq, S*T, 2) bf16, boxes of (64, G, T, 1)
  CacheView c;                 // paged (page size a multiple of 16; seq_len = prefix lengths)
                               // or ring (all R slots scanned, the valid ones kept)
  int S, T, Hkv, G;
  const int32_t* parent;       // [S, T] (ring layers: a row's depth sets how many of the
                               // oldest entries its path pushed out)
  const uint16_t* qhl;         // [2][qhl_rows, Hq, D]: q as bf16 hi (the first plane) and lo
  int ctas;
  int max_len;
  float* part;
  int* tiles;                  // out, U = S*Hkv: [U + 1] tile prefix over units, then per
                               // unit the first CTA of its span [U], the span's length [U]
                               // and the partial slot of its first segment [U]
  int* err;
};

// Ragged prefill in chunks of Tc tokens: the cache state a chunk starts from
// (the caller's plus the min(count, row0) tokens of earlier chunks) and the
// chunk's token count and root position, per stream, into scratch arrays.
struct PrefillMetaArgs {
  CacheView c;                 // the caller's cache metadata
  const int32_t* count;        // [S] new tokens of each stream (0..Tmax)
  const int32_t* start_pos;    // [S] position of each stream's token 0
  int S, Tmax, row0, Tc;
  int32_t* seq_c;              // paged: seq_len + m
  int32_t* head_c;             // ring: (head + m) mod R
  int32_t* cnt_c;              // ring: min(count + m, R)
  int32_t* pos_c;              // start_pos + row0
  int32_t* n_c;                // tokens of this chunk: clamp(count - row0, 0, Tc)
  int32_t* chain;              // [S, Tc] chain-tree parents: i - 1
  int* err;
};
cudaError_t launch_prefill_meta(const PrefillMetaArgs& a, cudaStream_t s);

// Tree-window join: merge the prefix segments of each row, score the row's
// path in the window (its ancestors and itself), gate, store, write back.
struct VerifyCombineArgs {
  CacheView c;
  int S, T, Hkv, G;
  int split_ctas;
  const int* tiles;            // written by the split pass (VerifySplitArgs::tiles)
  int max_len;
  const float* qhat;           // [S*T, Hq, D]
  const uint16_t* khat;        // [S*T, Hkv, D] rotated window keys (bf16 entries)
  const uint16_t* v;           // [S, T, Hkv, D]
  const int32_t* parent;       // [S, T]
  const uint16_t* gate;        // [S, T, Hq] or null
  const float* part;
  float* out;                  // [S, T, Hq, D]
  int write_back;
  int* err;
  // caller rows of v, gate and out: s * in_T + row0 + i (see RopeArgs); with
  // rows_valid, only rows i < rows_valid[s] are stored (prefill chunks)
  int in_T, row0;
  const int32_t* rows_valid;
};

// Decode grid: every resident CTA (`resident` on the whole GPU), but at
// least 4 stage tiles (one per streaming warp) per CTA for the largest amount
// of work the call may have: `units` units of up to `n_max` keys each.
inline int plan_decode_ctas(int resident, int units, int n_max, int tile_keys) {
  const int64_t tiles = static_cast<int64_t>(units) * ((n_max + tile_keys - 1) / tile_keys);
  int64_t ctas = (tiles + 3) / 4;
  if (ctas > resident) ctas = resident;
  if (ctas < 1) ctas = 1;
  return static_cast<int>(ctas);
}

// Each returns cudaErrorNotSupported for a shape with no compiled kernel.
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s, bool pdl = true);
// Decode with `ctas` CTAs (at most decode_ctas_per_sm per SM). With pdl the
// launch is a programmatic dependent of the previous one on the stream;
// without, it starts once everything before it on the stream has completed.
cudaError_t launch_decode(const DecodeArgs& a, int D, int ctas, cudaStream_t s, bool pdl = true);
// Tensor maps of a cache's K and V for the decode kernel over its [n_rows *
// Hkv * (R or P), D] bf16 rows, 128-byte swizzle: at D = 128 seen as (64 dims,
// row, 2 regions) with one box per 16-row group; at D = 256 as [rows, D] with
// boxes of 16 rows x 64 dims.
cudaError_t encode_cache_maps(const CacheView& c, int Hkv, int D, CUtensorMap* k, CUtensorMap* v, bool f8 = false);
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s);
// the same into a 4-bit cache (no gather), and the read-back of any format
cudaError_t launch_append_int4(const AppendArgs& a, cudaStream_t s);
cudaError_t launch_read(const ReadArgs& a, bool int4, bool f8, cudaStream_t s);
// decode over an E4M3 cache (decode_fp8.cu); GP = decode_group_pad(G)
cudaError_t launch_decode_fp8(const DecodeArgs& a, int D, int GP, int ctas, cudaStream_t s, bool pdl);
// decode over a 4-bit cache: CTAs of a call, the floats of a warp's state and the bytes of
// a unit's token in the workspace (per (stream, KV head)), the most warps of a CTA.
int int4_decode_ctas(int units, int n_max, int D, int GP, int num_sms);
constexpr size_t int4_token_bytes(int D, int GP) { return 8 * static_cast<size_t>(GP) + D + D / 8; }
constexpr int kInt4Warps = 12;
cudaError_t launch_decode_int4(const Int4DecodeArgs& a, int D, int ctas, cudaStream_t s);
cudaError_t launch_verify_split(const VerifySplitArgs& a, int D, cudaStream_t s);
cudaError_t launch_verify_combine(const VerifyCombineArgs& a, int D, cudaStream_t s);
// Keys per tile of the verify pass and its largest unit count.
constexpr int kVerifyTileKeys = 128;
// Fixed cost of one unit segment of the verify pass's split, in tiles.
constexpr int kVerifySegmentCost = 2;
constexpr int kVerifyMaxUnits = 512;
// Most rows (G * T) of a verify unit: one 128-row MMA tile.
constexpr int kVerifyMaxRows = 128;
// Tensor maps of the verify pass: the K pool as [rows, D] bf16 with boxes of
// 16 rows x 64 dims, the V pool as (64, rows, D/64) with boxes of (64, 16,
// D/64) (a 16-row group, all dims), and q hi/lo (qhl, planes of qhl_rows
// rows) as (D, Hq, S*T, 2) bf16 with boxes of (64, G, T, 1); all 128-byte
// swizzled.
cudaError_t encode_verify_maps(const CacheView& c, int Hkv, int D, const uint16_t* qhl, int qhl_rows, int Hq,
                               int G, int S, int T, CUtensorMap* k, CUtensorMap* v, CUtensorMap* q);

// Resident CTAs per SM of the decode kernel for (D, G) (0 if unsupported).
int decode_ctas_per_sm(int D, int G);
// Keys per stage tile of the decode kernel for (D, G).
int decode_tile_keys(int D, int G, bool f8 = false);
// Largest number of (stream, KV head) units of one decode call.
int decode_max_units();

cudaError_t launch_summarize(const SummarizeArgs& a, int D, cudaStream_t s);
// Pages of a CTA of the scores, for `units` units of up to `pages` pages, and
// the least it ever is (sizes the workspace).
int page_chunk_pages(int units, int pages, int num_sms);
constexpr int kPageChunkMin = 128;
// CTAs of a unit in the attention over up to `groups` 16-key groups.
int page_splits(int units, int groups, int num_sms);
// Shared memory of the selection: a bitmap of a stream's pages, the group's
// query in fp64 and up to 16,384 scores.
constexpr int kSelectBitmapMax = 96 * 1024;
constexpr int kSelectSmemMax = kSelectBitmapMax + (17 + 8 + 65) * 1024;
cudaError_t launch_page_select(PageArgs a, int D, cudaStream_t s);
cudaError_t launch_page_attend(const PageArgs& a, int D, bool f8, cudaStream_t s);
cudaError_t launch_linear_step(const LinearArgs& a, int D, int num_sms, cudaStream_t s);
// The prompt form: one launch, or three where the units' chunks are split.
cudaError_t launch_linear_prompt(const LinearArgs& a, int D, int num_sms, cudaStream_t s);
cudaError_t encode_linear_maps(LinearArgs& a, int D);

// Launch order per stream (launch_order.h).
// True when the last launch recorded on `stream` writes into the cache whose
// K array is `cache_k`.
bool prev_launch_writes(void* stream, const void* cache_k);
// Record a launch made on `stream` that writes into the cache with K array
// `cache_k` (null: writes no cache), or one whose results may be the next call's inputs.
void record_launch(void* stream, const void* cache_k);
void record_results(void* stream);
// Whether the next launch on `stream` has to come behind the whole of the last one, and
// that one has been made that does.
bool launch_in_order(void* stream);
void launch_started(void* stream);

// Raise `kernel`'s dynamic shared-memory limit to `bytes` on the current
// device, once per device (`done` holds one bit per device id below 64; the
// call is idempotent, so racing threads at worst repeat it).
template <typename Kernel>
cudaError_t opt_in_smem(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? (1ull << dev) : 0ull;
  if (bit != 0ull && (done.load(std::memory_order_acquire) & bit) != 0ull) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit != 0ull) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_as(bool programmatic, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                      cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = programmatic ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Launch with programmatic stream serialization: the kernel may begin while
// its predecessor in the stream finishes; every kernel here waits on the
// predecessor (griddepcontrol.wait) before it touches the predecessor's output -
// except for what is its input, so behind a launch of such results it has no such leave.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args&&... args) {
  const bool in_order = launch_in_order(stream);
  const cudaError_t e = launch_as(!in_order, kernel, grid, block, smem, stream, std::forward<Args>(args)...);
  if (in_order && e == cudaSuccess) launch_started(stream);
  return e;
}

// The same of a kernel that reads no inputs before it waits: behind such a launch it
// may begin early, and what it lets begin in turn comes after its wait.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_waiting(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                               cudaStream_t stream, Args&&... args) {
  const cudaError_t e = launch_as(true, kernel, grid, block, smem, stream, std::forward<Args>(args)...);
  if (e == cudaSuccess) launch_started(stream);
  return e;
}

}  // namespace dattn
