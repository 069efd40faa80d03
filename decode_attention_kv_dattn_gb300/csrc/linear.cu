// Linear attention with a decay for each head: the layers whose cache is one
// fp32 state S [D, D] (row = key dim, column = value dim) for each (row, KV
// head), whatever the context's length.
//
//   S_t = lam S_{t-1} + k_t v_t^T,   o_t = sigmoid(gate) q_t^T S_t / sqrt(D)
//
// with lam = exp(log_decay[h]) and the group's query heads reading their KV
// head's state. lam is held as fp32 hi + lo: a decay near 1 acts over many
// tokens, and an error of 2^-25 in each step would grow with that reach.
#include "linear.cuh"

namespace dattn {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kStepThreads = 256;

// ---------------------------------------------------------------- one token

// One CTA per (unit, W columns of the state). Each thread holds 4 columns of
// every RP-th row: the update and the group's dot products are done on the
// registers between one read and one write of the state, which bound the step
// (2 D^2 fp32 a unit): 64 streams of 8 heads of 128, 67 MB, 7.9 us in a graph
// that repeats the step (the states then stay in the L2 cache; 10 us at the
// memory's rate), 1 stream of 2 heads of 256 2.1 us.
template <int D, int W, int GP>
__global__ void __launch_bounds__(kStepThreads) linear_step_kernel(const LinearArgs a) {
  constexpr int LPR = W / 4;                // lanes of a row
  constexpr int RP = kStepThreads / LPR;    // rows of a pass
  constexpr int R = D / RP;                 // rows of a thread
  constexpr int RB = R < 8 ? R : 8;         // rows in flight a thread
  constexpr int SLICES = D / W;
  __shared__ float ks[D];
  __shared__ __align__(16) float qs[D * GP];
  __shared__ float red[kStepThreads / 32][GP][W];
  const int u = blockIdx.x / SLICES, slice = blockIdx.x - u * SLICES;
  const int b = u / a.Hkv, h = u - b * a.Hkv;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int row0 = t / LPR, col = slice * W + (t % LPR) * 4;
  // inputs: the caller's, not written by the launch before
  for (int d = t; d < D; d += kStepThreads) {
    ks[d] = bf16_to_f32(a.k[static_cast<int64_t>(u) * D + d]);
#pragma unroll
    for (int g = 0; g < GP; ++g)
      qs[d * GP + g] = g < a.G ? bf16_to_f32(a.q[(static_cast<int64_t>(u) * a.G + g) * D + d]) : 0.f;
  }
  const uint2 vw = *reinterpret_cast<const uint2*>(a.v + static_cast<int64_t>(u) * D + col);
  const float v[4] = {bf16_lo(vw.x), bf16_hi(vw.x), bf16_lo(vw.y), bf16_hi(vw.y)};
  const float lam = a.decay[h * kDecayStride + 1], lam_lo = a.decay[h * kDecayStride + kLinearChunk + 1];
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int row = state_row(a, b, t == 0 && h == 0 && slice == 0);
  float* S = a.state + (static_cast<int64_t>(max(row, 0)) * a.Hkv + h) * D * D + col;
  float acc[GP][4];
#pragma unroll
  for (int g = 0; g < GP; ++g) acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.f;
#pragma unroll
  for (int r0 = 0; r0 < R; r0 += RB) {
    float4 w[RB];
#pragma unroll
    for (int x = 0; x < RB; ++x)
      w[x] = row >= 0 ? *reinterpret_cast<const float4*>(S + static_cast<int64_t>(row0 + (r0 + x) * RP) * D)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < RB; ++x) {
      const int d = row0 + (r0 + x) * RP;
      const float kd = ks[d];
      w[x].x = fmaf(w[x].x, lam, fmaf(w[x].x, lam_lo, kd * v[0]));
      w[x].y = fmaf(w[x].y, lam, fmaf(w[x].y, lam_lo, kd * v[1]));
      w[x].z = fmaf(w[x].z, lam, fmaf(w[x].z, lam_lo, kd * v[2]));
      w[x].w = fmaf(w[x].w, lam, fmaf(w[x].w, lam_lo, kd * v[3]));
      if (a.write_back && row >= 0) *reinterpret_cast<float4*>(S + static_cast<int64_t>(d) * D) = w[x];
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        const float qd = qs[d * GP + g];
        acc[g][0] = fmaf(qd, w[x].x, acc[g][0]);
        acc[g][1] = fmaf(qd, w[x].y, acc[g][1]);
        acc[g][2] = fmaf(qd, w[x].z, acc[g][2]);
        acc[g][3] = fmaf(qd, w[x].w, acc[g][3]);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < GP; ++g)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) acc[g][x] += __shfl_xor_sync(kFull, acc[g][x], o);
      if (lane < LPR) red[warp][g][lane * 4 + x] = acc[g][x];
    }
  __syncthreads();
  for (int e = t; e < a.G * W; e += kStepThreads) {
    const int g = e / W, x = e - g * W;
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kStepThreads / 32; ++w) o += red[w][g][x];
    o *= a.scale;
    const int64_t head = static_cast<int64_t>(u) * a.G + g;
    if (a.gate) o /= 1.f + expf(-bf16_to_f32(a.gate[head]));
    a.out[head * D + slice * W + x] = o;
  }
}

template <int D, int W>
cudaError_t step_launch(const LinearArgs& a, cudaStream_t s) {
  const dim3 grid(a.B * a.Hkv * (D / W));
  auto k = a.G <= 2 ? linear_step_kernel<D, W, 2> : (a.G <= 4 ? linear_step_kernel<D, W, 4> : linear_step_kernel<D, W, 8>);
  return launch_pdl(k, grid, dim3(kStepThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_linear_step(const LinearArgs& a, int D, int num_sms, cudaStream_t s) {
  // Few units: narrower slices as long as there is an SM for each (a slice's time
  // is its rows' round trips), with 32-byte rows at the least. Measured, in a
  // graph, slices of 32 / 16 / 8 columns: 2 units of 256 3.3 / 2.7 / 2.1 us, 8 of
  // 256 3.3 / 2.4 / 3.0 us, 16 of 128 2.2 / 1.7 / 2.1 us, 16 of 256 2.9 / 3.2 /
  // 4.8 us, 512 of 128 7.9 / 12.1 us.
  const int units = a.B * a.Hkv;
  const int W = units * (D / 8) <= num_sms ? 8 : units * (D / 16) <= num_sms ? 16 : 32;
  if (D == 128) return W == 8 ? step_launch<128, 8>(a, s) : W == 16 ? step_launch<128, 16>(a, s) : step_launch<128, 32>(a, s);
  return W == 8 ? step_launch<256, 8>(a, s) : W == 16 ? step_launch<256, 16>(a, s) : step_launch<256, 32>(a, s);
}

}  // namespace dattn
