// Sigmoid + bias top-k router (one 64-lane wavefront per token).
//
// Routing parameters from the llama.cpp pull request "model: add Kimi-K3 text
// model", converter dry-run comment: 896 experts, 16 used, sigmoid expert
// score gating, per-expert bias exp_probs_b.  Scores are evaluated in fp64 so
// that the selected ids are reproducible bit for bit; ties go to the lower
// expert index; NaN scores rank last.
//
// Up to 1024 experts (16 per lane) one wave handles a token with the logits
// in registers: lane l owns experts l, l + 64, l + 128, ....  An fp32 score
// pre-filters: the k-th of the 64 fp32 lane-bests (a bitwise radix select over
// ballots) bounds the k-th fp32 score from below, so every expert of the exact
// top k has an fp32 score no lower than that bound minus a small margin (the
// fp32 error bound is stated at route_score32); those candidates (at most 64)
// are scored in fp64 and each counts how many of the others rank before it,
// which places the top k in order without a sort.
// Otherwise (heavy ties, non-finite scores at the threshold) the fp64 scores of
// all experts are used: the 64 fp64 lane-bests are sorted, the experts ranking
// at or before the k-th of them are compacted and sorted, and with more than
// 64 of those each lane sorts its experts and k rounds take the wave's best
// head (DPP exchanges inside 16-lane rows, row swaps across rows).  Larger E
// falls back to a kernel that writes the scores to LDS (or recomputes them)
// and, in round r, picks the best expert ranking strictly after round r-1's
// pick; it needs no "taken" flags, so nothing limits E.
#include "route_device.h"

namespace k3moe {
namespace {

// Register-resident router: NPER experts per lane (E <= 64 * NPER), a wave per token.
template <int NPER>
__global__ __launch_bounds__(256) void route_topk_reg_kernel(const float* __restrict__ z, const float* __restrict__ bias,
                                                              int64_t T, int E, int k, int normalize, float route_scale,
                                                              int32_t* __restrict__ ids, float* __restrict__ w) {
  const int lane = threadIdx.x & (kWaveSize - 1);
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / kWaveSize) + threadIdx.x / kWaveSize;
  if (t >= T) return;  // whole wave leaves; the kernel has no block-level barrier
  __shared__ RouteScratch scratch[4];
  int id = 0;
  float g = 0.0f;
  route_token_reg<NPER>(z + t * (int64_t)E, bias, E, k, normalize, route_scale, lane, scratch[threadIdx.x / kWaveSize], id, g);
  if (lane < k) {
    ids[t * k + lane] = id;
    w[t * k + lane] = g;
  }
}

template <bool kScoresInLds>
__global__ __launch_bounds__(256) void route_topk_kernel(const float* __restrict__ z, const float* __restrict__ bias,
                                                          int64_t T, int E, int k, int normalize, float route_scale,
                                                          int32_t* __restrict__ ids, float* __restrict__ w) {
  extern __shared__ double lds_scores[];
  const int lane = threadIdx.x & (kWaveSize - 1);
  const int wave = threadIdx.x / kWaveSize;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / kWaveSize) + wave;
  if (t >= T) return;  // whole wave leaves; the kernel has no block-level barrier
  const float* zt = z + t * (int64_t)E;
  double* s = lds_scores + (size_t)wave * (kScoresInLds ? E : 0);

  if (kScoresInLds) {
    for (int e = lane; e < E; e += kWaveSize) s[e] = route_score(zt[e], bias ? bias[e] : 0.0f);
    // LDS accesses of one wave complete in order; the fence keeps the compiler
    // from moving the reads below above these writes.
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }

  double prev_s = INFINITY;
  int prev_e = -1;  // nothing ranks before (+inf, -1)
  int my_id = 0;
  for (int r = 0; r < k; ++r) {
    double best_s = -INFINITY;
    int best_e = INT_MAX;  // sentinel: ranks after every real expert
    for (int e = lane; e < E; e += kWaveSize) {
      const double se = kScoresInLds ? s[e] : route_score(zt[e], bias ? bias[e] : 0.0f);
      if (ranks_before(prev_s, prev_e, se, e) && ranks_before(se, e, best_s, best_e)) {
        best_s = se;
        best_e = e;
      }
    }
#pragma unroll
    for (int m = 1; m < kWaveSize; m <<= 1) {
      const double os = __shfl_xor(best_s, m, kWaveSize);
      const int oe = __shfl_xor(best_e, m, kWaveSize);
      if (ranks_before(os, oe, best_s, best_e)) {
        best_s = os;
        best_e = oe;
      }
    }
    if (lane == r) my_id = best_e;
    prev_s = best_s;
    prev_e = best_e;
  }

  // Gate weights: sigmoid(z) of the selected experts (lane r holds slot r).
  double g = 0.0;
  if (lane < k) g = sigmoid64(zt[my_id]);
  double sum = g;
  if (normalize) {
    // Sum in slot order 0..k-1 so the result does not depend on a tree shape.
    sum = 0.0;
    for (int r = 0; r < k; ++r) sum += readlane_f64(g, r);  // lane by lane
  }
  if (lane < k) {
    double v = normalize ? g / sum : g;
    v = v * (double)route_scale;
    ids[t * k + lane] = my_id;
    w[t * k + lane] = (float)v;
  }
}

}  // namespace

hipError_t launch_route_topk(const float* z, const float* bias, int64_t T, int E, int k, int normalize,
                             float route_scale, int32_t* ids, float* w, hipStream_t s) {
  if (E <= 16 * kWaveSize) {
    const int64_t blocks = (T + 3) / 4;
#define K3_ROUTE(NP)                                                                                            \
  hipLaunchKernelGGL(route_topk_reg_kernel<NP>, dim3((unsigned)blocks), dim3(256), 0, s, z, bias, T, E, k, \
                     normalize, route_scale, ids, w)
    if (E <= kWaveSize) K3_ROUTE(1);
    else if (E <= 2 * kWaveSize) K3_ROUTE(2);
    else if (E <= 4 * kWaveSize) K3_ROUTE(4);
    else if (E <= 8 * kWaveSize) K3_ROUTE(8);
    else K3_ROUTE(16);
#undef K3_ROUTE
    return hipGetLastError();
  }
  const size_t per_wave = (size_t)E * sizeof(double);
  constexpr size_t kLdsBudget = 64 * 1024;
  if (per_wave <= kLdsBudget) {
    int waves = (int)(kLdsBudget / per_wave);
    waves = waves > 4 ? 4 : waves;
    const int64_t blocks = (T + waves - 1) / waves;
    hipLaunchKernelGGL(route_topk_kernel<true>, dim3((unsigned)blocks), dim3(waves * kWaveSize), per_wave * waves, s,
                       z, bias, T, E, k, normalize, route_scale, ids, w);
  } else {
    const int64_t blocks = (T + 3) / 4;
    hipLaunchKernelGGL(route_topk_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, s, z, bias, T, E, k,
                       normalize, route_scale, ids, w);
  }
  return hipGetLastError();
}

}  // namespace k3moe
