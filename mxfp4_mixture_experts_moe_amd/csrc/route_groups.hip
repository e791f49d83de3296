// Routing to the top k experts of the best groups (one wavefront per token).
//
// The gates are sigmoids or a softmax of the logits, scores are gates plus a
// bias, a group's score is the sum of its best one or two, and every decision
// is taken on fp64 scores with ties to the lower index, as in route.hip, so that
// the selected ids are reproducible bit for bit.
//
// The scores of a token lie in LDS ([E] fp64) beside those of its groups
// ([groups]).  The lanes take the groups in turn; the last of the kept groups is
// found by `keep` rounds of the best group that ranks strictly after the one
// before, which needs no flags; experts of the other groups are marked with NaN
// (NaN scores themselves have become -inf by then), and k such rounds take the
// experts.
#include "route_device.h"

namespace k3moe {
namespace {

struct GroupsArgs {
  const float *z, *bias;
  int64_t T;
  int E, groups, size, keep, group_top, k;
  int softmax, normalize;
  float route_scale;
  int32_t* ids;
  float* w;
};

// What the wave wrote to LDS is there for its own reads below (a wave's LDS
// accesses complete in order; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Softmax of a token: largest logit and fp64 sum of exponentials.  NaN logits
// are left out.
struct SoftmaxStats {
  float m;
  double sum;  // 1 where there is nothing to share
};
__device__ __forceinline__ double softmax_weight(float z, float m) {
  if (!(z > -INFINITY)) return z != z ? (double)z : 0.0;  // NaN stays NaN
  if (z == m) return 1.0;                                 // (an infinite m: shared by those that reach it)
  return m == INFINITY ? 0.0 : exp((double)z - (double)m);
}
__device__ __forceinline__ double gate64(float z, int softmax, const SoftmaxStats& st) {
  return softmax ? softmax_weight(z, st.m) / st.sum : sigmoid64(z);
}

// Best (s, e) of the wave, in every lane.
__device__ __forceinline__ void best_of_wave(double& s, int& e) {
#pragma unroll
  for (int m = 1; m < kWaveSize; m <<= 1) {
    const double os = __shfl_xor(s, m, kWaveSize);
    const int oe = __shfl_xor(e, m, kWaveSize);
    if (ranks_before(os, oe, s, e)) {
      s = os;
      e = oe;
    }
  }
}

// The entry of a[0 .. n-1] that ranks best among those strictly after (ps, pe);
// NaN entries are passed over.
__device__ __forceinline__ void best_after(const double* a, int n, int lane, double& ps, int& pe) {
  double bs = -INFINITY;
  int be = INT_MAX;  // sentinel: ranks after every real entry
  for (int i = lane; i < n; i += kWaveSize) {
    const double v = a[i];
    if (ranks_before(ps, pe, v, i) && ranks_before(v, i, bs, be)) {
      bs = v;
      be = i;
    }
  }
  best_of_wave(bs, be);
  ps = bs;
  pe = be;
}

__device__ __forceinline__ void route_token(const GroupsArgs& a, int64_t t, int lane, double* s, double* gs) {
  const float* const zt = a.z + t * (int64_t)a.E;
  SoftmaxStats st{0.0f, 1.0};
  if (a.softmax) {
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += kWaveSize) m = fmaxf(m, zt[e]);  // (passes over NaN)
#pragma unroll
    for (int d = 1; d < kWaveSize; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, kWaveSize));
    double sum = 0.0;
    for (int e = lane; e < a.E; e += kWaveSize) {
      const double v = softmax_weight(zt[e], m);
      sum += v == v ? v : 0.0;
    }
#pragma unroll
    for (int d = 1; d < kWaveSize; d <<= 1) sum += __shfl_xor(sum, d, kWaveSize);
    st = SoftmaxStats{m, sum > 0.0 ? sum : 1.0};
  }
  for (int e = lane; e < a.E; e += kWaveSize) {
    const double v = gate64(zt[e], a.softmax, st) + (a.bias ? (double)a.bias[e] : 0.0);
    s[e] = v == v ? v : -INFINITY;
  }
  wave_fence();

  if (a.keep < a.groups) {
    for (int g = lane; g < a.groups; g += kWaveSize) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < a.size; ++i) {
        const double v = s[g * a.size + i];
        b2 = v > b1 ? b1 : fmax(b2, v);
        b1 = fmax(b1, v);
      }
      const double sum = a.group_top == 2 && a.size > 1 ? b1 + b2 : b1;
      gs[g] = sum == sum ? sum : -INFINITY;  // (infinities of both signs)
    }
    wave_fence();
    double ls = INFINITY;
    int le = -1;  // nothing ranks before (+inf, -1)
    for (int r = 0; r < a.keep; ++r) best_after(gs, a.groups, lane, ls, le);
    for (int g = lane; g < a.groups; g += kWaveSize)
      if (ranks_before(ls, le, gs[g], g))  // after the last one kept
        for (int i = 0; i < a.size; ++i) s[g * a.size + i] = NAN;
    wave_fence();
  }

  double ps = INFINITY;
  int pe = -1, id = 0;
  for (int r = 0; r < a.k; ++r) {
    best_after(s, a.E, lane, ps, pe);
    if (lane == r) id = pe;
  }
  double g = 0.0;
  if (lane < a.k) g = gate64(zt[id], a.softmax, st);
  double sum = 1.0;
  if (a.normalize) {
    // in slot order 0 .. k-1, as moe_route_topk adds them
    sum = 0.0;
    for (int r = 0; r < a.k; ++r) sum += readlane_f64(g, r);
  }
  wave_fence();  // the scores are read before the next token's are written
  if (lane < a.k) {
    double v = a.normalize ? (sum == 0.0 ? 0.0 : g / sum) : g;
    v = v * (double)a.route_scale;
    a.ids[t * a.k + lane] = id;
    a.w[t * a.k + lane] = (float)v;
  }
}

__global__ __launch_bounds__(256) void route_groups_kernel(GroupsArgs a) {
  extern __shared__ double lds_scores[];
  const int lane = threadIdx.x & (kWaveSize - 1);
  const int wave = threadIdx.x / kWaveSize;
  double* const s = lds_scores + (size_t)wave * (a.E + a.groups);
  double* const gs = s + a.E;
  const int waves = blockDim.x / kWaveSize;
  // (a wave's tokens; the kernel has no block-level barrier)
  for (int64_t t = (int64_t)blockIdx.x * waves + wave; t < a.T; t += (int64_t)gridDim.x * waves)
    route_token(a, t, lane, s, gs);
}

}  // namespace

hipError_t launch_route_groups(const RouteGroupsCall& c, hipStream_t s) {
  GroupsArgs a{c.z, c.bias, c.T, c.E, c.groups, c.E / c.groups, c.keep, c.group_top, c.k, c.softmax, c.normalize, c.route_scale, c.ids, c.w};
  const size_t per_wave = (size_t)(c.E + c.groups) * sizeof(double);
  constexpr size_t kLdsBudget = 64 * 1024;
  int waves = (int)(kLdsBudget / per_wave);
  waves = waves > 4 ? 4 : waves < 1 ? 1 : waves;
  int64_t blocks = (c.T + waves - 1) / waves;
  blocks = blocks < (1 << 20) ? blocks : 1 << 20;  // (a grid dimension has fewer than 2^32 threads)
  hipLaunchKernelGGL(route_groups_kernel, dim3((unsigned)blocks), dim3(waves * kWaveSize), per_wave * waves, s, a);
  return hipGetLastError();
}

}  // namespace k3moe
