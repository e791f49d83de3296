// Routing to the top k experts of the best groups (one wavefront per token).
//
// The gates are sigmoids or a softmax of the logits, scores are gates plus a
// bias, a group's score is the sum of its best one or two, and every decision
// is taken on fp64 scores with ties to the lower index, as in route.hip, so that
// the selected ids are reproducible bit for bit.
//
// Up to 1024 experts and 64 groups a token's logits stay in registers (lane l:
// experts l, l + 64, ...).  fp32 scores, whose error has a bound (err below), take
// the decisions that they are sure of: a few lanes per group find its best two
// through LDS; the groups are kept by the threshold that their keep-th largest
// score is, unless another lies within the error of it; the experts of the kept
// groups that come within the error of the k-th best lane's best, at most 64,
// are scored in fp64 and ranked by counting.  Without a bias a softmax's experts
// are compared by their logits, which fp32 holds exactly.
// What fp32 is not sure of goes the plain way: heavy ties, values that are no
// numbers, masked rows, and every token where the bias masks a group, whose score
// then sets the error that is allowed for (896 experts, one of 16 groups masked: 8
// tokens 30 us, 16384 158, with a softmax 185).  So do larger sizes (8 and 3584
// tokens of 2048 experts 31 and 76 us, of 4096 48 and 225, with a softmax 65 and 313;
// of 1024 by registers 6.6 and 12 to 16).  There the fp64 scores of a token lie in
// LDS ([E]) beside those of its groups ([groups]); experts of the groups that are not
// kept are marked with NaN (NaN scores themselves have become -inf by then), and
// top_of() takes the best, of groups as of experts.
// A softmax's sum is taken with the library's exponential there and for groups that
// are near each other, and with the fitted one for experts: to 2e-14 the same.
//
// 16384 tokens of 896 take 38 us, bound by the vector instructions (the logits
// are 59 MB, 12 us at 5.1 TB/s); 8 tokens 6.8 us, one wave's way through them.  A
// wave a token without a loop, 120 -> 78 us (the loop's spilled scalars); groups
// too near for fp32 settled by two experts' fp64 scores instead of the plain way,
// 78 -> 45; as many logits a lane as there are instead of 4, 8 or 16, 45 -> 39.
#include "route_device.h"

#include <type_traits>

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

// Value of the lane that step k (0 .. 5) of a reduction exchanges with.
template <int k>
__device__ __forceinline__ uint32_t partner(uint32_t v, int lane) {
  if constexpr (k == 0) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false);        // lane ^ 1
  else if constexpr (k == 1) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false);   // lane ^ 2
  else if constexpr (k == 2) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false);  // mirrored in its half row
  else if constexpr (k == 3) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false);  // mirrored in its row
  else return swap_rows<k == 4 ? 16 : 32>(v, lane);
}
template <int k>
__device__ __forceinline__ float partner(float v, int lane) { return __uint_as_float(partner<k>(__float_as_uint(v), lane)); }
template <int k>
__device__ __forceinline__ double partner(double v, int lane) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)partner<k>((uint32_t)(b >> 32), lane) << 32 | partner<k>((uint32_t)b, lane)));
}
// f(k) for the first log2(count) steps: lanes l / count apart stay apart (steps 2
// and 3 mirror, after which the lanes of 8 and of 16 agree all the same).
template <typename F>
__device__ __forceinline__ void steps(int count, F&& f) {
  if (count > 1) f(std::integral_constant<int, 0>{});
  if (count > 2) f(std::integral_constant<int, 1>{});
  if (count > 4) f(std::integral_constant<int, 2>{});
  if (count > 8) f(std::integral_constant<int, 3>{});
  if (count > 16) f(std::integral_constant<int, 4>{});
  if (count > 32) f(std::integral_constant<int, 5>{});
}

// ranks_before without a branch.
__device__ __forceinline__ bool before(double sa, int ea, double sb, int eb) {
  return ((int)(sa > sb) | ((int)(sa == sb) & (int)(ea < eb))) != 0;
}

// The entry of a[0 .. n-1] that ranks best among those strictly after (ps, pe);
// NaN entries are passed over.
__device__ __forceinline__ void best_after(const double* a, int n, int lane, double& ps, int& pe) {
  double bs = -INFINITY;
  int be = INT_MAX;  // sentinel: ranks after every real entry
  for (int i0 = lane; i0 < n; i0 += 4 * kWaveSize) {
    double v[4];  // (read together; past the end the last entry again)
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = a[min(i0 + u * kWaveSize, n - 1)];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = min(i0 + u * kWaveSize, n - 1);
      const bool take = ((int)before(ps, pe, v[u], i) & (int)before(v[u], i, bs, be)) != 0;
      bs = take ? v[u] : bs;
      be = take ? i : be;
    }
  }
  steps(kWaveSize, [&](auto k) {
    const double os = partner<decltype(k)::value>(bs, lane);
    const int oe = (int)partner<decltype(k)::value>((uint32_t)be, lane);
    const bool take = before(os, oe, bs, be);
    bs = take ? os : bs;
    be = take ? oe : be;
  });
  ps = bs;
  pe = be;
}

// The k entries of a[0 .. n-1] that rank best, NaN entries apart, the r-th in lane
// r (k <= 64, and at least k entries are numbers).  Of the 64 lanes' best entries the
// k-th ranks at or after every one of the top k, so these are among the entries
// that rank at or before it: mostly few more than k, which are compacted into `few`
// and sorted; with more than 64, k rounds of best_after.
struct Few {
  double s[kWaveSize];
  int e[kWaveSize];
};
__device__ __forceinline__ int top_of(const double* a, int n, int k, int lane, Few& few) {
  double bs = -INFINITY;
  int be = INT_MAX;  // sentinel: ranks after every real entry
  for (int i = lane; i < n; i += kWaveSize) {
    const double v = a[i];
    const bool take = before(v, i, bs, be);
    bs = take ? v : bs;
    be = take ? i : be;
  }
  if (n > kWaveSize) {
    wave_sort64(bs, be, lane);
    const double ts = readlane_f64(bs, k - 1);
    const int te = __builtin_amdgcn_readlane(be, k - 1);
    int total = 0;
    for (int i0 = 0; i0 < n; i0 += kWaveSize) {
      const int i = i0 + lane;
      const double v = i < n ? a[i] : NAN;
      const bool in = ((int)before(v, i, ts, te) | ((int)(v == ts) & (int)(i == te))) != 0;
      const uint64_t mask = __builtin_amdgcn_ballot_w64(in);
      const int slot = total + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
      if (in && slot < kWaveSize) {
        few.s[slot] = v;
        few.e[slot] = i;
      }
      total += __builtin_popcountll(mask);
    }
    wave_fence();
    if (total > kWaveSize) {
      double ps = INFINITY;
      int pe = -1, id = 0;
      for (int r = 0; r < k; ++r) {
        best_after(a, n, lane, ps, pe);
        if (lane == r) id = pe;
      }
      return id;
    }
    bs = lane < total ? few.s[lane] : -INFINITY;
    be = lane < total ? few.e[lane] : INT_MAX;
  }
  wave_sort64(bs, be, lane);
  return be;
}

// Best two of the two best (b1 >= b2) seen here and (o1 >= o2) elsewhere.
__device__ __forceinline__ void best_two(double& b1, double& b2, double o1, double o2) {
  b2 = fmax(fmin(b1, o1), fmax(b2, o2));
  b1 = fmax(b1, o1);
}

__device__ __forceinline__ void route_token(const GroupsArgs& a, int64_t t, int lane, Few& few, double* s) {
  double* const gs = s + a.E;
  const float* const zt = a.z + t * (int64_t)a.E;
  // Experts e, e + 64, .. of the lane two at a time (their loads and exponentials
  // overlap); past the end the last one again, not counted.
  auto experts = [&](auto&& f) {
    for (int e0 = lane; e0 < a.E; e0 += 2 * kWaveSize) {
      float z[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) z[u] = zt[min(e0 + u * kWaveSize, a.E - 1)];
      f(e0, z);
    }
  };
  SoftmaxStats st{0.0f, 1.0};
  if (a.softmax) {
    float m = -INFINITY;
    experts([&](int, const float (&z)[2]) { m = fmaxf(m, fmaxf(z[0], z[1])); });  // (passes over NaN)
    steps(kWaveSize, [&](auto k) { m = fmaxf(m, partner<decltype(k)::value>(m, lane)); });
    double sum = 0.0;
    experts([&](int e0, const float (&z)[2]) {
      double v[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) v[u] = softmax_weight(z[u], m);
#pragma unroll
      for (int u = 0; u < 2; ++u) sum += v[u] == v[u] && e0 + u * kWaveSize < a.E ? v[u] : 0.0;
    });
    steps(kWaveSize, [&](auto k) { sum += partner<decltype(k)::value>(sum, lane); });
    st = SoftmaxStats{m, sum > 0.0 ? sum : 1.0};
  }
  experts([&](int e0, const float (&z)[2]) {
    double v[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) v[u] = gate64(z[u], a.softmax, st) + (a.bias ? (double)a.bias[min(e0 + u * kWaveSize, a.E - 1)] : 0.0);
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (e0 + u * kWaveSize < a.E) s[e0 + u * kWaveSize] = v[u] == v[u] ? v[u] : -INFINITY;
  });
  wave_fence();

  if (a.keep < a.groups) {
    int shift = 0;  // 2^shift lanes per group, as many groups at a time as that leaves
    while (shift < 6 && (int64_t)a.groups << (shift + 1) <= kWaveSize) ++shift;
    for (int g0 = 0; g0 < a.groups; g0 += kWaveSize >> shift) {
      const int g = g0 + (lane >> shift);
      double b1 = -INFINITY, b2 = -INFINITY;
      if (g < a.groups)
        for (int i = lane & ((1 << shift) - 1); i < a.size; i += 1 << shift) best_two(b1, b2, s[g * a.size + i], -INFINITY);
      for (int d = 1; d < 1 << shift; d <<= 1) best_two(b1, b2, __shfl_xor(b1, d, kWaveSize), __shfl_xor(b2, d, kWaveSize));
      const double sum = a.group_top == 2 && a.size > 1 ? b1 + b2 : b1;
      if (g < a.groups && (lane & ((1 << shift) - 1)) == 0) gs[g] = sum == sum ? sum : -INFINITY;  // (infinities of both signs)
    }
    wave_fence();
    double ls = INFINITY;  // the last group kept
    int le = -1;           // (nothing ranks before (+inf, -1))
    if (a.keep <= kWaveSize) {
      le = __builtin_amdgcn_readlane(top_of(gs, a.groups, a.keep, lane, few), a.keep - 1);
      ls = gs[le];
    } else {
      for (int r = 0; r < a.keep; ++r) best_after(gs, a.groups, lane, ls, le);
    }
    for (int e = lane; e < a.E; e += kWaveSize) {
      const int g = e / a.size;
      if (ranks_before(ls, le, gs[g], g)) s[e] = NAN;  // after the last one kept
    }
    wave_fence();
  }

  const int id = top_of(s, a.E, a.k, lane, few);
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

// ---------------------------------------------------------------------------
// The register path.

// exp(d) for d <= 0 to 1.5e-14 of it, 0 below -762: 2^y, y = d log2(e) = n + f,
// n = rint(y), 2^f by a fitted polynomial (verify_draft.hip).  Coefficients come
// from scalar registers (fma_scalar there).
__device__ __forceinline__ double fma_scalar(double a, double b, double c) {
  double r;
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "s"(c));
  return r;
}
template <int n>
__device__ __forceinline__ void exp_down(const double (&d)[n], double (&w)[n]) {
  constexpr double kShift = 6755399441055744.0, kLog2E = 1.4426950408889634;
  constexpr double kP[10] = {1.0, 0.6931471805598851, 0.2402265069572282, 0.055504108668415666, 0.009618129181164007,
                             0.0013333557625477394, 0.00015403440884395527, 1.5252990012952022e-05, 1.3258335417356016e-06,
                             1.0148340949089715e-07};
  double f[n];
  int e[n];
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const double x = fmax(d[i], -1100.0 / kLog2E), t = fma(x, kLog2E, kShift);
    e[i] = (int)(uint32_t)(uint64_t)__double_as_longlong(t);
    f[i] = fma(x, kLog2E, kShift - t);
    w[i] = kP[9];
  }
#pragma unroll
  for (int k = 8; k >= 0; --k)
#pragma unroll
    for (int i = 0; i < n; ++i) w[i] = fma_scalar(w[i], f[i], kP[k]);
#pragma unroll
  for (int i = 0; i < n; ++i) w[i] = ldexp(w[i], e[i]);
}

// LDS of a wave: candidates' fp64 score, gate and expert, their logits and
// biases; the top k by rank; behind it the fp32 scores [E].
struct FastScratch {
  double fs[kWaveSize], tg[kWaveSize];
  int fe[kWaveSize], te[kWaveSize];
  float cz[kWaveSize], cb[kWaveSize];
};

// Routes token t from registers; false where fp32 is not sure.  A group has 2^shift
// lanes, 2^shift * groups <= 64; inv_size: ceil(2^20 / size), which
// divides every index below 1024 by size exactly.
template <int NPER>
__device__ __forceinline__ bool route_token_fast(const GroupsArgs& a, int64_t t, int lane, int shift, uint32_t inv_size, FastScratch& x, float* score) {
  const int lanes = 1 << shift;
  // whether expert lane + 64 j exists (NPER, in twos, is no larger than it has to be)
  auto real = [&](int j) -> bool { return j < NPER - 2 || lane < a.E - kWaveSize * j; };
  // (a buffer ends with the token's row: what lies past it costs no address arithmetic and reads as zeros)
  const uint32_t at = 4u * (uint32_t)lane, bytes = 4u * (uint32_t)a.E;
  const __amdgpu_buffer_rsrc_t zr = __builtin_amdgcn_make_buffer_rsrc((void*)(a.z + t * (int64_t)a.E), 0, (int)bytes, 0x00020000);
  float z[NPER], b[NPER];
#pragma unroll
  for (int j = 0; j < NPER; ++j) z[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(zr, at + 256u * j, 0, 0));
  if (a.bias) {
    const __amdgpu_buffer_rsrc_t br = __builtin_amdgcn_make_buffer_rsrc((void*)a.bias, 0, (int)bytes, 0x00020000);
#pragma unroll
    for (int j = 0; j < NPER; ++j) b[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(br, at + 256u * j, 0, 0));
  } else {
#pragma unroll
    for (int j = 0; j < NPER; ++j) b[j] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < NPER; ++j) z[j] = real(j) ? z[j] : -INFINITY;

  // fp32 scores s, of experts past E -inf, and what groups add up (gs).  u = 2^-24:
  //   sigmoid: off by at most 2^-21 (1 + |s|) (route_device.h).
  //   softmax: e^(z - m) from the rounded difference and the hardware exp2 is off by
  //   (2 |z - m| + 3) u of itself, so by 3 u absolutely; their sum, of at least 1, by
  //   (2 (ln E + 1) + 3 + NPER + 6) u < 2^-18 of itself (terms weigh |z - m| by at
  //   most ln E + 1 on the whole): a gate by less than 2^-17 of the largest gate,
  //   and the bias' addition by u |s|.
  float s[NPER], m = 0.0f, top = 1.0f;
  const bool by_logit = a.softmax && !a.bias;
  if (a.softmax) {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NPER; ++j) m = fmaxf(m, z[j]);  // (passes over NaN)
    steps(kWaveSize, [&](auto k) { m = fmaxf(m, partner<decltype(k)::value>(m, lane)); });
    if (!(fabsf(m) < INFINITY)) return false;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NPER; ++j) {
      s[j] = __builtin_amdgcn_exp2f((z[j] - m) * 1.44269504088896341f);
      sum += s[j];  // (past E: 0)
    }
    steps(kWaveSize, [&](auto k) { sum += partner<decltype(k)::value>(sum, lane); });
    if (!(sum < INFINITY)) return false;  // (NaN)
    if (!by_logit) {
      top = __builtin_amdgcn_rcpf(sum);
#pragma unroll
      for (int j = 0; j < NPER; ++j) s[j] = s[j] * top + b[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < NPER; ++j) s[j] = route_score32(z[j], b[j]);
  }
  const float rel = a.softmax ? 0x1p-22f : 0x1p-21f, base = (a.softmax ? 0x1p-16f : 0x1p-21f) * top;  // |error of s| <= base + rel |s|

  // The kept groups, a bit per group's first lane.
  uint64_t kept = ~0ull;
  const int n_kept = a.keep * a.size;
  if (a.keep < a.groups) {
#pragma unroll
    for (int j = 0; j < NPER; ++j)
      if (real(j)) score[lane + kWaveSize * j] = s[j];
    wave_fence();
    const int g = lane / lanes, sub = lane & (lanes - 1);
    float b1 = -INFINITY, b2 = -INFINITY;
    if (g < a.groups)
      for (int i = sub; i < a.size; i += lanes) {
        const float v = score[g * a.size + i];
        b2 = __builtin_amdgcn_fmed3f(b1, b2, v);  // (b2 <= b1: the middle one is the second best)
        b1 = fmaxf(b1, v);
      }
    steps(lanes, [&](auto k) {
      const float o1 = partner<decltype(k)::value>(b1, lane), o2 = partner<decltype(k)::value>(b2, lane);
      b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
      b1 = fmaxf(b1, o1);
    });
    const float gs = a.group_top == 2 && a.size > 1 ? b1 + b2 : b1;
    const bool first = sub == 0 && g < a.groups;
    const float thr = wave_kth_largest(first && gs == gs ? gs : -INFINITY, a.keep);
    if (!(fabsf(thr) < INFINITY)) return false;
    // Twice the error of a sum of two scores, each as large as any of the groups'
    // best two; by logit, of e^(z - m), off by less than (2 |z - m| + 4) u of itself
    // where it is not below 2^-100 (and anything below 1e-30 counts as near).
    float err, one;  // .. and of one score
    if (by_logit) {
      err = one = thr * 0x1p-21f * (2.0f + fabsf(__builtin_amdgcn_logf(thr))) + 1e-30f;
    } else {
      float largest = first ? fmaxf(fabsf(b1), a.size > 1 ? fabsf(b2) : 0.0f) : 0.0f;
      steps(kWaveSize, [&](auto k) { largest = fmaxf(largest, partner<decltype(k)::value>(largest, lane)); });
      one = 4.0f * (base + rel * largest);
      err = 4.0f * (2.0f * base + 3.0f * rel * largest);
    }
    kept = __builtin_amdgcn_ballot_w64(first && gs >= thr);
    const uint64_t near = __builtin_amdgcn_ballot_w64(first && !(gs < thr - err));  // (NaN: near)
    if (__builtin_popcountll(kept) != a.keep || near != kept) {
      // Groups too near to the threshold for fp32: their scores in fp64, from their
      // best two experts, if it is sure which these are.
      const uint64_t above = __builtin_amdgcn_ballot_w64(first && gs > thr + err);
      if (by_logit && !(thr > 1e-20f)) return false;
      float t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
      int i1 = 0, i2 = 0;
      if (first)
        for (int i = g * a.size; i < (g + 1) * a.size; ++i) {
          const float v = score[i];
          if (v > t1) {
            t3 = t2;
            t2 = t1;
            i2 = i1;
            t1 = v;
            i1 = i;
          } else if (v > t2) {
            t3 = t2;
            t2 = v;
            i2 = i;
          } else {
            t3 = fmaxf(t3, v);
          }
        }
      const bool two = a.group_top == 2 && a.size > 1;
      const bool mine = ((near & ~above) >> lane) & 1ull;
      const float last = two ? t2 : t1, next = two ? t3 : t2;
      if (__builtin_amdgcn_ballot_w64(mine && !(next < last - one)) != 0) return false;
      double all = 1.0;
      if (a.softmax && a.bias) {
        all = 0.0;
        for (int e = lane; e < a.E; e += kWaveSize) all += softmax_weight(a.z[t * (int64_t)a.E + e], m);
        steps(kWaveSize, [&](auto k) { all += partner<decltype(k)::value>(all, lane); });
      }
      auto exact = [&](int e) {
        const float ze = a.z[t * (int64_t)a.E + e];
        return (a.softmax ? softmax_weight(ze, m) / all : sigmoid64(ze)) + (a.bias ? (double)a.bias[e] : 0.0);
      };
      double gd = exact(i1);
      if (two) gd += exact(i2);
      int rank = __builtin_popcountll(above);  // among the near ones, behind those above
      for (uint64_t rest = near & ~above; rest != 0; rest &= rest - 1) {
        const int l = __builtin_ctzll(rest);
        rank += ranks_before(readlane_f64(gd, l), l, gd, lane) ? 1 : 0;
      }
      kept = above | __builtin_amdgcn_ballot_w64(mine && rank < a.keep);
      if (__builtin_popcountll(kept) != a.keep) return false;
    }
  }
  // Bit g: group g is kept.  Whether expert lane + 64 j belongs to one, without a branch.
  const uint64_t groups = a.keep < a.groups ? __builtin_amdgcn_ballot_w64(lane < a.groups && (kept >> ((lane << shift) & 63) & 1ull) != 0) : kept;
  const uint32_t place = __umul24((uint32_t)lane, inv_size);
  auto in_kept = [&](int j) -> bool {
    const uint32_t g = (place + (uint32_t)(kWaveSize * j) * inv_size) >> 20;
    return ((int)real(j) & (int)(groups >> (g & 63u))) != 0;
  };

  // Candidates: s[j] >= theta.
  float theta = 0.0f;
  uint64_t mask[NPER];
  int total = 0;
  if (n_kept <= kWaveSize) {
#pragma unroll
    for (int j = 0; j < NPER; ++j) s[j] = in_kept(j) ? 1.0f : -1.0f;
  } else {
    float best = -INFINITY;
#pragma unroll
    for (int j = 0; j < NPER; ++j) {
      const float v = by_logit ? fmaxf(z[j] - m, -700.0f) : s[j];
      s[j] = in_kept(j) ? v : -INFINITY;
      best = fmaxf(best, s[j]);
    }
    const float thr = wave_kth_largest(best, a.k);
    if (!(fabsf(thr) < INFINITY)) return false;
    theta = thr - (by_logit ? 0x1p-21f * (1.0f + fabsf(thr)) : 4.0f * (base + rel * (1.0f + fabsf(thr))));
  }
#pragma unroll
  for (int j = 0; j < NPER; ++j) {
    mask[j] = __builtin_amdgcn_ballot_w64(s[j] >= theta);
    total += __builtin_popcountll(mask[j]);
  }
  if (total > kWaveSize) return false;
  int slot = 0;
#pragma unroll
  for (int j = 0; j < NPER; ++j) {
    const int below = __builtin_amdgcn_mbcnt_hi((uint32_t)(mask[j] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask[j], 0u));
    if (s[j] >= theta) {
      x.fe[slot + below] = lane + kWaveSize * j;
      x.cz[slot + below] = z[j];
      x.cb[slot + below] = b[j];
    }
    slot += __builtin_popcountll(mask[j]);
  }
  wave_fence();

  // The sum of a softmax in fp64, where a gate itself enters a score or a weight.
  double sum = 1.0;
  if (a.softmax && (a.bias || !a.normalize)) {
    sum = 0.0;
    constexpr int kBatch = NPER % 4 == 0 ? 4 : NPER % 2 == 0 ? 2 : 1;
#pragma unroll
    for (int j = 0; j < NPER; j += kBatch) {
      double d[kBatch], w[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) d[i] = (double)z[j + i] - (double)m;
      exp_down<kBatch>(d, w);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) sum += w[i];  // (past E: 0)
    }
    steps(kWaveSize, [&](auto k) { sum += partner<decltype(k)::value>(sum, lane); });
  }
  double cs = -INFINITY, cg = 0.0;
  int ce = INT_MAX;
  if (lane < total) {
    ce = x.fe[lane];
    cg = a.softmax ? softmax_weight(x.cz[lane], m) / sum : sigmoid64(x.cz[lane]);
    cs = cg + (double)x.cb[lane];
    cs = cs == cs ? cs : -INFINITY;
  }
  x.fs[lane] = cs;
  x.fe[lane] = ce;
  x.tg[lane] = 0.0;
  wave_fence();
  // distinct experts, so distinct ranks: the top k are ranks 0 .. k-1 (all eight
  // entries read first, and the test without branches, so that the reads overlap)
  int rank = 0;
  for (int j0 = 0; j0 < total; j0 += 8) {
    double os[8];
    int oe[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      os[i] = x.fs[j0 + i];
      oe[i] = x.fe[j0 + i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) rank += (int)((os[i] > cs) | ((os[i] == cs) & (oe[i] < ce)));
  }
  if (lane < total && rank < a.k) {
    x.tg[rank] = cg;
    x.te[rank] = ce;
  }
  wave_fence();
  double weight_sum = 1.0;
  if (a.normalize) {  // in rank order (past the k-th the entries are 0, which leaves the sum as it is)
    weight_sum = 0.0;
    for (int r0 = 0; r0 < a.k; r0 += 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) weight_sum += x.tg[r0 + i];
    }
  }
  if (lane < a.k) {
    const double g = x.tg[lane];
    const double v = a.normalize ? (weight_sum == 0.0 ? 0.0 : g / weight_sum) : g;
    a.ids[t * a.k + lane] = x.te[lane];
    a.w[t * a.k + lane] = (float)(v * (double)a.route_scale);
  }
  return true;
}

template <int NPER>
__global__ __launch_bounds__(256) void route_groups_fast_kernel(GroupsArgs a, int shift, uint32_t inv_size, int lds_wave) {
  extern __shared__ double lds_scores[];
  const int lane = threadIdx.x & (kWaveSize - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
  double* const own = lds_scores + (size_t)wave * lds_wave;
  FastScratch& x = *reinterpret_cast<FastScratch*>(own);
  float* const score = reinterpret_cast<float*>(own + sizeof(FastScratch) / sizeof(double));
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 4 + wave;
  if (t >= a.T) return;  // (a wave's token; the kernel has no block-level barrier)
  if (!route_token_fast<NPER>(a, t, lane, shift, inv_size, x, score)) {
    wave_fence();
    route_token(a, t, lane, *reinterpret_cast<Few*>(own), own + sizeof(Few) / sizeof(double));
  }
}

// ---------------------------------------------------------------------------
// Any size.
__global__ __launch_bounds__(256) void route_groups_kernel(GroupsArgs a) {
  extern __shared__ double lds_scores[];
  const int lane = threadIdx.x & (kWaveSize - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
  double* const own = lds_scores + (size_t)wave * (sizeof(Few) / sizeof(double) + a.E + a.groups);
  const int waves = blockDim.x / kWaveSize;
  // (a wave's tokens; the kernel has no block-level barrier)
  for (int64_t t = (int64_t)blockIdx.x * waves + wave; t < a.T; t += (int64_t)gridDim.x * waves)
    route_token(a, t, lane, *reinterpret_cast<Few*>(own), own + sizeof(Few) / sizeof(double));
}

}  // namespace

hipError_t launch_route_groups(const RouteGroupsCall& c, hipStream_t s) {
  GroupsArgs a{c.z, c.bias, c.T, c.E, c.groups, c.E / c.groups, c.keep, c.group_top, c.k, c.softmax, c.normalize, c.route_scale, c.ids, c.w};
  const size_t per_wave = sizeof(Few) + (size_t)(c.E + c.groups) * sizeof(double);
  if (c.E <= 16 * kWaveSize && c.groups <= kWaveSize) {
    int shift = 6;
    while (c.groups << shift > kWaveSize) --shift;
    const uint32_t inv_size = ((1u << 20) + a.size - 1) / a.size;
    size_t fast = sizeof(FastScratch) + (size_t)(c.E + 1) / 2 * sizeof(double);
    fast = fast > per_wave ? fast : per_wave;
    const int64_t wgs = (c.T + 3) / 4, wide = wgs < (1 << 20) ? wgs : 1 << 20;  // (a grid dimension has fewer than 2^32 threads)
    const dim3 grid((unsigned)wide, (unsigned)((wgs + wide - 1) / wide));
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(4 * kWaveSize), 4 * fast, s, a, shift, inv_size, (int)(fast / sizeof(double))); };
    switch ((c.E + 2 * kWaveSize - 1) / (2 * kWaveSize)) {  // experts per lane, in twos
      case 1: c.E <= kWaveSize ? go(route_groups_fast_kernel<1>) : go(route_groups_fast_kernel<2>); break;
      case 2: go(route_groups_fast_kernel<4>); break;
      case 3: go(route_groups_fast_kernel<6>); break;
      case 4: go(route_groups_fast_kernel<8>); break;
      case 5: go(route_groups_fast_kernel<10>); break;
      case 6: go(route_groups_fast_kernel<12>); break;
      case 7: go(route_groups_fast_kernel<14>); break;
      default: go(route_groups_fast_kernel<16>); break;
    }
    return hipGetLastError();
  }
  constexpr size_t kLdsBudget = 64 * 1024;
  int waves = (int)(kLdsBudget / per_wave);
  waves = waves > 4 ? 4 : waves < 1 ? 1 : waves;
  int64_t blocks = (c.T + waves - 1) / waves;
  blocks = blocks < (1 << 20) ? blocks : 1 << 20;  // (a grid dimension has fewer than 2^32 threads)
  hipLaunchKernelGGL(route_groups_kernel, dim3((unsigned)blocks), dim3(waves * kWaveSize), per_wave * waves, s, a);
  return hipGetLastError();
}

}  // namespace k3moe
