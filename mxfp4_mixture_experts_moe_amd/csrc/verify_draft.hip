// Verification of drafted tokens against the target's distribution.
//
// Row w of a sequence gives p = softmax(logits / T); proposal x of position w is
// accepted where u q(x) < p(x), and the next token comes from max(p - q, 0) at
// the first one that is not, or from p itself, by its cumulative sum in index
// order.  A sum over the vocabulary decides between neighbours that hold 1e-6 of
// it, so an fp32 sum's order would move the token; everything here is fp64
// from the logits on, and two runs (or another order of summation) differ only
// where a uniform lies within about 1e-14 of a border.
//
// Two launches, over chunks of 4096 vocabulary entries:
//   stats   every row's chunks: largest logit, its lowest index (greedy), sum of
//           exponentials relative to the chunk's own largest;
//   choose  out of the chunks' sums the rows', which proposals are accepted, and
//           the next token: the chunk that holds it by a scan of the chunks'
//           shares, then the entry by a scan of the chunk.  The shares of p are the
//           first launch's sums, so without draft distributions one workgroup per
//           sequence does (the proposal's own chunk is summed again without it);
//           with them a workgroup per chunk sums its share of max(p - q, 0), after
//           deciding the acceptances for itself (a few KB from the L2), and the one
//           that finishes last goes on to the token.  "Last" is a counter per
//           sequence that the first launch clears; nothing waits.
//
// The first launch is bound by the logits' bytes beside the fp64 polynomials: 256
// rows of 163840 f32 38 to 42 us, 4.0 to 4.4 TB/s (about 24 us of it are the polynomials alone);
// the second by a chain of loads, sums and barriers: 32 sequences 15 to 19 us, of
// which 8 are the bytes of a row and its q; one sequence without q 7.
#include "k3moe_internal.h"

#include <math.h>

#include <type_traits>

namespace k3moe {
namespace {

// Threads of a workgroup: of the first launch, and of the second, whose waves
// take a row's sums each.
constexpr int kThreads = 256, kChooseThreads = 512;

struct ChunkStat {
  float m;     // largest logit, -inf: none
  int32_t at;  // its lowest index (greedy rows only)
  double z;    // sum of exp((l - m) / T)
};

struct VerifyArgs {
  const uint8_t* logits;
  const int32_t* draft;
  const float* q;
  const int32_t* len;
  const float* temperature;
  const float *u_accept, *u_sample;
  int64_t S;
  int W, V, chunks;
  ChunkStat* stats;  // [S * W][chunks]
  double* mass;      // [S][chunks]
  uint32_t* done;    // [S]
  int32_t *accepted, *tokens;
  float* accept_prob;
};

template <int kType>
constexpr int kSize = kType == K3MOE_DTYPE_F32 ? 4 : 2;
template <int kType>
constexpr int kVec = 16 / kSize<kType>;  // logits of a 16-byte load

template <int kType>
__device__ __forceinline__ float logit(const uint8_t* row, int64_t i) {
  if constexpr (kType == K3MOE_DTYPE_F32) {
    return reinterpret_cast<const float*>(row)[i];
  } else if constexpr (kType == K3MOE_DTYPE_BF16) {
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
  } else {
    return (float)reinterpret_cast<const _Float16*>(row)[i];
  }
}
// Logits v .. v + kVec - 1 of a row of V (rows start at any multiple of the
// type's size); -inf past its end.  whole: none of the caller's lie past it.
template <int kType>
__device__ __forceinline__ void logits16(const uint8_t* row, int v, int V, bool whole, float* l) {
  constexpr int n = kVec<kType>;
  if (whole) {
    uint32_t d[4];
    __builtin_memcpy(d, row + (int64_t)v * kSize<kType>, 16);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      if constexpr (kType == K3MOE_DTYPE_F32) {
        l[i] = __uint_as_float(d[i]);
      } else if constexpr (kType == K3MOE_DTYPE_BF16) {
        l[i] = __uint_as_float(i & 1 ? d[i / 2] & 0xFFFF0000u : d[i / 2] << 16);
      } else {
        const uint16_t h = (uint16_t)(i & 1 ? d[i / 2] >> 16 : d[i / 2]);
        l[i] = (float)__builtin_bit_cast(_Float16, h);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) l[i] = v + i < V ? logit<kType>(row, v + i) : -INFINITY;
  }
}

// a * b + c with c from scalar registers.  (The compiler would copy every
// coefficient of a series to vector registers first, for the two-operand form:
// as many moves again.)
__device__ __forceinline__ double fma_scalar(double a, double b, double c) {
  double r;
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "s"(c));
  return r;
}

// exp((l - m) / T) for logits l <= m of a row or chunk whose largest is m: 0 for
// NaN and -inf.  As 2^y with y = (l - m) log2(e) / T = n + f, n = rint(y): 2^f on
// |f| <= 1/2 by a polynomial fitted to it (1 at f = 0; largest relative error
// 1.5e-14, near-minimax, by reweighted least squares on Chebyshev nodes).
struct Scale {
  double m, c, least;  // c: log2(e) / T; least: l - m is taken no lower (its weight is 0 there)
  bool infinite;       // m is +inf (shared by the logits that reach it) or -inf (no logit is above it)
};
// What a temperature gives: log2(e) / T and the lowest difference of logits.
struct Heat {
  double c, least;
};
__device__ __forceinline__ Heat heat_of(const float* temperature, int64_t s) {
  constexpr double kLog2E = 1.4426950408889634;
  if (!temperature) return Heat{kLog2E, -1100.0 / kLog2E};
  const double t = (double)temperature[s];
  // (T = inf: all finite logits weigh 1, and -inf still nothing)
  return Heat{fmax(kLog2E / t, 1e-300), fmax(-1100.0 / kLog2E * t, -1.7e308)};
}
__device__ __forceinline__ Scale scale_of(float m, const Heat& h) { return Scale{(double)m, h.c, h.least, fabsf(m) == INFINITY}; }
// ... for an m that is the same in the whole wave.
__device__ __forceinline__ Scale scale_of_wave(float m, const Heat& h) {
  return scale_of(__uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(m))), h);
}
// The weights of n logits; one coefficient after the other for all of them, which
// keeps it in its registers.
template <int n>
__device__ __forceinline__ void weights(const float* l, const Scale& s, double* w) {
  if (s.infinite) {
#pragma unroll
    for (int i = 0; i < n; ++i) w[i] = l[i] == INFINITY ? 1.0 : 0.0;
    return;
  }
  constexpr double kShift = 6755399441055744.0;  // 1.5 * 2^52: an integer's bits end up in the lowest of the sum
  constexpr double kP[10] = {1.0, 0.6931471805598851, 0.2402265069572282, 0.055504108668415666, 0.009618129181164007,
                             0.0013333557625477394, 0.00015403440884395527, 1.5252990012952022e-05, 1.3258335417356016e-06,
                             1.0148340949089715e-07};
  double f[n];
  int e[n];
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const double d = fmax((double)l[i] - s.m, s.least);  // (the difference first: a low temperature makes much of its last bits; NaN: least)
    const double t = fma(d, s.c, kShift);
    e[i] = (int)(uint32_t)(uint64_t)__double_as_longlong(t);
    f[i] = fma(d, s.c, kShift - t);
    w[i] = kP[9];
  }
#pragma unroll
  for (int k = 8; k >= 0; --k)
#pragma unroll
    for (int i = 0; i < n; ++i) w[i] = fma_scalar(w[i], f[i], kP[k]);
#pragma unroll
  for (int i = 0; i < n; ++i) w[i] = ldexp(w[i], e[i]);
}
__device__ __forceinline__ double weight(float l, const Scale& s) {
  double w;
  weights<1>(&l, s, &w);
  return w;
}

// Reductions over a wave, the result in every lane: exchanges inside rows of 16
// lanes by DPP, then with the other rows (the gfx950 row swaps), no LDS trips.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kCtrl, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t other_row(uint32_t v, int lane, bool far) {
  const auto r = far ? __builtin_amdgcn_permlane32_swap(v, v, false, false) : __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return (lane & (far ? 32 : 16)) ? r[0] : r[1];
}
template <int kStep>
__device__ __forceinline__ uint32_t partner(uint32_t v, int lane) {
  if constexpr (kStep == 0) return dpp<0xB1>(v);        // lane ^ 1
  else if constexpr (kStep == 1) return dpp<0x4E>(v);   // lane ^ 2
  else if constexpr (kStep == 2) return dpp<0x141>(v);  // mirrored in its half row
  else if constexpr (kStep == 3) return dpp<0x140>(v);  // mirrored in its row
  else return other_row(v, lane, kStep == 5);
}
template <int kStep>
__device__ __forceinline__ double partner(double v, int lane) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)partner<kStep>((uint32_t)(b >> 32), lane) << 32 | partner<kStep>((uint32_t)b, lane)));
}
template <typename F>
__device__ __forceinline__ void six_steps(F&& f) {
  f(std::integral_constant<int, 0>{});
  f(std::integral_constant<int, 1>{});
  f(std::integral_constant<int, 2>{});
  f(std::integral_constant<int, 3>{});
  f(std::integral_constant<int, 4>{});
  f(std::integral_constant<int, 5>{});
}
__device__ __forceinline__ float wave_max(float v, int lane) {
  six_steps([&](auto k) { v = fmaxf(v, __uint_as_float(partner<decltype(k)::value>(__float_as_uint(v), lane))); });
  return v;
}
__device__ __forceinline__ double wave_sum(double v, int lane) {
  six_steps([&](auto k) { v += partner<decltype(k)::value>(v, lane); });
  return v;
}
__device__ __forceinline__ int wave_min(int v, int lane) {
  six_steps([&](auto k) { v = min(v, (int)partner<decltype(k)::value>((uint32_t)v, lane)); });
  return v;
}
// Value of another lane by DPP, 0 where there is none.
template <int kCtrl, int kRows>
__device__ __forceinline__ double moved(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, kCtrl, kRows, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), kCtrl, kRows, 0xF, false);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
// Sum over the lanes up to this one: inside rows of 16, then the rows before.
__device__ __forceinline__ double wave_scan(double v) {
  v += moved<0x111, 0xF>(v);  // lane - 1 of the row
  v += moved<0x112, 0xF>(v);
  v += moved<0x114, 0xF>(v);
  v += moved<0x118, 0xF>(v);
  v += moved<0x142, 0xA>(v);  // the last lane of the row before, in rows 1 and 3
  v += moved<0x143, 0xC>(v);  // lane 31, in rows 2 and 3
  return v;
}
__device__ __forceinline__ double lane_before(double v) { return moved<0x138, 0xF>(v); }
__device__ __forceinline__ double last_lane(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63)));
}

__device__ __forceinline__ bool greedy_of(const VerifyArgs& a, int64_t s) { return a.temperature && !(a.temperature[s] > 0.0f); }

template <int kType>
__global__ __launch_bounds__(kThreads) void stats_kernel(VerifyArgs a) {
  constexpr int kWaves = kThreads / 64, kEach = kVocabChunk / kThreads;
  __shared__ ChunkStat part[kWaves];
  const int64_t r = blockIdx.x / (unsigned)a.chunks;
  const int c = (int)(blockIdx.x - r * a.chunks);
  const int64_t s = r / a.W;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (c == 0 && r == s * a.W && threadIdx.x == 0) a.done[s] = 0u;
  const uint8_t* const row = a.logits + r * a.V * kSize<kType>;
  constexpr int n = kVec<kType>;
  const int v0 = c * kVocabChunk + (int)threadIdx.x * n;
  const bool whole = (c + 1) * kVocabChunk <= a.V;
  float l[kEach];
#pragma unroll
  for (int i = 0; i < kEach; i += n) logits16<kType>(row, v0 + i * kThreads, a.V, whole, l + i);
  const bool greedy = greedy_of(a, s);
  const Heat heat = heat_of(a.temperature, s);
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kEach; ++i) m = fmaxf(m, l[i]);  // (passes over NaN)
  m = wave_max(m, lane);
  double z = 0.0;
  int at = INT_MAX;
  if (greedy) {
#pragma unroll
    for (int i = kEach - 1; i >= 0; --i)
      if (l[i] == m && m > -INFINITY) at = v0 + i / n * n * kThreads + i % n;
    at = wave_min(at, lane);
  } else {
    const Scale sc = scale_of_wave(m, heat);
#pragma unroll
    for (int i = 0; i < kEach; i += 4) {
      double w[4];
      weights<4>(l + i, sc, w);
      z += (w[0] + w[1]) + (w[2] + w[3]);
    }
    z = wave_sum(z, lane);
  }
  if (lane == 0) part[wave] = ChunkStat{m, at, z};
  __syncthreads();
  if (threadIdx.x < 64) {  // the waves' together, each at its own largest so far
    const ChunkStat x = part[lane < kWaves ? lane : 0];
    m = wave_max(x.m, lane);
    z = lane < kWaves && !greedy ? x.z * weight(x.m, scale_of_wave(m, heat)) : 0.0;
    at = greedy && x.m == m ? x.at : INT_MAX;
    z += partner<0>(z, lane);
    z += partner<1>(z, lane);  // (the four waves')
    at = wave_min(at, lane);
    if (lane == 0) a.stats[r * a.chunks + c] = ChunkStat{m, at, z};
  }
}

// A row's largest logit, its lowest index and its sum, out of the chunks'; by one wave, in every lane.
struct RowStat {
  float m;
  int at;
  double z;
};
__device__ __forceinline__ RowStat row_stat(const ChunkStat* st, int chunks, int lane, const Heat& heat, bool greedy) {
  const ChunkStat own = lane < chunks ? st[lane] : ChunkStat{-INFINITY, INT_MAX, 0.0};
  float m = own.m;
  for (int c = lane + 64; c < chunks; c += 64) m = fmaxf(m, st[c].m);
  m = wave_max(m, lane);
  const Scale sc = scale_of_wave(m, heat);
  auto take = [&](const ChunkStat& x) { return greedy ? 0.0 : x.z * weight(x.m, sc); };
  double z = take(own);
  int at = greedy && own.m == m ? own.at : INT_MAX;
  for (int c = lane + 64; c < chunks; c += 64) {
    const ChunkStat x = st[c];
    z += take(x);
    if (greedy && x.m == m) at = min(at, x.at);
  }
  return RowStat{m, greedy ? wave_min(at, lane) : INT_MAX, greedy ? 0.0 : wave_sum(z, lane)};
}

// What is sampled from, entry v of a row: max(p - q, 0) or p.
struct Source {
  Scale sc;
  double inv_z;
  const float* q;  // null: q is 1 at x
  int x;           // the proposal, -1: none
  bool residual;
};
// Entries v .. v + kVec - 1 (0 past the row's end).
template <int kType>
__device__ __forceinline__ void entries16(const Source& d, const uint8_t* row, int v, int V, bool whole, double* e) {
  constexpr int n = kVec<kType>;
  float l[n], q[n];
  logits16<kType>(row, v, V, whole, l);
  if (d.residual && d.q) {
#pragma unroll
    for (int i = 0; i < n; i += 4) logits16<K3MOE_DTYPE_F32>(reinterpret_cast<const uint8_t*>(d.q), v + i, V, whole, q + i);
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) q[i] = d.residual && v + i == d.x ? 1.0f : 0.0f;
  }
  weights<n>(l, d.sc, e);
#pragma unroll
  for (int i = 0; i < n; ++i) {
    e[i] *= d.inv_z;
    if (d.residual) e[i] = fmax(e[i] - (double)q[i], 0.0);
    if (!whole && v + i >= V) e[i] = 0.0;
  }
}
// This thread's part of a chunk's share.
template <int kType>
__device__ __forceinline__ double chunk_part(const Source& d, const uint8_t* row, int c, int V) {
  constexpr int n = kVec<kType>, kEach = kVocabChunk / kChooseThreads;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < kEach; i += n) {
    double e[n];
    entries16<kType>(d, row, c * kVocabChunk + (i * kChooseThreads + (int)threadIdx.x * n), V, (c + 1) * kVocabChunk <= V, e);
#pragma unroll
    for (int j = 0; j < n; ++j) sum += e[j];
  }
  return sum;
}
// The sum over the workgroup, in thread 0.
constexpr int kChooseWaves = kChooseThreads / 64;
__device__ __forceinline__ double block_sum(double v, double (&part)[kChooseWaves]) {
  v = wave_sum(v, threadIdx.x & 63);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < kChooseWaves; ++i) v += part[i];
  return v;
}

// kPer: chunks of a workgroup (0: without draft distributions, one workgroup per sequence).
template <int kType, int kPer>
__global__ __launch_bounds__(kChooseThreads) void choose_kernel(VerifyArgs a) {
  constexpr bool kProbs = kPer > 0;
  constexpr int kWaves = kChooseWaves, kEach = kVocabChunk / kChooseThreads;
  __shared__ RowStat rows[kMaxVerifyWidth];
  __shared__ double part[kWaves], own_mass, sh_target, sh_before;
  __shared__ int sh_count, sh_last, sh_found, sh_residual, wat[kWaves], wlast[kWaves];
  const unsigned wgs = kProbs ? (unsigned)(a.chunks + kPer - 1) / (unsigned)(kProbs ? kPer : 1) : 1u;  // of a sequence
  const unsigned id = blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t s = id / wgs;
  if (s >= a.S) return;
  const int c = (int)(id - s * wgs);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int W = a.W, V = a.V, D = W - 1;
  const bool greedy = greedy_of(a, s);
  const Heat heat = heat_of(a.temperature, s);
  // the proposals, one lane each: what their test reads, asked for ahead of the sums
  int x = -1;
  float xl = -INFINITY, xq = 1.0f, xu = 0.0f;
  if (wave == 0 && lane < D) {
    x = a.draft[s * D + lane];
    xu = a.u_accept[s * D + lane];
    if (x >= 0 && x < V) {
      xl = logit<kType>(a.logits + (s * W + lane) * V * kSize<kType>, x);
      if constexpr (kProbs) xq = a.q[(s * D + lane) * V + x];
    }
  }
  int n = a.len ? a.len[s] : D;
  n = n < 0 ? 0 : n > D ? D : n;
  for (int w = wave; w < W; w += kWaves) {
    const RowStat st = row_stat(a.stats + (s * W + w) * a.chunks, a.chunks, lane, heat, greedy);
    if (lane == 0) rows[w] = st;
  }
  __syncthreads();
  if (wave == 0) {
    bool take = false;
    double chance = 0.0;
    if (lane < n && x >= 0 && x < V) {
      const RowStat st = rows[lane];
      if (greedy) {
        take = x == st.at;
        chance = take ? 1.0 : 0.0;
      } else if (st.z > 0.0) {
        const double p = weight(xl, scale_of(st.m, heat)) / st.z, q = (double)xq;
        take = (double)xu * q < p;
        chance = q < p ? 1.0 : q > 0.0 ? p / q : 0.0;
      }
    }
    const uint64_t no = ~__builtin_amdgcn_ballot_w64(take);
    const int count = no ? __builtin_ctzll(no) : 64;  // (D <= 63)
    if (lane == 0) sh_count = count;
    if (c == 0) {
      if (lane < D && a.accept_prob) a.accept_prob[s * D + lane] = (float)chance;
      if (lane == 0) a.accepted[s] = count;
      if (lane < W && lane != count) a.tokens[s * W + lane] = lane < count ? x : -1;
    }
  }
  __syncthreads();
  const int count = sh_count;
  const RowStat st = rows[count];
  int32_t* const token = a.tokens + s * W + count;
  if (greedy) {
    if (c == 0 && threadIdx.x == 0) *token = st.at == INT_MAX ? -1 : st.at;
    return;
  }

  const uint8_t* const row = a.logits + (s * W + count) * V * kSize<kType>;
  Source d{scale_of_wave(st.m, heat), st.z > 0.0 ? 1.0 / st.z : 0.0, nullptr, -1, count < n};
  if (d.residual) {
    d.x = a.draft[s * D + count];
    if constexpr (kProbs) d.q = a.q + (s * D + count) * V;
  }
  const bool inside = d.x >= 0 && d.x < V;
  const int own = !kProbs && d.residual && inside ? d.x / kVocabChunk : -1;  // the chunk whose share of max(p - q, 0) is not that of p
  if constexpr (kProbs) {
    if (d.residual) {  // (else p's shares are there)
      __shared__ double sums[kProbs ? kPer : 1][kWaves];
      double own_sum[kProbs ? kPer : 1];
#pragma unroll
      for (int i = 0; i < kPer; ++i) own_sum[i] = c * kPer + i < a.chunks ? chunk_part<kType>(d, row, c * kPer + i, V) : 0.0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        own_sum[i] = wave_sum(own_sum[i], lane);
        if (lane == 0) sums[i][wave] = own_sum[i];
      }
      __syncthreads();
      if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          double mass = 0.0;
          for (int w = 0; w < kWaves; ++w) mass += sums[i][w];
          if (c * kPer + i < a.chunks) __hip_atomic_store(a.mass + s * a.chunks + c * kPer + i, mass, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        // The shares are written through to where the last workgroup's device-scope
        // loads find them before the count says so.  (Release and acquire would write
        // back and invalidate a whole L2 for every workgroup: 42 us instead of 20 for
        // 32 rows of 163840.)
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        sh_last = __hip_atomic_fetch_add(a.done + s, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == wgs - 1u;
      }
      __syncthreads();
      if (!sh_last) return;
    } else if (c != 0) {
      return;
    }
  } else if (own >= 0) {
    const double mass = block_sum(chunk_part<kType>(d, row, own, V), part);
    if (threadIdx.x == 0) own_mass = mass;
  }
  __syncthreads();

  // The chunk: the first whose cumulative sum exceeds the target; past the end (a
  // uniform of 1), the last that holds anything.
  if (wave == 0) {
    const double u = (double)a.u_sample[s];
    const ChunkStat* const cs = a.stats + (s * W + count) * a.chunks;
    bool residual = d.residual;
    auto share = [&](int i) -> double {
      if (i >= a.chunks) return 0.0;
      if (kProbs && residual) return __hip_atomic_load(a.mass + s * a.chunks + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (residual && i == own) return own_mass;
      return cs[i].z * weight(cs[i].m, d.sc) * d.inv_z;
    };
    double total, v, incl;  // (v, incl: the first 64 chunks', of which most rows have no more)
    for (;;) {
      v = share(lane);
      incl = wave_scan(v);
      total = last_lane(incl);
      for (int i0 = 64; i0 < a.chunks; i0 += 64) total += last_lane(wave_scan(share(i0 + lane)));
      if (!residual || total > 0.0) break;
      residual = false;  // p nowhere above q: p itself
    }
    const double target = u * total;
    int found = -1;
    double base = 0.0, before = 0.0;
    for (int i0 = 0;;) {
      const double prev = lane_before(incl), excl = base + prev;
      const uint64_t any = __builtin_amdgcn_ballot_w64(v > 0.0), over = __builtin_amdgcn_ballot_w64(v > 0.0 && base + incl > target);
      if (any) {
        const int at = over ? __builtin_ctzll(over) : 63 - __builtin_clzll(any);
        found = i0 + at;
        before = __shfl(excl, at, 64);
      }
      if (over) break;
      base += last_lane(incl);
      i0 += 64;
      if (i0 >= a.chunks) break;
      v = share(i0 + lane);
      incl = wave_scan(v);
    }
    if (lane == 0) {
      sh_found = found;
      sh_before = before;
      sh_target = target;
      sh_residual = residual;
    }
  }
  __syncthreads();
  const int f = sh_found;
  if (f < 0) {
    if (threadIdx.x == 0) *token = -1;
    return;
  }
  // The entry: eight in a row per thread.
  d.residual = sh_residual != 0;
  const double target = sh_target;
  const int b0 = f * kVocabChunk + (int)threadIdx.x * kEach;
  double e[kEach], mine = 0.0;
#pragma unroll
  for (int i = 0; i < kEach; i += kVec<kType>) entries16<kType>(d, row, b0 + i, V, (f + 1) * kVocabChunk <= V, e + i);
#pragma unroll
  for (int i = 0; i < kEach; ++i) mine += e[i];
  const double incl = wave_scan(mine);
  if (lane == 63) part[wave] = incl;
  __syncthreads();
  double sum = sh_before;
  for (int i = 0; i < wave; ++i) sum += part[i];
  sum += lane_before(incl);
  int at = INT_MAX, last = -1;  // first entry over the target; last one that holds anything
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    sum += e[i];
    if (e[i] > 0.0) {
      last = b0 + i;
      if (sum > target) at = min(at, b0 + i);
    }
  }
  at = wave_min(at, lane);
  last = -wave_min(-last, lane);
  if (lane == 0) {
    wat[wave] = at;
    wlast[wave] = last;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kWaves; ++i) {
      at = min(at, wat[i]);
      last = max(last, wlast[i]);
    }
    *token = at != INT_MAX ? at : last;
  }
}

size_t up(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

VerifyDraftLayout verify_draft_layout(int64_t S, int W, int V) {
  VerifyDraftLayout l{};
  l.chunks = (V + kVocabChunk - 1) / kVocabChunk;
  l.stats = 0;
  l.mass = up(sizeof(ChunkStat) * (size_t)(S * W) * l.chunks);
  l.done = l.mass + up(sizeof(double) * (size_t)S * l.chunks);
  l.total = l.done + up(sizeof(uint32_t) * (size_t)S);
  return l;
}

hipError_t launch_verify_draft(const VerifyDraftCall& c, hipStream_t s) {
  const VerifyDraftLayout l = verify_draft_layout(c.S, c.W, c.V);
  uint8_t* const ws = static_cast<uint8_t*>(c.workspace);
  VerifyArgs a{};
  a.logits = static_cast<const uint8_t*>(c.logits);
  a.draft = c.draft;
  a.q = c.q;
  a.len = c.len;
  a.temperature = c.temperature;
  a.u_accept = c.u_accept;
  a.u_sample = c.u_sample;
  a.S = c.S;
  a.W = c.W;
  a.V = c.V;
  a.chunks = l.chunks;
  a.stats = reinterpret_cast<ChunkStat*>(ws + l.stats);
  a.mass = reinterpret_cast<double*>(ws + l.mass);
  a.done = reinterpret_cast<uint32_t*>(ws + l.done);
  a.accepted = c.accepted;
  a.tokens = c.tokens;
  a.accept_prob = c.accept_prob;
  // Chunks of a workgroup of the second launch: each takes the proposals' test
  // first, so two where that leaves more workgroups than CUs, four where it leaves
  // four for each (by one, two, four, us: 13 x 5 x 32003 16, 17, 20; 32 x 8 x 163840
  // 63, 58, 58; 128 x 4 x 163840 140, 127, 119).
  const int64_t cus = device_cu_count();
  const int per = !c.q ? 0 : c.S * ((l.chunks + 3) / 4) >= 4 * cus ? 4 : c.S * ((l.chunks + 1) / 2) > cus ? 2 : 1;
  const unsigned wgs = (unsigned)(c.S * (per ? (l.chunks + per - 1) / per : 1));
  const unsigned rows = 1 + (wgs >> 22);  // (a grid dimension has fewer than 2^32 threads)
  const dim3 g1((unsigned)(c.S * c.W * l.chunks)), g2((wgs + rows - 1) / rows, rows);
  auto go = [&](auto type) -> hipError_t {
    constexpr int kType = decltype(type)::value;
    hipLaunchKernelGGL(stats_kernel<kType>, g1, dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (per == 0) hipLaunchKernelGGL((choose_kernel<kType, 0>), g2, dim3(kChooseThreads), 0, s, a);
    else if (per == 1) hipLaunchKernelGGL((choose_kernel<kType, 1>), g2, dim3(kChooseThreads), 0, s, a);
    else if (per == 2) hipLaunchKernelGGL((choose_kernel<kType, 2>), g2, dim3(kChooseThreads), 0, s, a);
    else hipLaunchKernelGGL((choose_kernel<kType, 4>), g2, dim3(kChooseThreads), 0, s, a);
    return hipGetLastError();
  };
  if (c.dtype == K3MOE_DTYPE_F32) return go(std::integral_constant<int, K3MOE_DTYPE_F32>{});
  if (c.dtype == K3MOE_DTYPE_BF16) return go(std::integral_constant<int, K3MOE_DTYPE_BF16>{});
  return go(std::integral_constant<int, K3MOE_DTYPE_F16>{});
}

}  // namespace k3moe
