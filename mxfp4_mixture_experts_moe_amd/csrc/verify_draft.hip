// Verification of drafted tokens against the target's distribution.
//
// Row w of a sequence gives p = softmax(logits / T); proposal x of position w is
// accepted where u q(x) < p(x), and the next token comes from max(p - q, 0) at
// the first one that is not, or from p itself, by its cumulative sum in index
// order.  A sum over the vocabulary decides between neighbours that hold 1e-6 of
// it, so an fp32 sum's order would move the token; everything here is fp64
// from the logits on, and two runs (or another order of summation) differ only
// where a uniform lies within about 1e-15 of a border.
//
// Two launches, both over chunks of 4096 vocabulary entries:
//   stats   every row's chunks: largest logit, its lowest index (greedy), sum of
//           exponentials relative to the chunk's own largest;
//   choose  per sequence, the chunks of the one row that is sampled from: the
//           rows' totals out of the chunks' (each workgroup for itself, a few KB
//           from the L2), which proposals are accepted, the chunk's share of max(p
//           - q, 0); the workgroup that finishes last adds the shares up in
//           order, finds the chunk that holds the token, and the token in it.
// "Last" is a counter per sequence that the first launch clears; nothing waits.
#include "k3moe_internal.h"

#include <math.h>

namespace k3moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kEach = kVocabChunk / kThreads;  // entries per thread

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

// Logit i of a row.
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
template <int kType>
constexpr int kSize = kType == K3MOE_DTYPE_F32 ? 4 : 2;

// exp((l - m) / T) for l <= m; 0 for NaN and -inf; an infinite m is shared by those that reach it.
__device__ __forceinline__ double weight(float l, float m, double inv_t) {
  if (!(l > -INFINITY)) return 0.0;
  if (l == m) return 1.0;
  return m == INFINITY ? 0.0 : exp(((double)l - (double)m) * inv_t);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = min(v, __shfl_xor(v, d, 64));
  return v;
}

__device__ __forceinline__ float temperature_of(const VerifyArgs& a, int64_t s) { return a.temperature ? a.temperature[s] : 1.0f; }

template <int kType>
__global__ __launch_bounds__(kThreads) void stats_kernel(VerifyArgs a) {
  __shared__ float wm[kWaves];
  __shared__ double wz[kWaves];
  __shared__ int wi[kWaves];
  const int64_t r = blockIdx.x / (unsigned)a.chunks;
  const int c = (int)(blockIdx.x - r * a.chunks);
  const int64_t s = r / a.W;
  const int wave = threadIdx.x >> 6;
  if (c == 0 && r == s * a.W && threadIdx.x == 0) a.done[s] = 0u;
  const uint8_t* const row = a.logits + r * a.V * kSize<kType>;
  const int v0 = c * kVocabChunk;
  float l[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int v = v0 + i * kThreads + (int)threadIdx.x;
    l[i] = v < a.V ? logit<kType>(row, v) : -INFINITY;
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kEach; ++i) m = fmaxf(m, l[i]);  // (passes over NaN)
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) wm[wave] = m;
  __syncthreads();
  m = wm[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) m = fmaxf(m, wm[i]);
  const float t = temperature_of(a, s);
  const bool greedy = !(t > 0.0f);
  double z = 0.0;
  int at = INT_MAX;
  if (greedy) {
#pragma unroll
    for (int i = kEach - 1; i >= 0; --i)
      if (l[i] == m && m > -INFINITY) at = v0 + i * kThreads + (int)threadIdx.x;
    at = wave_min(at);
  } else {
    const double inv_t = 1.0 / (double)t;
#pragma unroll
    for (int i = 0; i < kEach; ++i) z += weight(l[i], m, inv_t);
    z = wave_sum(z);
  }
  if ((threadIdx.x & 63) == 0) {
    wz[wave] = z;
    wi[wave] = at;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kWaves; ++i) {
      z += wz[i];
      at = min(at, wi[i]);
    }
    a.stats[r * a.chunks + c] = ChunkStat{m, at, z};
  }
}

// A row's largest logit, its lowest index and its sum, out of the chunks'; by one wave, in every lane.
struct RowStat {
  float m;
  int at;
  double z;
};
__device__ __forceinline__ RowStat row_stat(const ChunkStat* st, int chunks, int lane, double inv_t, bool greedy) {
  float m = -INFINITY;
  for (int c = lane; c < chunks; c += 64) m = fmaxf(m, st[c].m);
  m = wave_max(m);
  double z = 0.0;
  int at = INT_MAX;
  for (int c = lane; c < chunks; c += 64) {
    const ChunkStat x = st[c];
    if (greedy) {
      if (x.m == m) at = min(at, x.at);
    } else {
      z += x.z * weight(x.m, m, inv_t);
    }
  }
  return RowStat{m, wave_min(at), wave_sum(z)};
}

// What is sampled from, entry v of a row: max(p - q, 0) or p.
struct Source {
  float m;
  double inv_t, inv_z;
  const float* q;  // null: q is 1 at x
  int x;           // -1: p itself
  bool residual;
};
__device__ __forceinline__ double entry(const Source& d, float l, int v) {
  const double p = weight(l, d.m, d.inv_t) * d.inv_z;
  if (!d.residual) return p;
  return fmax(p - (d.q ? (double)d.q[v] : v == d.x ? 1.0 : 0.0), 0.0);
}

template <int kType>
__global__ __launch_bounds__(kThreads) void choose_kernel(VerifyArgs a) {
  __shared__ RowStat rows[kMaxVerifyWidth];
  __shared__ double wz[kWaves];
  __shared__ double scan[kThreads];
  __shared__ int sh_count, sh_last, sh_found;
  __shared__ double sh_before;
  const int64_t s = blockIdx.x / (unsigned)a.chunks;
  const int c = (int)(blockIdx.x - s * a.chunks);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int W = a.W, V = a.V, D = W - 1;
  const float t = temperature_of(a, s);
  const bool greedy = !(t > 0.0f);
  const double inv_t = greedy ? 1.0 : 1.0 / (double)t;
  int n = a.len ? a.len[s] : D;
  n = n < 0 ? 0 : n > D ? D : n;
  for (int w = wave; w <= n; w += kWaves) {
    const RowStat st = row_stat(a.stats + (s * W + w) * a.chunks, a.chunks, lane, inv_t, greedy);
    if (lane == 0) rows[w] = st;
  }
  __syncthreads();
  // the proposals, one lane each
  if (wave == 0) {
    bool take = false;
    if (lane < D) {
      const int x = a.draft[s * D + lane];
      double chance = 0.0;
      if (lane < n && x >= 0 && x < V) {
        const RowStat st = rows[lane];
        if (greedy) {
          take = x == st.at;
          chance = take ? 1.0 : 0.0;
        } else if (st.z > 0.0) {
          const double p = weight(logit<kType>(a.logits + (s * W + lane) * V * kSize<kType>, x), st.m, inv_t) / st.z;
          const double q = a.q ? (double)a.q[(s * D + lane) * V + x] : 1.0;
          take = (double)a.u_accept[s * D + lane] * q < p;
          chance = q < p ? 1.0 : q > 0.0 ? p / q : 0.0;
        }
      }
      if (c == 0 && a.accept_prob) a.accept_prob[s * D + lane] = (float)chance;
    }
    const uint64_t no = ~__builtin_amdgcn_ballot_w64(take);
    const int count = no ? __builtin_ctzll(no) : 64;  // (D <= 63)
    if (lane == 0) sh_count = count;
    if (c == 0) {
      if (lane == 0) a.accepted[s] = count;
      if (lane < W && lane != count) a.tokens[s * W + lane] = lane < count ? a.draft[s * D + lane] : -1;
    }
  }
  __syncthreads();
  const int count = sh_count;
  const RowStat st = rows[count];
  if (greedy) {
    if (c == 0 && threadIdx.x == 0) a.tokens[s * W + count] = st.at == INT_MAX ? -1 : st.at;
    return;
  }

  const uint8_t* const row = a.logits + (s * W + count) * V * kSize<kType>;
  Source d{st.m, inv_t, st.z > 0.0 ? 1.0 / st.z : 0.0, nullptr, -1, count < n};
  if (d.residual) {
    d.x = a.draft[s * D + count];
    d.q = a.q ? a.q + (s * D + count) * V : nullptr;
  }
  const int v0 = c * kVocabChunk;
  double mass = 0.0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int v = v0 + i * kThreads + (int)threadIdx.x;
    if (v < V) mass += entry(d, logit<kType>(row, v), v);
  }
  mass = wave_sum(mass);
  if (lane == 0) wz[wave] = mass;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kWaves; ++i) mass += wz[i];
    __hip_atomic_store(a.mass + s * a.chunks + c, mass, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sh_last = __hip_atomic_fetch_add(a.done + s, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)a.chunks - 1u;
  }
  __syncthreads();
  if (!sh_last) return;

  // The last workgroup of the sequence: the chunk, then the entry.
  const double u = (double)a.u_sample[s];
  const ChunkStat* const cs = a.stats + (s * W + count) * a.chunks;
  if (threadIdx.x == 0) {
    auto load = [&](int i) { return __hip_atomic_load(a.mass + s * a.chunks + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    auto share = [&](int i) { return d.residual ? load(i) : cs[i].z * weight(cs[i].m, d.m, inv_t) * d.inv_z; };
    double total = 0.0;
    for (int i = 0; i < a.chunks; ++i) total += share(i);
    if (d.residual && !(total > 0.0)) {  // p nowhere above q: p itself
      d.residual = false;
      total = 0.0;
      for (int i = 0; i < a.chunks; ++i) total += share(i);
    }
    sh_count = d.residual;
    // the first chunk whose cumulative sum exceeds the target; past the end (a uniform of 1), the last that holds anything
    double sum = 0.0, before = 0.0;
    int found = -1;
    for (int i = 0; i < a.chunks; ++i) {
      const double x = share(i);
      if (x > 0.0) {
        found = i;
        before = sum;
        if (sum + x > u * total) break;
      }
      sum += x;
    }
    sh_found = found;
    sh_before = before;
    wz[0] = u * total;
  }
  __syncthreads();
  d.residual = sh_count != 0;
  const int f = sh_found;
  if (f < 0) {
    if (threadIdx.x == 0) a.tokens[s * W + count] = -1;
    return;
  }
  const double target = wz[0];
  const int b0 = f * kVocabChunk + (int)threadIdx.x * kEach;
  double e[kEach], own = 0.0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    e[i] = b0 + i < V ? entry(d, logit<kType>(row, b0 + i), b0 + i) : 0.0;
    own += e[i];
  }
  scan[threadIdx.x] = own;
  __syncthreads();
  for (int step = 1; step < kThreads; step <<= 1) {
    const double o = (int)threadIdx.x >= step ? scan[threadIdx.x - step] : 0.0;
    __syncthreads();
    scan[threadIdx.x] += o;
    __syncthreads();
  }
  double sum = sh_before + (threadIdx.x ? scan[threadIdx.x - 1] : 0.0);
  int at = INT_MAX, last = -1;  // first entry over the target; last one that holds anything
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    sum += e[i];
    if (e[i] > 0.0) {
      last = b0 + i;
      if (sum > target) at = min(at, b0 + i);
    }
  }
  at = wave_min(at);
  last = -wave_min(-last);
  __shared__ int wat[kWaves], wlast[kWaves];
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
    a.tokens[s * W + count] = at != INT_MAX ? at : last;
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
  const dim3 g1((unsigned)(c.S * c.W * l.chunks)), g2((unsigned)(c.S * l.chunks)), block(kThreads);
  auto go = [&](auto k1, auto k2) -> hipError_t {
    hipLaunchKernelGGL(k1, g1, block, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k2, g2, block, 0, s, a);
    return hipGetLastError();
  };
  if (c.dtype == K3MOE_DTYPE_F32) return go(stats_kernel<K3MOE_DTYPE_F32>, choose_kernel<K3MOE_DTYPE_F32>);
  if (c.dtype == K3MOE_DTYPE_BF16) return go(stats_kernel<K3MOE_DTYPE_BF16>, choose_kernel<K3MOE_DTYPE_BF16>);
  return go(stats_kernel<K3MOE_DTYPE_F16>, choose_kernel<K3MOE_DTYPE_F16>);
}

}  // namespace k3moe
