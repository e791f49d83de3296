// The whole routed layer for a few tokens (T <= 16) in two launches: a plan
// (routing, grouping, x in operand order) and one persistent kernel that runs
// gate/up, down and the weighted sum of all experts without a launch between
// them.  Weights, routing and arithmetic are those of moe_route_topk and
// moe_mxfp4_ffn (bf16 x, exact MXFP4 weights, fp32 MFMA accumulation, SiLU(g) *
// u in fp32), except that h enters the down product as three bf16 parts
// (h = hi + mid + lo, exact to 2^-24), so its rounding stays below that of the
// fp32 sums.
//
// With a few tokens the layer is a stream over the chosen experts' bytes
// (about 4 flop per byte and row): what costs time beside the stream are its
// interruptions, the drain and refill of the memory pipeline at every launch.
// The persistent kernel has none: a wave takes units of work from one list,
//   1. gate/up units: 16 features of w1 and of w3 for a tile of up to 4 rows of
//      one expert, over all of D;
//   2. down units: 32 features of w2 for one grouped row (three columns: its
//      hi, mid and lo parts), over all of I;
//   3. sum units: 32 features of out for all tokens, slots in order;
// in that order, expert by expert, and streams their weights through a private
// ring of three LDS stages that runs on across units.
//
// Hand-over.  A down unit needs every gate/up unit of its tile, a sum unit every
// down unit of its features.  Units are taken by a global ticket (atomic add),
// and a wave works on its units in ticket order, so a unit waits only for
// units of lower tickets, each of which has been taken by a wave that is
// already running and that waits for still lower ones only: by induction every
// wait ends, however many of the workgroups are resident and whatever else
// the device runs.  (The wait loops are bounded all the same; a wait that ran
// out would give NaN outputs.)  A wave never waits with an unfinished unit in
// its ring: a down unit that is not ready is held back until the ring is empty.
//
// Visibility.  Results (h parts, y) are written with device-scope stores, which
// go through the XCD's L2, and counted (device-scope add, no return) once the
// store has completed, that is once a later wait of the in-order vector-memory
// counter covers it: three stages later, at no cost, or at once where the ring
// runs dry.  A release fence would write back the whole L2 instead.  The
// reader checks the count, then takes an acquire fence, after which its plain
// loads see what was counted.  A wave checks only until it has seen every
// gate/up unit counted.
#include "route_device.h"
#include "stream_device.h"

namespace k3moe {
namespace {

// ---------------------------------------------------------------------------
// Plan.  Workgroup 0 routes (a wave per token), groups the T * k entries by
// expert and clears the counters of the main kernel; the others write x in the
// operand order of the decoded blocks (P order).
constexpr int kPlanThreads = 1024;
constexpr int kGuTileRows = 4;

struct LayerPlan {
  const float* logits;
  const float* bias;
  const uint16_t* x;
  int T, D, E, k, normalize;
  float route_scale;
  int32_t* ids;    // [T, k]
  float* w;        // [T, k]
  uint16_t* xp;    // [T, D]
  int4* gt;        // gate/up tiles: expert, first row, rows
  int2* rows;      // grouped rows: expert, gate/up tile
  int32_t* row_tok;
  int32_t* slot_row;
  int32_t* head;   // [0] gate/up tiles, [1] next ticket, [2] gate/up units counted
  uint32_t* flags;
  int n_flags;
};

template <int NPER>
__global__ __launch_bounds__(kPlanThreads) void layer_plan_kernel(LayerPlan p) {
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    // position 8i + 2t (+1) of a 32-block holds element 4i + t (16 + 4i + t)
    const int64_t n = (int64_t)p.T * p.D / 8;
    const int64_t u = (int64_t)(blockIdx.x - 1) * kPlanThreads + tid;
    if (u >= n) return;
    const uint16_t* src = p.x + (u >> 2) * 32 + 4 * (u & 3);
    const uint2 lo = *reinterpret_cast<const uint2*>(src), hi = *reinterpret_cast<const uint2*>(src + 16);
    uint4 r;
    r.x = __builtin_amdgcn_perm(hi.x, lo.x, 0x05040100u);
    r.y = __builtin_amdgcn_perm(hi.x, lo.x, 0x07060302u);
    r.z = __builtin_amdgcn_perm(hi.y, lo.y, 0x05040100u);
    r.w = __builtin_amdgcn_perm(hi.y, lo.y, 0x07060302u);
    reinterpret_cast<uint4*>(p.xp)[u] = r;
    return;
  }
  __shared__ uint32_t s_mask[K3MOE_MAX_EXPERTS_FFN];  // tokens of each expert
  __shared__ uint32_t s_base[K3MOE_MAX_EXPERTS_FFN];  // first row | first gate/up tile << 16
  __shared__ int s_ids[K3MOE_MAX_LAYER_TOKENS * K3MOE_MAX_TOPK];
  __shared__ int s_sum[kPlanThreads / 64][2];
  const int lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < p.E; e += kPlanThreads) s_mask[e] = 0u;
  for (int i = tid; i < p.n_flags; i += kPlanThreads) p.flags[i] = 0u;
  const int n = p.T * p.k;
  if constexpr (NPER > 0) {
    __shared__ RouteScratch scratch[kPlanThreads / 64];
    if (wave < p.T) {
      int id = 0;
      float g = 0.0f;
      route_token_reg<NPER>(p.logits + (int64_t)wave * p.E, p.bias, p.E, p.k, p.normalize, p.route_scale, lane, scratch[wave], id, g);
      if (lane < p.k) {
        p.ids[wave * p.k + lane] = id;
        p.w[wave * p.k + lane] = g;
        s_ids[wave * p.k + lane] = id;
      }
    }
  } else {
    for (int i = tid; i < n; i += kPlanThreads) s_ids[i] = p.ids[i];
  }
  __syncthreads();
  // a token's ids are distinct experts in range (the router's), so every entry is a row
  if (tid < n) atomicOr(&s_mask[s_ids[tid]], 1u << (tid / p.k));
  __syncthreads();
  // rows and tiles in expert order: thread i scans experts [i * per, (i + 1) * per)
  const int per = (p.E + kPlanThreads - 1) / kPlanThreads;
  int c[2] = {0, 0};
  for (int e = tid * per; e < min((tid + 1) * per, p.E); ++e) {
    const int m = __popc(s_mask[e]);
    c[0] += m;
    c[1] += (m + kGuTileRows - 1) / kGuTileRows;
  }
  int incl[2] = {c[0], c[1]};
#pragma unroll
  for (int d = 1; d < 64; d <<= 1)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int o = __shfl_up(incl[j], d, 64);
      if (lane >= d) incl[j] += o;
    }
  if (lane == 63) s_sum[wave][0] = incl[0], s_sum[wave][1] = incl[1];
  __syncthreads();
  int at[2] = {incl[0] - c[0], incl[1] - c[1]}, tiles = 0;
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    if (w < wave) at[0] += s_sum[w][0], at[1] += s_sum[w][1];
    tiles += s_sum[w][1];
  }
  for (int e = tid * per; e < min((tid + 1) * per, p.E); ++e) {
    const int m = __popc(s_mask[e]);
    if (m == 0) continue;
    s_base[e] = (uint32_t)at[0] | (uint32_t)at[1] << 16;
    for (int r = 0; r < m; r += kGuTileRows) p.gt[at[1]++] = make_int4(e, at[0] + r, min(kGuTileRows, m - r), 0);
    at[0] += m;
  }
  __syncthreads();
  if (tid < n) {
    const int e = s_ids[tid], t = tid / p.k;
    const int rank = __popc(s_mask[e] & ((1u << t) - 1u));
    const uint32_t b = s_base[e];
    const int row = (int)(b & 0xFFFFu) + rank;
    p.slot_row[tid] = row;
    p.row_tok[row] = t;
    p.rows[row] = make_int2(e, (int)(b >> 16) + rank / kGuTileRows);
  }
  if (tid == 0) {
    p.head[0] = tiles;
    p.head[1] = 0;
    p.head[2] = 0;
  }
}

// ---------------------------------------------------------------------------
constexpr int kWaves = 4;            // waves per workgroup, one workgroup per CU
constexpr int kRing = 3;             // LDS stages per wave
constexpr int kStageK = 512;         // K per stage: 16 blocks of each row
constexpr int kStageRowBytes = 272;  // bytes of a weight row per whole stage
constexpr int kRowDw = 68;
constexpr int kMatBytes = 16 * kStageRowBytes;  // a 16-row group of a stage
constexpr int kWBytes = 2 * kMatBytes;
constexpr int kActRow = 1040;        // LDS bytes per activation row (1024 + 16)
constexpr int kActRows = 4;
constexpr int kStageBytes = kWBytes + kActRows * kActRow;
constexpr int kMatLoads = 5;         // 16-byte-a-lane loads of a group's stage (4352 bytes)
constexpr int kW = 2 * kMatLoads;    // weight loads per stage
constexpr int kNt = 2;               // cache policy of the weight loads: nontemporal
constexpr int kSpinLimit = 1 << 21;
static_assert(kWaves * kRing * kStageBytes <= 160 * 1024, "LDS");

enum { kGateUp = 0, kDown = 1, kSum = 2, kNone = 3 };

struct LayerArgs {
  const uint16_t* xp;
  const uint8_t *w1, *w3, *w2;
  int D, I, T, k;
  const int4* gt;
  const int2* rows;
  const int32_t* row_tok;
  const int32_t* slot_row;
  const float* w;
  int32_t* head;
  uint32_t* flags;  // [rows] gate/up units done per tile, then [D / 32] down units done per feature group
  uint16_t* h;      // [3][rows][hstride] bf16 parts in P order
  int64_t hplane;   // elements between the parts
  int hstride;      // elements between rows
  float* y;         // [rows][D]
  float* out;       // [T, D]
};

struct Unit {
  int kind, fg, expert, row0, nrows, tile;
};

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ void store_dev(uint16_t* p, uint32_t v) {
  __hip_atomic_store(p, (uint16_t)v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_dev(float* p, f32x4_t v) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 a = {v[0], v[1]}, b = {v[2], v[3]};
  uint64_t* q = reinterpret_cast<uint64_t*>(p);
  __hip_atomic_store(q, __builtin_bit_cast(uint64_t, a), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(q + 1, __builtin_bit_cast(uint64_t, b), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Blocks of the last, shorter stage (width blocks per row): MFMA rounds one at
// a time, block b of row rho at byte (rho * width + b) * 17 of the group.
__device__ __forceinline__ void tail_round(const uint8_t* group, int rho, int b, int width, bf16x8_t op[4]) {
  const int bb = min(b, width - 1);
  const uint32_t at = (uint32_t)(rho * width + bb) * 17u, sh = at & 3u;
  const uint32_t* d = reinterpret_cast<const uint32_t*>(group) + (at >> 2);
  const uint32_t sel = 0x03020100u + 0x01010101u * (sh + 1u);  // bytes sh + 1 .. of two neighbouring dwords
  uint32_t v[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = d[i];
  const float sf = e8m0_to_f32(__builtin_amdgcn_ubfe(v[0], 8 * sh, 8));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t q = __builtin_amdgcn_perm(v[i + 1], v[i], sel);
    op[i] = decode_dword(b < width ? q : 0u, sf);
  }
}

__global__ __launch_bounds__(kWaves * 64, 1) void layer_main_kernel(LayerArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves][kRing][kStageBytes];
  __shared__ int fifo[kWaves][4][8];
  __shared__ int s_first;

  const int lane = threadIdx.x & 63;
  const int wave = uni(threadIdx.x >> 6);
  const int rho = lane & 15, g = lane >> 4;
  const int nrows = a.T * a.k;
  const int nfg = a.I >> 4, nfu = a.D >> 5;
  const int n_gu = *as_const(a.head) * nfg, n_dn = nrows * nfu;
  const uint32_t row_b13 = (uint32_t)(a.D >> 5) * 17, row_b2 = (uint32_t)(a.I >> 5) * 17;
  const int nst13 = (a.D + kStageK - 1) / kStageK, nst2 = (a.I + kStageK - 1) / kStageK;

  auto claim = [&]() -> int {
    int v = 0;
    if (lane == 0) v = __hip_atomic_fetch_add(a.head + 1, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return uni(v);
  };
  auto unit_of = [&](int t) -> Unit {
    if (t < n_gu) {
      const int i = t / nfg;
      const auto q = as_const(reinterpret_cast<const int32_t*>(a.gt)) + 4 * i;
      return Unit{kGateUp, t - i * nfg, q[0], q[1], q[2], i};
    }
    t -= n_gu;
    if (t < n_dn) {
      const int r = t / nfu;
      const auto q = as_const(reinterpret_cast<const int32_t*>(a.rows)) + 2 * r;
      return Unit{kDown, t - r * nfu, q[0], r, 1, q[1]};
    }
    t -= n_dn;
    return Unit{t < nfu ? kSum : kNone, t, 0, 0, 0, 0};
  };

  // the workgroup's first four tickets in one add
  if (threadIdx.x == 0) s_first = __hip_atomic_fetch_add(a.head + 1, kWaves, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  Unit iu = unit_of(uni(s_first) + wave);  // the unit to issue next (or being issued)

  uint32_t woff[kMatLoads];
#pragma unroll
  for (int j = 0; j < kMatLoads; ++j) {
    const int c = 64 * j + lane;
    woff[j] = c < 16 * 17 ? 16u * (uint32_t)c : 0u;
  }
  const bool wtail = lane < 16 * 17 - 64 * (kMatLoads - 1);

  // ---- issue side
  const uint8_t* wbase[2];
  uint32_t wrows = 0;  // bytes of a 16-row group
  uint32_t xsrc[kActRows];
  int is = 0, ist = 0;      // stage of iu, its number of stages
  bool open = false;        // iu's loads have begun
  bool bad = false;         // a bounded wait ran out
  bool all_done = false;    // every gate/up unit has been seen counted
  int pushed = 0, popped = 0;

  auto prep = [&]() {
    if (iu.kind == kGateUp) {
      const size_t off = (size_t)iu.expert * a.I * row_b13 + (size_t)(16 * iu.fg) * row_b13;
      wbase[0] = a.w1 + off;
      wbase[1] = a.w3 + off;
      wrows = 16 * row_b13;
      ist = nst13;
#pragma unroll
      for (int m = 0; m < kActRows; ++m)
        xsrc[m] = (uint32_t)as_const(a.row_tok)[iu.row0 + (m < iu.nrows ? m : 0)] * (uint32_t)a.D * 2;
    } else {
      const size_t off = (size_t)iu.expert * a.D * row_b2 + (size_t)(32 * iu.fg) * row_b2;
      wrows = 16 * row_b2;
      wbase[0] = a.w2 + off;
      wbase[1] = a.w2 + off + wrows;
      ist = nst2;
    }
    is = 0;
    open = true;
    int* f = fifo[wave][pushed & 3];
    ++pushed;
    if (lane == 0) {
      f[0] = iu.kind, f[1] = iu.fg, f[2] = iu.row0, f[3] = iu.nrows, f[4] = iu.tile;
    }
  };
  // issues one stage of iu into ring buffer `buf`; returns its activation loads
  auto issue = [&](int buf) -> int {
    uint8_t* dst = &lds[wave][buf][0];
    const uint32_t wso = (uint32_t)(kMatBytes * is);
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
      const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc((void*)wbase[mi], 0, (int)wrows, 0x00020000);
#pragma unroll
      for (int j = 0; j < kMatLoads - 1; ++j) {
        const uint32_t vo = woff[j];
        __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (__attribute__((address_space(3))) void*)(uintptr_t)(dst + mi * kMatBytes + 1024 * j),
                                                 16, vo, wso, 0, kNt);
      }
      if (wtail) {
        const uint32_t vo = woff[kMatLoads - 1];
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            wr, (__attribute__((address_space(3))) void*)(uintptr_t)(dst + mi * kMatBytes + 1024 * (kMatLoads - 1)), 16, vo, wso, 0, kNt);
      }
    }
    uint8_t* adst = dst + kWBytes;
    const uint32_t aso = (uint32_t)(kStageK * 2 * is);
    int n = 0;
    if (iu.kind == kGateUp) {
      const __amdgpu_buffer_rsrc_t xr =
          __builtin_amdgcn_make_buffer_rsrc((void*)a.xp, 0, (int)((uint32_t)a.T * (uint32_t)a.D * 2), 0x00020000);
#pragma unroll
      for (int m = 0; m < kActRows; ++m)
        if (m < iu.nrows) {
          const uint32_t so = xsrc[m] + aso;
          __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (__attribute__((address_space(3))) void*)(uintptr_t)(adst + kActRow * m), 16,
                                                   16 * lane, so, 0, 0);
        }
      n = iu.nrows;
    } else {
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        const uint16_t* hb = a.h + m * a.hplane + (int64_t)iu.row0 * a.hstride;
        const __amdgpu_buffer_rsrc_t hr = __builtin_amdgcn_make_buffer_rsrc((void*)hb, 0, a.I * 2, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(hr, (__attribute__((address_space(3))) void*)(uintptr_t)(adst + kActRow * m), 16,
                                                 16 * lane, aso, 0, 0);
      }
      n = 3;
    }
    if (++is == ist) {
      open = false;
      iu = unit_of(claim());
    }
    return n;
  };
  auto seen = [&](const uint32_t* f) -> uint32_t {
    return (uint32_t)uni((int)__hip_atomic_load(f, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  };
  // whether iu can be issued now (no waiting)
  auto ready = [&]() -> bool {
    if (iu.kind == kGateUp) return true;
    if (iu.kind != kDown) return false;
    if (all_done) return true;
    if (seen(a.flags + iu.tile) < (uint32_t)nfg) return false;
    all_done = seen(reinterpret_cast<const uint32_t*>(a.head) + 2) >= (uint32_t)n_gu;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    return true;
  };

  // ---- publishing
  int pub[3] = {-1, -1, -1};  // flags of finished units, by age in stages
  auto publish = [&](int f) {
    if (f >= 0 && lane == 0) {
      (void)__hip_atomic_fetch_add(a.flags + f, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (f < nrows) (void)__hip_atomic_fetch_add(a.head + 2, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  };
  auto flush = [&]() {
    wait_vm<0>();
#pragma unroll
    for (int i = 2; i >= 0; --i) {
      publish(pub[i]);
      pub[i] = -1;
    }
  };

  f32x4_t acc[2][2];
#pragma unroll
  for (int mi = 0; mi < 2; ++mi) acc[mi][0] = acc[mi][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const uint32_t qsel = 0x03020100u + 0x01010101u * (uint32_t)(g + 1);

  int buf_i = 0, buf_c = 0, inflight = 0;
  int na[kRing] = {0, 0, 0};  // activation loads of the stages in flight, oldest first
  Unit cu{kNone, 0, 0, 0, 0, 0};
  int cs = 0, cst = 0;  // stage of cu, its number of stages (0: no unit)
  int boff = kWBytes;

  for (;;) {
    while (inflight < kRing) {
      if (!open) {
        if (!ready()) break;
        prep();
      }
      const int n = issue(buf_i);
      buf_i = buf_i == kRing - 1 ? 0 : buf_i + 1;
      if (inflight == 0) na[0] = n;
      else if (inflight == 1) na[1] = n;
      else na[2] = n;
      ++inflight;
    }
    if (inflight == 0) {
      // the ring is empty and iu cannot start: count what is finished, then wait
      flush();
      if (iu.kind == kNone) break;
      const uint32_t* f = a.flags + (iu.kind == kDown ? iu.tile : nrows + iu.fg);
      const uint32_t need = iu.kind == kDown ? (uint32_t)nfg : (uint32_t)nrows;
      int spins = 0;
      while (seen(f) < need) {
        __builtin_amdgcn_s_sleep(2);
        if (++spins > kSpinLimit) {
          bad = true;
          break;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      if (iu.kind == kSum) {
        // eight lanes a token (four features each), eight tokens at a time
        const int f4 = 32 * iu.fg + 4 * (lane & 7);
        for (int t = lane >> 3; t < a.T; t += 8) {
          f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
          for (int j = 0; j < a.k; ++j) {
            const float wt = a.w[t * a.k + j];
            const f32x4_t v = *reinterpret_cast<const f32x4_t*>(a.y + (int64_t)a.slot_row[t * a.k + j] * a.D + f4);
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[c] = fmaf(wt, v[c], sum[c]);
          }
          if (bad) sum[0] = sum[1] = sum[2] = sum[3] = __uint_as_float(0x7FC00000u);
          *reinterpret_cast<f32x4_t*>(a.out + (int64_t)t * a.D + f4) = sum;
        }
        iu = unit_of(claim());
      } else {
        prep();
        const int n = issue(buf_i);
        buf_i = buf_i == kRing - 1 ? 0 : buf_i + 1;
        na[0] = n;
        inflight = 1;
      }
      continue;
    }

    // the oldest stage has landed once only the loads of the newer ones are out
    if (inflight == 3)
      wait_vm_plus<2 * kW>(na[1] + na[2]);
    else if (inflight == 2)
      wait_vm_plus<kW>(na[1]);
    else
      wait_vm<0>();
    // a unit finished three stages ago: its stores are older than these loads
    publish(pub[2]);
    pub[2] = pub[1];
    pub[1] = pub[0];
    pub[0] = -1;
    if (cst == 0) {
      const int* f = fifo[wave][popped & 3];
      ++popped;
      cu.kind = uni(f[0]), cu.fg = uni(f[1]), cu.row0 = uni(f[2]), cu.nrows = uni(f[3]), cu.tile = uni(f[4]);
      cs = 0;
      cst = cu.kind == kGateUp ? nst13 : nst2;
      // column rho reads activation row rho: tile row (gate/up), part of h
      // (down); the other columns repeat row 0 and are dropped
      boff = kWBytes + kActRow * (rho < (cu.kind == kGateUp ? cu.nrows : 3) ? rho : 0);
    }
    const uint8_t* st = &lds[wave][buf_c][0];
    buf_c = buf_c == kRing - 1 ? 0 : buf_c + 1;
    --inflight;
    na[0] = na[1];
    na[1] = na[2];
    const int width = (cu.kind == kGateUp ? a.D : a.I) / 32 - 16 * cs;  // blocks left
    const uint8_t* bl = st + boff;
    if (width >= 16) {
      const uint32_t* wl = reinterpret_cast<const uint32_t*>(st);
      bf16x8_t bop[4][4];
#pragma unroll
      for (int rnd = 0; rnd < 4; ++rnd)
#pragma unroll
        for (int i = 0; i < 4; ++i) bop[rnd][i] = *reinterpret_cast<const bf16x8_t*>(bl + 64 * (4 * rnd + g) + 16 * i);
      uint32_t wd[2][4][5];
#pragma unroll
      for (int mi = 0; mi < 2; ++mi)
#pragma unroll
        for (int rnd = 0; rnd < 4; ++rnd)
#pragma unroll
          for (int j = 0; j < 5; ++j) wd[mi][rnd][j] = wl[(16 * mi + rho) * kRowDw + 17 * rnd + 4 * g + j];
#pragma unroll
      for (int r0 = 0; r0 < 4; r0 += 2) {
        bf16x8_t aop[2][2][4];
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) decode_dwords(wd[mi][r0 + rr], g, qsel, aop[mi][rr]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int rr = 0; rr < 2; ++rr)
#pragma unroll
            for (int mi = 0; mi < 2; ++mi)
              acc[mi][rr] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(aop[mi][rr][i], bop[r0 + rr][i], acc[mi][rr], 0, 0, 0);
      }
    } else {
      for (int rnd = 0; 4 * rnd < width; ++rnd) {
        const int b = 4 * rnd + g;
        bf16x8_t aop[2][4];
        tail_round(st, rho, b, width, aop[0]);
        tail_round(st + kMatBytes, rho, b, width, aop[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 q = *reinterpret_cast<const uint4*>(bl + 64 * b + 16 * i);
          if (b >= width) q = make_uint4(0u, 0u, 0u, 0u);  // past K: whatever the buffer holds
          const bf16x8_t bo = __builtin_bit_cast(bf16x8_t, q);
#pragma unroll
          for (int mi = 0; mi < 2; ++mi)
            acc[mi][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(aop[mi][i], bo, acc[mi][0], 0, 0, 0);
        }
      }
    }

    if (++cs == cst) {
      // lane holds, in column rho, features 4g + v of both 16-row groups
      f32x4_t sum[2];
#pragma unroll
      for (int mi = 0; mi < 2; ++mi) {
        sum[mi] = acc[mi][0] + acc[mi][1];
        acc[mi][0] = acc[mi][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      if (cu.kind == kGateUp) {
        if (rho < cu.nrows) {
          // feature 16 fg + 4g + v is element 16 (fg & 1) + 4g + v of I-block
          // fg / 2, at its P-order position 8g + 2v + (fg & 1)
          uint16_t* h = a.h + (int64_t)(cu.row0 + rho) * a.hstride + 32 * (cu.fg >> 1) + 8 * g + (cu.fg & 1);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float gt = sum[0][v], up = sum[1][v];
            const float hv = gt / (1.0f + expf(-gt)) * up;
            const uint32_t hi = f32_to_bf16_bits(hv);
            // no remainder of an infinity or a NaN
            const float r1 = (hi & 0x7F80u) == 0x7F80u ? 0.0f : hv - __uint_as_float(hi << 16);
            const uint32_t mid = f32_to_bf16_bits(r1);
            const uint32_t lo = f32_to_bf16_bits(r1 - __uint_as_float(mid << 16));
            store_dev(h + 2 * v, hi);
            store_dev(h + a.hplane + 2 * v, mid);
            store_dev(h + 2 * a.hplane + 2 * v, lo);
          }
        }
        pub[0] = cu.tile;
      } else {
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            sum[mi][v] += __shfl_down(sum[mi][v], 1, 16) + __shfl_down(sum[mi][v], 2, 16);
        if (rho == 0) {
          float* y = a.y + (int64_t)cu.row0 * a.D + 32 * cu.fg + 4 * g;
          if (bad) sum[0][0] = sum[1][0] = __uint_as_float(0x7FC00000u);
#pragma unroll
          for (int mi = 0; mi < 2; ++mi) store_dev(y + 16 * mi, sum[mi]);
        }
        pub[0] = nrows + cu.fg;
      }
      cst = 0;
    }
  }
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct LayerWorkspace {
  size_t ids, w, xp, gt, rows, row_tok, slot_row, head, flags, h, y, total;
  int64_t n, n_flags;
  int hstride;
};
LayerWorkspace layer_layout(int64_t T, int32_t D, int32_t I, int32_t k) {
  LayerWorkspace l{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  l.n = T * k;
  l.n_flags = l.n + D / 32;
  l.hstride = (I + 127) / 128 * 128;  // rows start on 256-byte lines
  l.ids = take(4 * l.n);
  l.w = take(4 * l.n);
  l.xp = take((size_t)T * D * 2);
  l.gt = take(16 * l.n);
  l.rows = take(8 * l.n);
  l.row_tok = take(4 * l.n);
  l.slot_row = take(4 * l.n);
  l.head = take(16);
  l.flags = take(4 * l.n_flags);
  l.h = take((size_t)3 * l.n * l.hstride * 2);
  l.y = take((size_t)l.n * D * 4);
  l.total = off;
  return l;
}

}  // namespace

size_t layer_workspace_bytes(int64_t T, int32_t D, int32_t I, int32_t k) { return layer_layout(T, D, I, k).total; }

hipError_t launch_layer(const LayerCall& c, hipStream_t s) {
  const LayerWorkspace l = layer_layout(c.T, c.D, c.I, c.k);
  uint8_t* const ws = static_cast<uint8_t*>(c.workspace);
  LayerPlan p{};
  p.logits = c.logits;
  p.bias = c.bias;
  p.x = c.x;
  p.T = c.T;
  p.D = c.D;
  p.E = c.E;
  p.k = c.k;
  p.normalize = c.normalize;
  p.route_scale = c.route_scale;
  p.ids = c.ids ? c.ids : reinterpret_cast<int32_t*>(ws + l.ids);
  p.w = c.w ? c.w : reinterpret_cast<float*>(ws + l.w);
  p.xp = reinterpret_cast<uint16_t*>(ws + l.xp);
  p.gt = reinterpret_cast<int4*>(ws + l.gt);
  p.rows = reinterpret_cast<int2*>(ws + l.rows);
  p.row_tok = reinterpret_cast<int32_t*>(ws + l.row_tok);
  p.slot_row = reinterpret_cast<int32_t*>(ws + l.slot_row);
  p.head = reinterpret_cast<int32_t*>(ws + l.head);
  p.flags = reinterpret_cast<uint32_t*>(ws + l.flags);
  p.n_flags = (int)l.n_flags;
  const unsigned blocks = 1 + (unsigned)(((int64_t)c.T * c.D / 8 + kPlanThreads - 1) / kPlanThreads);
  const dim3 grid(blocks), block(kPlanThreads);
  if (c.E <= 64) hipLaunchKernelGGL(layer_plan_kernel<1>, grid, block, 0, s, p);
  else if (c.E <= 128) hipLaunchKernelGGL(layer_plan_kernel<2>, grid, block, 0, s, p);
  else if (c.E <= 256) hipLaunchKernelGGL(layer_plan_kernel<4>, grid, block, 0, s, p);
  else if (c.E <= 512) hipLaunchKernelGGL(layer_plan_kernel<8>, grid, block, 0, s, p);
  else if (c.E <= 1024) hipLaunchKernelGGL(layer_plan_kernel<16>, grid, block, 0, s, p);
  else {
    // more experts than a wave keeps in registers: the router's own launch first
    const hipError_t e = launch_route_topk(c.logits, c.bias, c.T, c.E, c.k, c.normalize, c.route_scale, p.ids, p.w, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(layer_plan_kernel<0>, grid, block, 0, s, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;

  LayerArgs a{};
  a.xp = p.xp;
  a.w1 = c.w1;
  a.w3 = c.w3;
  a.w2 = c.w2;
  a.D = c.D;
  a.I = c.I;
  a.T = c.T;
  a.k = c.k;
  a.gt = p.gt;
  a.rows = p.rows;
  a.row_tok = p.row_tok;
  a.slot_row = p.slot_row;
  a.w = p.w;
  a.head = p.head;
  a.flags = p.flags;
  a.h = reinterpret_cast<uint16_t*>(ws + l.h);
  a.hplane = l.n * l.hstride;
  a.hstride = l.hstride;
  a.y = reinterpret_cast<float*>(ws + l.y);
  a.out = c.out;
  const int64_t units = l.n * (c.I / 16 + c.D / 32) + c.D / 32;
  int64_t wgs = (units + kWaves - 1) / kWaves;
  const int cus = device_cu_count();
  if (wgs > cus) wgs = cus;
  hipLaunchKernelGGL(layer_main_kernel, dim3((unsigned)wgs), dim3(kWaves * 64), 0, s, a);
  return hipGetLastError();
}

}  // namespace k3moe
