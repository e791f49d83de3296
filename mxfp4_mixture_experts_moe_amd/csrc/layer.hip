// The whole routed layer for a few tokens (T <= 16) in two launches: a plan
// (routing, grouping, x in operand form) and one persistent kernel that runs
// gate/up, down and the weighted sum of all experts without a launch between
// them.  Weights, routing and formulas are those of moe_route_topk and
// moe_mxfp4_ffn.
//
// Products.  The 4-bit weights go into the block-scaled matrix instructions as
// they are stored (16 bytes of codes and one scale byte per block), so decoding
// costs five register operations a block.  The other operand is fp8 there, so
// activations enter as fixed-point digits: with q = v / 2^s, 2^s chosen per
// 32-block so that the block's largest |q| lies in [8, 16),
//   d0 = rint(q), d1 = rint(32 (q - d0)), d2 = rint(32 (32 (q - d0) - d1)), ...
// every digit an integer of magnitude <= 16 (exact in e4m3), digit p with the
// scale 2^(s - 5p) in a column of its own; the columns are added in fp32.  The
// instruction adds the products of a block in a fixed-point window of about
// 2^14 below the largest (measured; e4m3 operands of 8 binades already lose
// bits) and everything else in fp32: digits times E2M1 codes span 0.5 .. 96 and
// stay inside, so each column is as exact as an fp32 sum.  x takes four
// digits (2^-19 of its block's largest; a bf16 value within 2^-11 of that is
// exact), h five (2^-24).
//
// With a few tokens the layer is a stream over the chosen experts' bytes
// (about 4 flop per byte and row): what costs time beside the stream are its
// interruptions, the drain and refill of the memory pipeline at every launch.
// The persistent kernel has none: a wave takes units of work from one list,
//   1. gate/up units: 32 features of w1 and of w3 for a tile of up to two rows
//      of one expert, over all of D;
//   2. down units: 32 features of w2 for one grouped row, over all of I;
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
// out would give NaN outputs.)  A wave waits only with its earlier units
// finished: the weights of a down unit go into the ring whether its h is
// complete or not, its h follows when a look at the tile's count allows it, and
// if the unit's first stage comes up without, the wave waits then.
//
// Visibility.  Results (digits of h, y) are written with device-scope stores,
// which go through the XCD's L2, and counted (device-scope add, no return) once
// the store has completed, that is once a later wait of the in-order
// vector-memory counter covers it: three stages later, at no cost, or at once
// where the ring runs dry.  A release fence would write back the whole L2
// instead.  The reader checks the count and then reads with device-scope loads,
// which a stale line of its own L2 cannot answer; an acquire fence per check
// would invalidate that L2 (57 ns each, measured, for every wave of the XCD in
// turn).  A wave checks only until it has seen every gate/up unit counted.
#include "mx_common.h"
#include "route_device.h"
#include "stream_device.h"

#include <type_traits>

namespace k3moe {
namespace {

constexpr int kXDigits = 4, kHDigits = 5;
constexpr int kPlane = 512;     // bytes of one digit of a row's stage
constexpr int kXRow = kXDigits * kPlane;        // x: digits of a (row, stage); its scales are apart
constexpr int kHRow = kHDigits * kPlane + 16;   // h: digits and scales of a (row, stage)

// Operand order.  A lane's 16 code bytes of a block hold elements j and j + 16 in
// byte j, so digit bytes go in the order 0, 16, 1, 17, ...: element e < 16 at
// byte 2e of the block's 32, element 16 + e at byte 2e + 1.  Of a stage's plane,
// the 16-byte chunk c (block c / 2) sits at chunk c with its low three bits
// xor the digit number, so that the columns of a read fall into different
// banks.  The 16 scale bytes of a stage are transposed, block 4 r + g at byte
// 4 g + r: a lane of group g reads its four rounds as one dword.
//
// Eight values in that order (those of quarter i of the block: elements 4i + t
// and 16 + 4i + t) as N digits: out[p] = eight bytes.
template <int N>
__device__ __forceinline__ void digits8(const float (&v)[8], uint32_t e, uint2 (&out)[N]) {
  const float unit = __uint_as_float((257u - e) << 23);  // 2^(130 - e): |v| * unit < 16
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = v[i] * unit;
#pragma unroll
  for (int p = 0; p < N; ++p) {
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d[i] = rintf(q[i]);
      q[i] = (q[i] - d[i]) * 32.0f;  // exact: both are multiples of the unit's last bit
    }
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(d[0], d[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(d[2], d[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(d[4], d[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(d[6], d[7], hi, true);
    out[p] = make_uint2((uint32_t)lo, (uint32_t)hi);
  }
}
// Exponent field of a block for digits8, from its largest magnitude's bits: at
// least 23, so that the scale byte e - 3 of digit 0 leaves room for 5 * 4 less.
__device__ __forceinline__ uint32_t digit_exp(uint32_t top) { return max(top >> 23, 23u); }
// Byte offset in a stage's plane of quarter i of block bb, digit p.
__device__ __forceinline__ int digit_at(int bb, int i, int p) {
  const int c = 2 * bb + (i >> 1);
  return 16 * ((c & ~7) | ((c ^ p) & 7)) + 8 * (i & 1);
}

// ---------------------------------------------------------------------------
// Plan.  Workgroup 0 routes (a wave per token), groups the T * k entries by
// expert and clears the counters of the main kernel; the others write x as
// digits.
constexpr int kPlanThreads = 1024;
constexpr int kGuTileRows = 2;

struct LayerPlan {
  const float* logits;
  const float* bias;
  const uint16_t* x;
  int T, D, E, k, normalize;
  float route_scale;
  int32_t* ids;    // [T, k]
  float* w;        // [T, k]
  uint8_t* xd;     // [T][stages][kXRow] digits of x
  uint8_t* xs;     // [T][stages][16] their scale bytes
  int4* gt;        // gate/up tiles: expert, first row | rows << 16, tokens of the rows (a byte each), expert's tiles
                   // (first | count << 16)
  int4* rows;      // grouped rows: expert, expert's rows (first | count << 16), expert's first gate/up tile
  int32_t* slot_row;
  int32_t* head;   // [0] gate/up tiles, [1] next ticket
  uint32_t* flags;
  int n_flags;
};

template <int NPER>
__global__ __launch_bounds__(kPlanThreads) void layer_plan_kernel(LayerPlan p) {
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    // four lanes a block, eight elements each
    const int nb = p.D >> 5, nst = (nb + 15) >> 4;
    const int u = (int)(blockIdx.x - 1) * kPlanThreads + tid;
    if (u >= p.T * nb * 4) return;
    const int i = u & 3, t = (u >> 2) / nb, b = (u >> 2) - t * nb;
    const uint16_t* src = p.x + (int64_t)t * p.D + 32 * b + 4 * i;
    const uint2 lo = *reinterpret_cast<const uint2*>(src), hi = *reinterpret_cast<const uint2*>(src + 16);
    float v[8];
    v[0] = __uint_as_float(lo.x << 16), v[2] = __uint_as_float(lo.x & 0xFFFF0000u);
    v[4] = __uint_as_float(lo.y << 16), v[6] = __uint_as_float(lo.y & 0xFFFF0000u);
    v[1] = __uint_as_float(hi.x << 16), v[3] = __uint_as_float(hi.x & 0xFFFF0000u);
    v[5] = __uint_as_float(hi.y << 16), v[7] = __uint_as_float(hi.y & 0xFFFF0000u);
    const uint32_t e = digit_exp(mx_block_top(v));
    uint2 d[kXDigits];
    digits8<kXDigits>(v, e, d);
    const int64_t piece = (int64_t)t * nst + (b >> 4);
#pragma unroll
    for (int q = 0; q < kXDigits; ++q)
      *reinterpret_cast<uint2*>(p.xd + piece * kXRow + q * kPlane + digit_at(b & 15, i, q)) = d[q];
    if (i == 0) p.xs[piece * 16 + 4 * (b & 3) + ((b & 15) >> 2)] = (uint8_t)(e - 3u);
    return;
  }
  __shared__ uint32_t s_mask[K3MOE_MAX_EXPERTS_FFN];  // tokens of each expert
  __shared__ uint32_t s_base[K3MOE_MAX_EXPERTS_FFN];  // first row
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
    s_base[e] = (uint32_t)at[0];
    uint32_t toks = s_mask[e];
    const int t0 = at[1], nt = (m + kGuTileRows - 1) / kGuTileRows;
    for (int r = 0; r < m; ++r) p.rows[at[0] + r] = make_int4(e, at[0] | m << 16, t0, 0);
    for (int r = 0; r < m; r += kGuTileRows) {
      int tk = 0;
      const int nr = min(kGuTileRows, m - r);
      for (int i = 0; i < nr; ++i) {
        tk |= __builtin_ctz(toks) << (8 * i);
        toks &= toks - 1u;
      }
      p.gt[at[1]++] = make_int4(e, (at[0] + r) | nr << 16, tk, t0 | nt << 16);
    }
    at[0] += m;
  }
  __syncthreads();
  if (tid < n) {
    const int e = s_ids[tid], t = tid / p.k;
    const int rank = __popc(s_mask[e] & ((1u << t) - 1u));
    p.slot_row[tid] = (int)s_base[e] + rank;
  }
  if (tid == 0) {
    p.head[0] = tiles;
    p.head[1] = 0;
  }
}

// ---------------------------------------------------------------------------
constexpr int kWaves = 4;            // waves per workgroup, one workgroup per CU
constexpr int kRing = 3;             // LDS stages per wave
constexpr int kMatBytes = 16 * 272;  // a 16-row group of a whole stage: 16 rows x 16 blocks of 17 bytes
constexpr int kRowDw = 68;           // dwords of a row of it
constexpr int kWBytes = 2 * kMatBytes;
constexpr int kXRowLds = kXRow + 64; // second row of a gate/up tile: four 16-byte banks on
constexpr int kActBytes = kXRowLds + kXRow;  // also holds the kHRow bytes of a down row
constexpr int kStageBytes = kWBytes + kActBytes + 64;  // + scale bytes of x
constexpr int kChunks = 2 * 16 * 17; // 16-byte chunks of a stage's two groups
constexpr int kW = (kChunks + 63) / 64;  // weight loads per stage; the last is partial
constexpr int kNt = 2;               // cache policy of the weight loads: nontemporal
constexpr int kDevScope = 16;        // cache policy of a load that must see other XCDs' stores (sc1)
constexpr int kSpinLimit = 1 << 21;
constexpr int kChunk = 4;            // tickets a workgroup draws at once
// Counters sit on lines of their own: device-scope adds to one line are served
// one after another, 11.4 ns each (measured; to different lines they overlap).
constexpr int kFlagStride = 32;
static_assert(kHRow <= kActBytes, "a down row fits the activation part");
static_assert(kWaves * kRing * kStageBytes <= 160 * 1024, "LDS");

enum { kGateUp = 0, kDown = 1, kSum = 2, kNone = 3 };

struct LayerArgs {
  const uint8_t *xd, *xs;
  const uint8_t *w1, *w3, *w2;
  int D, I, T, k;
  const int4* gt;
  const int4* rows;
  const int32_t* slot_row;
  const float* w;
  int32_t* head;
  uint32_t* flags;  // gate/up units done per tile ([rows]), then down units done per feature group ([D / 32])
  uint8_t* h;       // [rows][hstride] digits and scales of h, stage by stage
  int hstride;
  float* y;         // [rows][D]
  float* out;       // [T, D]
};

// A unit of work. row: first row of the tile (gate/up) or the row (down); rows:
// its rows; tile: gate/up tile; toks: its tokens, a byte each.
struct Unit {
  int kind, fg, expert, row, rows, tile, toks;
};

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ void store_dev(uint8_t* p, uint2 v) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), (uint64_t)v.y << 32 | v.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_dev(float* p, f32x4_t v) {
  uint8_t* q = reinterpret_cast<uint8_t*>(p);
  store_dev(q, make_uint2(__float_as_uint(v[0]), __float_as_uint(v[1])));
  store_dev(q + 8, make_uint2(__float_as_uint(v[2]), __float_as_uint(v[3])));
}

// Sums of one 16-row group: codes of four rounds (block 4 rnd + g of row rho) times the staged digits.
struct BOperand {
  u32x4_t q[4][2];  // per round: positions 16 g .. of the round's first and second 64
  uint32_t scale;   // byte rnd: scale of block 4 rnd + g
};
template <int kRnd>
__device__ __forceinline__ f32x4_t mfma_round(const uint32_t (&a)[4], uint32_t sa, const BOperand& b, f32x4_t c) {
  const i32x8_t av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const u32x4_t lo = b.q[kRnd][0], hi = b.q[kRnd][1];
  const i32x8_t bv = {(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 0, 0, (int)sa, kRnd, (int)b.scale);
}

// Both 16-row groups of a stage in LDS at `st`.  A block starts at byte sh of
// its first dword: sh = g in a whole stage; (rho * width + block) * 17 % 4 in
// the last, shorter one (kTail), whose blocks from `width` on count as zeros.
template <bool kTail>
__device__ __forceinline__ void stage_sums(const uint8_t* st, int rho, int g, int width, const BOperand& b, f32x4_t& c0,
                                           f32x4_t& c1) {
  uint32_t d[2][4][5];
  uint32_t sh[4];
#pragma unroll
  for (int rnd = 0; rnd < 4; ++rnd) {
    int at;
    if constexpr (kTail) {
      at = (rho * width + min(4 * rnd + g, width - 1)) * 17;
      sh[rnd] = (uint32_t)at & 3u;
      at >>= 2;
    } else {
      at = rho * kRowDw + 17 * rnd + 4 * g;
      sh[rnd] = (uint32_t)g;
    }
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int j = 0; j < 5; ++j) d[mi][rnd][j] = reinterpret_cast<const uint32_t*>(st + mi * kMatBytes)[at + j];
  }
  auto round = [&](auto rc) __attribute__((always_inline)) {
    constexpr int rnd = decltype(rc)::value;
    const uint32_t sel = 0x04030201u + 0x01010101u * sh[rnd];
    uint32_t a[2][4], sa[2];
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
#pragma unroll
      for (int i = 0; i < 4; ++i) a[mi][i] = __builtin_amdgcn_perm(d[mi][rnd][i + 1], d[mi][rnd][i], sel);
      sa[mi] = d[mi][rnd][0] >> (8 * sh[rnd]);  // byte 0 counts
      if (kTail && 4 * rnd + g >= width) {
        a[mi][0] = a[mi][1] = a[mi][2] = a[mi][3] = 0u;
        sa[mi] = 127u;
      }
    }
    c0 = mfma_round<rnd>(a[0], sa[0], b, c0);
    c1 = mfma_round<rnd>(a[1], sa[1], b, c1);
  };
  round(std::integral_constant<int, 0>{});
  round(std::integral_constant<int, 1>{});
  round(std::integral_constant<int, 2>{});
  round(std::integral_constant<int, 3>{});
}

__global__ __launch_bounds__(kWaves * 64, 1) void layer_main_kernel(LayerArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves][kRing][kStageBytes];
  __shared__ int fifo[kWaves][4][4];  // units in the ring: kind | late << 1 | fg << 2, row | rows << 16, tile
  __shared__ unsigned long long s_pool;

  const int lane = threadIdx.x & 63;
  const int wave = uni(threadIdx.x >> 6);
  const int rho = lane & 15, g = lane >> 4;
  const int nrows = a.T * a.k;
  const int nfg = a.I >> 5, nfu = a.D >> 5;
  const int n_gt = *as_const(a.head);
  const int n_gu = n_gt * nfg, n_dn = nrows * nfu;
  const int nst13 = (nfu + 15) >> 4, nst2 = (nfg + 15) >> 4;
  const float rcp_fg = 1.0f / (float)nfg, rcp_fu = 1.0f / (float)nfu;

  // n / d for 0 <= n < 2^23 by d's reciprocal r (one step off at most)
  auto div = [](int n, int d, float r) __attribute__((always_inline)) {
    int q = (int)((float)n * r);
    q -= q * d > n ? 1 : 0;
    q += (q + 1) * d <= n ? 1 : 0;
    return uni(q);
  };
  // Units of one expert are neighbours, its tiles (rows) fastest: what reads
  // the same weights runs at the same time, mostly in one workgroup.
  auto unit_of = [&](int t) __attribute__((always_inline)) -> Unit {
    if (t < n_gu) {
      const auto p = as_const(reinterpret_cast<const int32_t*>(a.gt));
      const int first = p[4 * div(t, nfg, rcp_fg) + 3];
      const int t0 = first & 0xFFFF, nt = first >> 16;
      const int in = t - t0 * nfg, fg = nt == 1 ? in : div(in, nt, 1.0f / (float)nt), i = t0 + in - fg * nt;
      return Unit{kGateUp, fg, p[4 * i], p[4 * i + 1] & 0xFFFF, p[4 * i + 1] >> 16, i, p[4 * i + 2]};
    }
    t -= n_gu;
    if (t < n_dn) {
      const auto q = as_const(reinterpret_cast<const int32_t*>(a.rows)) + 4 * div(t, nfu, rcp_fu);
      const int r0 = q[1] & 0xFFFF, nr = q[1] >> 16;
      const int in = t - r0 * nfu, fu = nr == 1 ? in : div(in, nr, 1.0f / (float)nr), r = in - fu * nr;
      return Unit{kDown, fu, q[0], r0 + r, 1, q[2] + r / kGuTileRows, 0};
    }
    t -= n_dn;
    return Unit{t < nfu ? kSum : kNone, t, 0, 0, 0, 0, 0};
  };

  // Tickets: the workgroup draws kChunk consecutive ones at a time and its
  // waves take them from LDS (low half: the next ticket, high half: how many
  // are left, or kRefill while the wave that found none fetches more; that wave
  // is running and waits only for its add to return).
  constexpr uint32_t kRefill = 0xFFFFFFFFu;
  if (threadIdx.x == 0) s_pool = 0ull;
  __syncthreads();
  auto claim = [&]() __attribute__((always_inline)) -> int {
    int v = 0;
    if (lane == 0)
      for (;;) {
        unsigned long long s = __hip_atomic_load(&s_pool, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        const uint32_t left = (uint32_t)(s >> 32);
        if (left == kRefill) {
          __builtin_amdgcn_s_sleep(1);
        } else if (left > 0) {
          if (__hip_atomic_compare_exchange_strong(&s_pool, &s, s + 1ull - (1ull << 32), __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                                   __HIP_MEMORY_SCOPE_WORKGROUP)) {
            v = (int)(uint32_t)s;
            break;
          }
        } else if (__hip_atomic_compare_exchange_strong(&s_pool, &s, (unsigned long long)kRefill << 32, __ATOMIC_RELAXED,
                                                        __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP)) {
          v = __hip_atomic_fetch_add(a.head + 1, kChunk, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(&s_pool, (unsigned long long)(kChunk - 1) << 32 | (uint32_t)(v + 1), __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_WORKGROUP);
          break;
        }
      }
    return uni(v);
  };

  // Weight load j takes chunks 64 j + lane of a stage: byte 16 c of the first
  // group's run up to chunk 271, then of the second group's, a group on in the
  // matrix.  The instruction's own offset counts for the LDS address, too, so
  // loads 0-3, 4-7 and 8 share a base each, and their lane offsets are
  const int lane16 = 16 * lane;  // 0-3
  int wofs4 = 0, wofs5 = 0;      // 4; 5-8
  const bool wlast = lane < kChunks - 64 * (kW - 1);
  static_assert(kW == 9, "three bases");

  // ---- issue side.  A stage is the same 512 columns of two neighbouring 16-row
  // groups of one matrix: of w2 (down), or of w1 and then of w3 (gate/up), where
  // the digits of x travel with w1.
  Unit iu = unit_of(claim());        // the unit being issued, or the next one
  Unit nu{kNone, 0, 0, 0, 0, 0, 0};  // the one after it, drawn while iu's loads go out
  bool drawn = true;
  const uint8_t *wb0 = nullptr, *wb1 = nullptr;  // the next stage's weights; gate/up: and those of the stage after it
  int grp2x = 0;             // bytes of a stage's two whole groups, less what lies before the stage
  int act0 = 0, act1 = 0;    // where the stage's activations are: rows of x, or (act0) the row of h
  int sco = 0;               // per lane: scale bytes of tile row `lane`
  int left = 0;              // stages of iu not yet issued (0: iu's loads have not begun)
  int inflight = 0, buf_i = 0, pushed = 0;
  bool bad = false;          // a bounded wait ran out
  bool all_done = false;     // every gate/up unit has been seen counted
  bool has_h = false;        // iu is a down unit whose h is complete

  auto seen = [&](int f) __attribute__((always_inline)) -> uint32_t {
    return (uint32_t)uni((int)__hip_atomic_load(a.flags + f * kFlagStride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  };
  // whether the down unit iu has its h (no waiting)
  auto look = [&]() __attribute__((always_inline)) -> bool {
    if (all_done) return true;
    if (seen(iu.tile) < (uint32_t)nfg) return false;
    bool all = true;  // whether that was the last look this wave needs
    for (int i = lane; i < n_gt; i += 64)
      all = all && __hip_atomic_load(a.flags + i * kFlagStride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= (uint32_t)nfg;
    all_done = __all(all);
    return true;
  };
  auto wait_for = [&](int f, uint32_t need) __attribute__((always_inline)) {
    int spins = 0;
    while (seen(f) < need) {
      __builtin_amdgcn_s_sleep(2);
      if (++spins > kSpinLimit) {
        bad = true;
        break;
      }
    }
  };
  auto prep = [&]() __attribute__((always_inline)) {
    // (plain values first, assigned once: the compiler would merge assignments
    // at the ends of two branches into one through memory)
    const bool gu = iu.kind == kGateUp;
    const int gb = (gu ? nfu : nfg) * 272;  // bytes of a 16-row group
    const size_t off = ((size_t)iu.expert * (size_t)(2 * (gu ? nfg : nfu)) + (size_t)(2 * iu.fg)) * (size_t)gb;
    const int t0 = iu.toks & 255, t1 = (iu.toks >> 8) & 255;
    wb0 = (gu ? a.w1 : a.w2) + off;
    wb1 = a.w3 + off;
    grp2x = 2 * gb;
    wofs5 = gb + lane16 - 256;
    wofs4 = lane < 16 ? 4096 + lane16 : wofs5;
    left = gu ? 2 * nst13 : nst2;
    act0 = gu ? t0 * nst13 * kXRow : iu.row * a.hstride;
    act1 = t1 * nst13 * kXRow;
    sco = (lane == 1 ? t1 : t0) * nst13 * 16;
    has_h = gu || look();
    int* const f = fifo[wave][pushed & 3];
    ++pushed;
    if (lane == 0) {
      f[0] = iu.kind | (has_h ? 0 : 2) | iu.fg << 2;
      f[1] = iu.row | iu.rows << 16;
      f[2] = iu.tile;
    }
    drawn = false;
  };
  auto load_h = [&](uint8_t* dst, int at) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)a.h, 0, nrows * a.hstride, 0x00020000);
    const int so = uni(at);
    const auto l = (__attribute__((address_space(3))) void*)(uintptr_t)dst;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 0, kDevScope);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 1024, kDevScope);
    if (lane < (kHRow - 2048) / 16) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 2048, kDevScope);
  };
  auto load_x = [&](uint8_t* dst, int at) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)a.xd, 0, a.T * nst13 * kXRow, 0x00020000);
    const int so = uni(at);
    const auto l = (__attribute__((address_space(3))) void*)(uintptr_t)dst;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 1024, 0);
  };
  // the next stage of iu into the ring
  auto issue = [&]() __attribute__((always_inline)) {
    uint8_t* const dst = &lds[wave][buf_i][0];
    uint8_t* const ad = dst + kWBytes;
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc((void*)wb0, 0, grp2x, 0x00020000);
    const auto l0 = (__attribute__((address_space(3))) void*)(uintptr_t)dst;
    const auto l4 = (__attribute__((address_space(3))) void*)(uintptr_t)(dst + 4096);
    const auto l8 = (__attribute__((address_space(3))) void*)(uintptr_t)(dst + 8192);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, l0, 16, lane16, 0, 0, kNt);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, l0, 16, lane16, 0, 1024, kNt);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, l0, 16, lane16, 0, 2048, kNt);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, l0, 16, lane16, 0, 3072, kNt);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, l4, 16, wofs4, 0, 0, kNt);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, l4, 16, wofs5, 0, 1024, kNt);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, l4, 16, wofs5, 0, 2048, kNt);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, l4, 16, wofs5, 0, 3072, kNt);
    if (wlast) __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, l8, 16, wofs5, 4096, 0, kNt);
    --left;
    if (iu.kind == kGateUp) {
      if (left & 1) {  // w1 (an even number of stages, w1 and w3 by turns)
        load_x(ad, act0);
        act0 += kXRow;
        if (iu.rows > 1) {
          load_x(ad + kXRowLds, act1);
          act1 += kXRow;
        }
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)a.xs, 0, a.T * nst13 * 16, 0x00020000);
        if (lane < iu.rows)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(uintptr_t)(ad + kActBytes), 16, sco, 0, 0, 0);
        sco += 16;
      }
      const uint8_t* const next = wb0 + kMatBytes;  // of the same matrix, two stages on
      wb0 = wb1;
      wb1 = next;
      grp2x -= (left & 1) ? 0 : kMatBytes;
    } else {
      if (has_h) load_h(ad, act0);
      act0 += kHRow;
      wb0 += kMatBytes;
      grp2x -= kMatBytes;
    }
    ++inflight;
    buf_i = buf_i == kRing - 1 ? 0 : buf_i + 1;
    if (left == 0) {
      if (!drawn) nu = unit_of(claim());
      drawn = true;
      iu = nu;
    }
  };

  // ---- publishing
  int pub[3] = {-1, -1, -1};  // flags of finished units, by age in stages
  auto publish = [&](int f) __attribute__((always_inline)) {
    if (f >= 0 && lane == 0)
      (void)__hip_atomic_fetch_add(a.flags + f * kFlagStride, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  auto flush = [&]() __attribute__((always_inline)) {
    wait_vm<0>();
#pragma unroll
    for (int i = 2; i >= 0; --i) {
      publish(pub[i]);
      pub[i] = -1;
    }
  };

  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  f32x4_t acc[2][2] = {{zero, zero}, {zero, zero}};  // [w1 / w3 by turns][16-row group]
  BOperand bop{};
  // LDS offsets of this lane's digits.  gate/up: column 4 r + p is digit p of
  // tile row r; columns from 8 on repeat.  down: columns 0 .. 4 are the digits.
  const int xp = rho & 3, hp = rho < kHDigits ? rho : 0;
  const int xoff0 = xp * kPlane + 16 * (g ^ xp), xoff1 = xp * kPlane + 16 * ((4 + g) ^ xp);
  const int hoff0 = hp * kPlane + 16 * (g ^ hp), hoff1 = hp * kPlane + 16 * ((4 + g) ^ hp);
  const uint32_t xsub = 0x05050505u * (uint32_t)xp, hsub = 0x05050505u * (uint32_t)hp;

  int buf_c = 0, popped = 0;
  for (;;) {
    while (inflight < kRing && iu.kind < kSum) {
      if (left == 0) prep();
      issue();
    }
    if (inflight == 0) break;
    // ---- one unit
    const int* const f = fifo[wave][popped & 3];
    ++popped;
    const int f0 = uni(f[0]), f1 = uni(f[1]), tile = uni(f[2]);
    const bool down = (f0 & 1) != 0;
    const int row = f1 & 0xFFFF, rows = f1 >> 16, fg = f0 >> 2;
    const int nst = down ? nst2 : 2 * nst13;
    const int cut = (down ? nfg : nfu) & 15;  // blocks of a last, shorter stage (0: none)
    // column rho's tile row (gate/up) and this lane's operand pieces
    const int r = !down && rows > 1 && (rho & 4) ? kXRowLds : 0;
    const int off0 = kWBytes + r + (down ? hoff0 : xoff0), off1 = kWBytes + r + (down ? hoff1 : xoff1);
    const int offs = kWBytes + 4 * g + (down ? kHDigits * kPlane : kActBytes + (r ? 16 : 0));
    const uint32_t sub = down ? hsub : xsub;
    if (f0 & 2) {
      // The unit's weights went ahead of its h.  Every earlier unit of this
      // wave is finished: count them, wait for the tile, load h for the stages
      // that are in the ring.
      flush();
      wait_for(tile, (uint32_t)nfg);
      for (int j = 0, b = buf_c; j < inflight && j < nst; ++j, b = b == kRing - 1 ? 0 : b + 1)
        load_h(&lds[wave][b][0] + kWBytes, row * a.hstride + j * kHRow);
      wait_vm<0>();
      if (left > 0 && inflight < nst) has_h = true;  // iu is this unit
    }
    for (int s = 0; s < nst; ++s) {
      if (inflight < kRing && iu.kind < kSum) {
        if (left == 0) prep();
        issue();
      }
      if (!drawn && left > 0) {  // with the ring full
        nu = unit_of(claim());
        drawn = true;
      }
      // The oldest stage has landed once only the loads of the newer ones are
      // out: their weights and, within a unit, activations (gate/up: of one of
      // two neighbouring stages; down: of both).  Fewer are assumed where that
      // is not sure, which waits for a little more.
      if (inflight < kRing) {
        if (inflight == 2) wait_vm<kW>();
        else wait_vm<0>();
      } else if (s + 2 >= nst) {
        wait_vm<2 * kW>();
      } else if (!down) {
        wait_vm<2 * kW + 3>();
      } else {
        wait_vm<2 * kW + 6>();
      }
      // a unit finished three stages ago: its stores are older than these loads
      publish(pub[2]);
      pub[2] = pub[1];
      pub[1] = pub[0];
      pub[0] = -1;
      const uint8_t* const st = &lds[wave][buf_c][0];
      buf_c = buf_c == kRing - 1 ? 0 : buf_c + 1;
      --inflight;
      const int width = cut != 0 && (down ? s == nst - 1 : s >= nst - 2) ? cut : 16;
      if (down || (s & 1) == 0) {
        bop.scale = *reinterpret_cast<const uint32_t*>(st + offs) - sub;
#pragma unroll
        for (int rnd = 0; rnd < 4; ++rnd) {
          bop.q[rnd][0] = *reinterpret_cast<const u32x4_t*>(st + off0 + 128 * rnd);
          bop.q[rnd][1] = *reinterpret_cast<const u32x4_t*>(st + off1 + 128 * rnd);
        }
        if (width < 16) {  // blocks past K: whatever the buffer holds
#pragma unroll
          for (int rnd = 0; rnd < 4; ++rnd) {
            if (4 * rnd + (g >> 1) >= width) bop.q[rnd][0] = u32x4_t{0u, 0u, 0u, 0u};
            if (4 * rnd + 2 + (g >> 1) >= width) bop.q[rnd][1] = u32x4_t{0u, 0u, 0u, 0u};
            if (4 * rnd + g >= width) bop.scale = (bop.scale & ~(0xFFu << (8 * rnd))) | 127u << (8 * rnd);
          }
        }
      }
      // acc[0] takes this stage; in a gate/up unit w1's and w3's sums take turns
      if (width == 16) stage_sums<false>(st, rho, g, width, bop, acc[0][0], acc[0][1]);
      else stage_sums<true>(st, rho, g, width, bop, acc[0][0], acc[0][1]);
      if (!down)
#pragma unroll
        for (int mi = 0; mi < 2; ++mi) {
          const f32x4_t o = acc[0][mi];
          acc[0][mi] = acc[1][mi];
          acc[1][mi] = o;
        }
    }

    // lane holds, in column rho, features 4 g + v of each 16-row group
    if (!down) {
      float gt[8], up[8];  // feature 4 g + v of group i at 2 v + i: the digits' byte order
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float c = acc[0][i][v], u = acc[1][i][v];
          gt[2 * v + i] = c + (__shfl_down(c, 1, 16) + (__shfl_down(c, 2, 16) + __shfl_down(c, 3, 16)));
          up[2 * v + i] = u + (__shfl_down(u, 1, 16) + (__shfl_down(u, 2, 16) + __shfl_down(u, 3, 16)));
        }
      float h[8];
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] = gt[i] / (1.0f + expf(-gt[i])) * up[i];
        top = max(top, __float_as_uint(h[i]) & 0x7FFFFFFFu);
      }
      top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
      if ((rho & 3) == 0 && (rho >> 2) < rows) {
        const uint32_t e = digit_exp(top);
        uint2 dg[kHDigits];
        digits8<kHDigits>(h, e, dg);
        uint8_t* const hb = a.h + (int64_t)(row + (rho >> 2)) * a.hstride + (fg >> 4) * kHRow;
#pragma unroll
        for (int p = 0; p < kHDigits; ++p) store_dev(hb + p * kPlane + digit_at(fg & 15, g, p), dg[p]);
        if (g == 0)
          __hip_atomic_store(hb + kHDigits * kPlane + 4 * (fg & 3) + ((fg & 15) >> 2), (uint8_t)(e - 3u), __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_AGENT);
      }
      pub[0] = tile;
    } else {
      f32x4_t sum[2];
#pragma unroll
      for (int mi = 0; mi < 2; ++mi)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float c = acc[0][mi][v];
          sum[mi][v] = c + (__shfl_down(c, 1, 16) + (__shfl_down(c, 2, 16) + (__shfl_down(c, 3, 16) + __shfl_down(c, 4, 16))));
        }
      if (rho == 0) {
        float* const y = a.y + (int64_t)row * a.D + 32 * fg + 4 * g;
        if (bad) sum[0][0] = sum[1][0] = __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int mi = 0; mi < 2; ++mi) store_dev(y + 16 * mi, sum[mi]);
      }
      pub[0] = nrows + fg;
    }
    acc[0][0] = acc[0][1] = acc[1][0] = acc[1][1] = zero;
  }

  // ---- nothing left to stream: count what is finished, then the sums
  flush();
  for (; iu.kind == kSum; iu = unit_of(claim())) {
    wait_for(nrows + iu.fg, (uint32_t)nrows);
    // eight lanes a token (four features each), eight tokens and 16 slots at a time
    const __amdgpu_buffer_rsrc_t yr = __builtin_amdgcn_make_buffer_rsrc((void*)a.y, 0, nrows * a.D * 4, 0x00020000);
    const uint32_t f4 = (uint32_t)(32 * iu.fg + 4 * (lane & 7));
    for (int t = lane >> 3; t < a.T; t += 8) {
      f32x4_t sum = zero;
      for (int j0 = 0; j0 < a.k; j0 += 16) {
        uint32_t at[16];
        float wt[16];
        u32x4_t v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int q = t * a.k + min(j0 + j, a.k - 1);
          at[j] = (uint32_t)a.slot_row[q] * (uint32_t)a.D * 4 + 4 * f4;
          wt[j] = a.w[q];
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __builtin_amdgcn_raw_buffer_load_b128(yr, at[j], 0, kDevScope);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j0 + j < a.k)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t bits = v[j][c];
              sum[c] = fmaf(wt[j], __uint_as_float(bits), sum[c]);
            }
      }
      if (bad) sum[0] = sum[1] = sum[2] = sum[3] = __uint_as_float(0x7FC00000u);
      *reinterpret_cast<f32x4_t*>(a.out + (int64_t)t * a.D + f4) = sum;
    }
  }
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct LayerWorkspace {
  size_t ids, w, xd, xs, gt, rows, slot_row, head, flags, h, y, total;
  int64_t n, n_flags;
  int hstride;
};
LayerWorkspace layer_layout(int64_t T, int32_t D, int32_t I, int32_t k) {
  LayerWorkspace l{};
  size_t off = 0;
  auto take = [&](size_t bytes) __attribute__((always_inline)) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  const int nst13 = (D / 32 + 15) / 16, nst2 = (I / 32 + 15) / 16;
  l.n = T * k;
  l.n_flags = (l.n + D / 32) * kFlagStride;
  l.hstride = (int)align256((size_t)nst2 * kHRow);
  l.ids = take(4 * l.n);
  l.w = take(4 * l.n);
  l.xd = take((size_t)T * nst13 * kXRow);
  l.xs = take((size_t)T * nst13 * 16);
  l.gt = take(16 * l.n);
  l.rows = take(16 * l.n);
  l.slot_row = take(4 * l.n);
  l.head = take(16);
  l.flags = take(4 * l.n_flags);
  l.h = take((size_t)l.n * l.hstride);
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
  p.xd = ws + l.xd;
  p.xs = ws + l.xs;
  p.gt = reinterpret_cast<int4*>(ws + l.gt);
  p.rows = reinterpret_cast<int4*>(ws + l.rows);
  p.slot_row = reinterpret_cast<int32_t*>(ws + l.slot_row);
  p.head = reinterpret_cast<int32_t*>(ws + l.head);
  p.flags = reinterpret_cast<uint32_t*>(ws + l.flags);
  p.n_flags = (int)l.n_flags;
  const unsigned blocks = 1 + (unsigned)((c.T * (c.D / 8) + kPlanThreads - 1) / kPlanThreads);
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
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;

  LayerArgs a{};
  a.xd = p.xd;
  a.xs = p.xs;
  a.w1 = c.w1;
  a.w3 = c.w3;
  a.w2 = c.w2;
  a.D = c.D;
  a.I = c.I;
  a.T = c.T;
  a.k = c.k;
  a.gt = p.gt;
  a.rows = p.rows;
  a.slot_row = p.slot_row;
  a.w = p.w;
  a.head = p.head;
  a.flags = p.flags;
  a.h = ws + l.h;
  a.hstride = l.hstride;
  a.y = reinterpret_cast<float*>(ws + l.y);
  a.out = c.out;
  const int64_t units = l.n * (c.I / 32 + c.D / 32) + c.D / 32;
  int64_t wgs = (units + kWaves - 1) / kWaves;
  const int cus = device_cu_count();
  if (wgs > cus) wgs = cus;
  hipLaunchKernelGGL(layer_main_kernel, dim3((unsigned)wgs), dim3(kWaves * 64), 0, s, a);
  return hipGetLastError();
}

}  // namespace k3moe
