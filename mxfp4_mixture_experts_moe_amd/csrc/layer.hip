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
// stay inside, so each column is as exact as an fp32 sum.  Both x and h take
// five digits: 2^-24 of the block's largest, half a step of fp32 there, and a
// bf16 element down to 2^-17 of it is held exactly.  (Four for x, 2^-19, exact
// down to 2^-12, cost the other elements of a block their bits where one stands
// far above them: with channels of 2^13 times the rest that no weight reads, the
// outputs were off by up to 18 times the bound of an fp32 sum.)
//
// With a few tokens the layer is a stream over the chosen experts' bytes
// (about 4 flop per byte and row): what costs time beside the stream are its
// interruptions, the drain and refill of the memory pipeline at every launch.
// The persistent kernel has none: a wave takes units of work from one list,
//   1. gate/up units: 32 features of w1 and of w3 for a tile of up to two rows
//      of one expert, over all of D;
//   2. down units: 32 features of w2 for a tile, over all of I;
//   3. sum units: 32 features of out for all tokens, slots in order;
// in that order, expert by expert, and streams their weights through a private
// ring of three LDS stages that runs on across units.
//
// Measured (graph replay; 16 experts a token, D = 3584, I = 3072): one token 64
// to 65 us, 281 MB of weights (plan 4.8, first weights in LDS 6 to 8 us into the
// second launch, the stream at 5.6 TB/s, sums 4); eight tokens 286 to 292 us, 1.58
// GB, 5.4-5.5 TB/s; the two calls moe_route_topk and moe_mxfp4_ffn take 64 to 72
// and 290 to 297 us there.
// 13 tokens, 5 of 61 experts, D = 1056, I = 736: 37 us against 186; one token,
// 2 of 8 experts, D = 128, I = 256: 17 us against 22.  What bounds it: the bytes
// with many tokens, plan, first loads and sums with one.
//
// Hand-over.  A down unit needs h from every gate/up unit of its tile, a sum unit
// every down unit of its features.  Units are taken by a global ticket (atomic
// add), and a wave works on its units in ticket order, so a unit waits only for
// units of lower tickets, each of which has been taken by a wave that is
// already running and that waits for still lower ones only: by induction every
// wait ends, however many of the workgroups are resident and whatever else
// the device runs.  (The wait loops are bounded all the same; a wait that ran
// out would give NaN outputs.)
//
// h carries its own "here": the plan fills it with bytes that no digit and no
// scale takes, a down unit's loads run ahead like any others, and when a
// stage's operand comes out of LDS each of its pieces (the eight bytes of one
// store) is compared with that filling; where one is missing the stage is
// loaded again.  That costs about 30 vector operations a stage and no trip to
// memory.  (Counting finished gate/up units per tile instead cost a look at the
// count for each down unit, which waits for every load before it, and a count
// that could go out only once the stores had completed, four stages after the
// unit: 85 us instead of 77 for one token of 16 experts, D = 3584, I = 3072.)
//
// Visibility.  Results (digits of h, y) are written with device-scope stores,
// which go through the XCD's L2.  h is read through the caches at first (the
// features of a down matrix read the same rows over and over), where a line may
// be older than the last store to it, but not older than the plan; the check
// finds that, and the second look is a device-scope load, which no stale line
// answers.  y is read with device-scope loads only, and counted per feature group
// (device-scope add, no return) once the stores have completed, that is once a
// later wait of the in-order vector-memory counter covers them: three stages
// later, at no cost, or at once where the ring runs dry.  On the reading side the
// wave's branch on the count holds the loads of y back; that the compiler does,
// too, takes a barrier to it (a relaxed load orders nothing).  Fences would write
// back or invalidate a whole L2 instead (57 ns each, measured, for every wave of
// the XCD in turn).
#include "mx_common.h"
#include "route_device.h"
#include "stream_device.h"

#include <type_traits>

namespace k3moe {
namespace {

constexpr int kDigits = 5;
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kPlane = 512;                // bytes of one digit of a row's stage
constexpr int kRow = kDigits * kPlane + 16;  // digits and scales of a (row, stage), of x and of h

// What h holds before it is written.  A digit is an integer or NaN, so no byte
// of it is e4m3's smallest subnormal; a scale byte is at most 252.
constexpr uint32_t kNoDigit = 0x01010101u, kNoScale = 0xFFFFFFFFu;

// Operand order.  A lane's 16 code bytes of a block hold elements j and j + 16 in
// byte j, so digit bytes go in the order 0, 16, 1, 17, ...: element e < 16 at
// byte 2e of the block's 32, element 16 + e at byte 2e + 1.  Of a stage's plane,
// the 16-byte chunk c (block c / 2) sits at chunk c with its low three bits
// xor the digit number, so that the columns of a read fall into different
// banks.  The 16 scale bytes of a stage are transposed, block 4 r + g at byte
// 4 g + r: a lane of group g reads its four rounds as one dword.
//
// Eight values in that order (those of quarter i of the block: elements 4i + t
// and 16 + 4i + t) as digits: out[p] = eight bytes.
__device__ __forceinline__ void digits8(const float (&v)[8], uint32_t e, uint2 (&out)[kDigits]) {
  const float unit = __uint_as_float((257u - e) << 23);  // 2^(130 - e): |v| * unit < 16
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = v[i] * unit;
#pragma unroll
  for (int p = 0; p < kDigits; ++p) {
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
constexpr int kTileRows = 2;

struct LayerPlan {
  const float* logits;
  const float* bias;
  const uint16_t* x;
  int T, D, E, k, normalize;
  float route_scale;
  int32_t* ids;    // [T, k]
  float* w;        // [T, k]
  uint8_t* xd;     // [T][stages][kRow] digits and scales of x
  int4* tiles;     // expert, first row | rows << 16, tokens of the rows (a byte each), the expert's tiles (first | count << 16)
  int32_t* slot_row;
  int32_t* head;   // [0] tiles, [1] next ticket
  uint32_t* flags;
  int n_flags;     // a multiple of 4
  u32x4_t* h;      // cleared to what no gate/up unit writes
  int n_h;         // its 16-byte pieces
  int x_wgs;       // workgroups that write x
};

template <int NPER>
__global__ __launch_bounds__(kPlanThreads) void layer_plan_kernel(LayerPlan p) {
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    // four lanes a block, eight elements each
    const int nb = p.D >> 5, nst = (nb + 15) >> 4;
    const int u = (int)(blockIdx.x - 1) * kPlanThreads + tid;
    if ((int)blockIdx.x > p.x_wgs) {
      const int c = u - p.x_wgs * kPlanThreads, f = c - p.n_h;
      const uint32_t v = c % (kRow / 16) == kRow / 16 - 1 ? kNoScale : kNoDigit;
      if (c < p.n_h) p.h[c] = u32x4_t{v, v, v, v};
      else if (f < p.n_flags / 4) reinterpret_cast<u32x4_t*>(p.flags)[f] = u32x4_t{0u, 0u, 0u, 0u};
      return;
    }
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
    uint2 d[kDigits];
    digits8(v, e, d);
    uint8_t* const piece = p.xd + ((int64_t)t * nst + (b >> 4)) * kRow;
#pragma unroll
    for (int q = 0; q < kDigits; ++q) *reinterpret_cast<uint2*>(piece + q * kPlane + digit_at(b & 15, i, q)) = d[q];
    if (i == 0) piece[kDigits * kPlane + 4 * (b & 3) + ((b & 15) >> 2)] = (uint8_t)(e - 3u);
    return;
  }
  __shared__ uint32_t s_mask[K3MOE_MAX_EXPERTS_FFN];  // tokens of each expert
  __shared__ uint32_t s_base[K3MOE_MAX_EXPERTS_FFN];  // first row
  __shared__ int s_ids[K3MOE_MAX_LAYER_TOKENS * K3MOE_MAX_TOPK];
  __shared__ int s_sum[kPlanThreads / 64][2];
  const int lane = tid & 63, wave = tid >> 6;
  const int n = p.T * p.k;
  __shared__ RouteScratch scratch[NPER > 0 ? kPlanThreads / 64 : 1];
  if (p.T == 1) {
    // one token: its experts are distinct, a tile each, in slot order; one wave
    // (4.8 us for 896 experts; grouped like more tokens 6.5)
    if (wave != 0) return;
    int id = 0;
    if constexpr (NPER > 0) {
      float g = 0.0f;
      route_token_reg<NPER>(p.logits, p.bias, p.E, p.k, p.normalize, p.route_scale, lane, scratch[0], id, g);
      if (lane < n) p.ids[lane] = id, p.w[lane] = g;
    } else {
      id = p.ids[min(lane, n - 1)];
    }
    if (lane < n) {
      p.tiles[lane] = make_int4(id, lane | 1 << 16, 0, lane | 1 << 16);
      p.slot_row[lane] = lane;
    }
    if (lane == 0) p.head[0] = n, p.head[1] = 0;
    return;
  }
  for (int e = tid; e < p.E; e += kPlanThreads) s_mask[e] = 0u;
  if constexpr (NPER > 0) {
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
    c[1] += (m + kTileRows - 1) / kTileRows;
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
    const int t0 = at[1], nt = (m + kTileRows - 1) / kTileRows;
    for (int r = 0; r < m; r += kTileRows) {
      int tk = 0;
      const int nr = min(kTileRows, m - r);
      for (int i = 0; i < nr; ++i) {
        tk |= __builtin_ctz(toks) << (8 * i);
        toks &= toks - 1u;
      }
      p.tiles[at[1]++] = make_int4(e, (at[0] + r) | nr << 16, tk, t0 | nt << 16);
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
constexpr int kRing = 3;             // weight stages per wave in LDS
constexpr int kMatBytes = 16 * 272;  // a 16-row group of a whole stage: 16 rows x 16 blocks of 17 bytes
constexpr int kChunks = 2 * 16 * 17; // 16-byte chunks of a stage's two groups
constexpr int kW = (kChunks + 63) / 64;  // weight loads per stage
// Every load is made by the whole wave (its last lanes may bring bytes that
// nothing reads): a branch on the lane inside the stage loop would make the
// compiler linearise the loop and carry the wave-uniform state in vector
// registers.
constexpr int kSlot = kW * 1024;       // bytes of a weight stage in LDS
constexpr int kRowLds = 3 * 1024 + 128;  // second row of a tile: other banks than the first
constexpr int kActBytes = kRowLds + 3 * 1024;  // a stage's activations
constexpr int kActBufs = 2;
constexpr int kNt = 2;               // cache policy of the weight loads: nontemporal
constexpr int kDevScope = 16;        // cache policy of loads and stores that other XCDs must agree on (sc1)
constexpr int kSpinLimit = 1 << 21;
constexpr int kChunk = 4;            // tickets a workgroup draws at once (2 or 8: 73 us instead of 70 for one token, D = 3584, I = 3072)
constexpr int kNoLane = INT32_MIN;  // buffer offset past every buffer: the lane's store is dropped
// Counters sit on lines of their own: device-scope adds to one line are served
// one after another, 11.4 ns each (measured; to different lines they overlap).
constexpr int kFlagStride = 32;
constexpr int kWaveLds = kRing * kSlot + kActBufs * kActBytes;
static_assert(kRow <= 3 * 1024, "activation buffers");
static_assert(kWaves * kWaveLds + 1024 <= 160 * 1024, "LDS");

enum { kGateUp = 0, kDown = 1, kSum = 2, kNone = 3 };

struct LayerArgs {
  const uint8_t* xd;
  const uint8_t *w1, *w3, *w2;
  int D, I, T, k;
  const int4* tiles;
  const int32_t* slot_row;
  const float* w;
  int32_t* head;
  uint32_t* flags;  // down units done per feature group ([D / 32])
  uint8_t* h;       // [rows][hstride] digits and scales of h, stage by stage
  int hstride;
  float* y;         // [rows][D]
  float* out;       // [T, D]
};

// A unit of work of a tile: its first row, its rows and their tokens (a byte each).
struct Unit {
  int kind, fg, expert, row, rows, toks;
};

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The first lane's atomics (no branch on the lane: the execution mask is set
// for the one instruction; the callers run with every lane on).
__device__ __forceinline__ void count_dev(uint32_t* p) {
  asm volatile("s_mov_b64 exec, 1\n\tglobal_atomic_add %0, %1, %2\n\ts_mov_b64 exec, -1" ::"v"(0), "v"(1), "s"(p) : "memory");
}
__device__ __forceinline__ int draw_dev(int32_t* p, int n) {
  int v;
  asm volatile(
      "s_mov_b64 exec, 1\n\tglobal_atomic_add %0, %1, %2, %3 sc0\n\ts_waitcnt vmcnt(0)\n\ts_mov_b64 exec, -1"
      : "=&v"(v)
      : "v"(0), "v"(n), "s"(p)
      : "memory");
  return uni(v);
}
// Compare and swap of an LDS word pair; returns what was there.
__device__ __forceinline__ uint64_t swap_lds(uint32_t at, uint64_t was, uint64_t now) {
  uint64_t v;
  asm volatile("s_mov_b64 exec, 1\n\tds_cmpst_rtn_b64 %0, %1, %2, %3\n\ts_waitcnt lgkmcnt(0)\n\ts_mov_b64 exec, -1"
               : "=&v"(v)
               : "v"(at), "v"(was), "v"(now)
               : "memory");
  return (uint64_t)(uint32_t)uni((int)(v >> 32)) << 32 | (uint32_t)uni((int)(uint32_t)v);
}

// Rounds.  A stage's 16 blocks go in four rounds of four, one block per lane
// group: group j takes block 4 ((rnd + j) % 4) + j in round rnd.  (The plain
// order 4 rnd + j would put the 64 reads of a dword, 68 dwords a row apart, into
// 16 of the 64 banks.)  The fp8 operand's registers 0-3 of lane group g belong
// to group g / 2's block (its half g % 2), registers 4-7 to group 2 + g / 2's.
__device__ __forceinline__ int round_block(int rnd, int j) { return 4 * ((rnd + j) & 3) + j; }

struct BOperand {
  u32x4_t q[4][2];  // per round: registers 0-3, 4-7
  uint32_t scale;   // byte rnd: scale of this lane group's block
};
template <int kRnd>
__device__ __forceinline__ f32x4_t mfma_round(const uint32_t (&a)[4], uint32_t sa, const BOperand& b, f32x4_t c) {
  const i32x8_t av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const u32x4_t lo = b.q[kRnd][0], hi = b.q[kRnd][1];
  const i32x8_t bv = {(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 0, 0, (int)sa, kRnd, (int)b.scale);
}

// Both 16-row groups of a stage: this lane's blocks of row rho as five dwords
// each.  A block starts at byte sh of its first dword: sh = g in a whole stage;
// (rho * width + block) * 17 % 4 in the last, shorter one (kTail), whose blocks
// from `width` on count as zeros.
template <bool kTail>
__device__ __forceinline__ int block_at(int rho, int g, int rnd, int width) {
  const int b = round_block(rnd, g);
  return kTail ? (rho * width + min(b, width - 1)) * 17 : rho * 272 + 17 * b;
}
// at[rnd]: the block's first dword in its group, in bytes.
__device__ __forceinline__ void stage_read(const uint8_t* st, const int (&at)[4], uint32_t (&d)[2][4][5]) {
#pragma unroll
  for (int rnd = 0; rnd < 4; ++rnd)
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int j = 0; j < 5; ++j) d[mi][rnd][j] = reinterpret_cast<const uint32_t*>(st + at[rnd] + mi * kMatBytes)[j];
}
template <bool kTail>
__device__ __forceinline__ void stage_sums(const uint32_t (&d)[2][4][5], int rho, int g, int width, const BOperand& b, f32x4_t& c0,
                                           f32x4_t& c1) {
  auto round = [&](auto rc) __attribute__((always_inline)) {
    constexpr int rnd = decltype(rc)::value;
    const uint32_t sh = kTail ? (uint32_t)block_at<kTail>(rho, g, rnd, width) & 3u : (uint32_t)g;
    const uint32_t sel = 0x04030201u + 0x01010101u * sh;
    uint32_t a[2][4], sa[2];
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
#pragma unroll
      for (int i = 0; i < 4; ++i) a[mi][i] = __builtin_amdgcn_perm(d[mi][rnd][i + 1], d[mi][rnd][i], sel);
      sa[mi] = d[mi][rnd][0] >> (8 * sh);  // byte 0 counts
      if constexpr (kTail) {
        const bool in = round_block(rnd, g) < width;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[mi][i] = in ? a[mi][i] : 0u;
        sa[mi] = in ? sa[mi] : 127u;
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

// v of lane + kN of the same 16 lanes (0 past their end).
template <int kN>
__device__ __forceinline__ float row_down(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x100 + kN, 0xF, 0xF, true));
}

// In column 5 r: a row's sum, its digits' columns smallest first.
__device__ __forceinline__ float digit_sum(float c) {
  return c + (row_down<1>(c) + (row_down<2>(c) + (row_down<3>(c) + row_down<4>(c))));
}

__global__ __launch_bounds__(kWaves * 64, 1) void layer_main_kernel(LayerArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves][kWaveLds];
  __shared__ int fifo[kWaves][4][2];  // units in the ring: kind | fg << 1, row | rows << 16
  __shared__ unsigned long long s_pool;

  const int lane = threadIdx.x & 63;
  const int wave = uni(threadIdx.x >> 6);
  const int rho = lane & 15, g = lane >> 4;
  uint8_t* const wl = &lds[wave][0];                   // weight stages
  uint8_t* const al = wl + kRing * kSlot;              // activation buffers
  const int nfg = a.I >> 5, nfu = a.D >> 5;
  const int n_tiles = *as_const(a.head);
  const int n_gu = n_tiles * nfg, n_dn = n_tiles * nfu;
  const int nst13 = (nfu + 15) >> 4, nst2 = (nfg + 15) >> 4;

  // n / d for 0 <= n < 2^23 by d's reciprocal (one step off at most)
  auto div = [](int n, int d) __attribute__((always_inline)) {
    int q = (int)((float)n * __builtin_amdgcn_rcpf((float)d));
    q -= q * d > n ? 1 : 0;
    q += (q + 1) * d <= n ? 1 : 0;
    return uni(q);
  };
  // Units of one expert are neighbours, its tiles fastest: what reads the same
  // weights runs at the same time, mostly in one workgroup.
  auto unit_of = [&](int t) __attribute__((always_inline)) -> Unit {
    const bool gu = t < n_gu;
    const int in = gu ? t : t - n_gu;
    if (in >= n_dn && !gu) return Unit{in - n_dn < nfu ? kSum : kNone, in - n_dn, 0, 0, 0, 0};
    const int per = gu ? nfg : nfu;  // units of a tile
    const auto p = as_const(reinterpret_cast<const int32_t*>(a.tiles));
    const int first = p[4 * div(in, per) + 3];
    const int t0 = first & 0xFFFF, nt = first >> 16;
    const int k = in - t0 * per, fg = nt == 1 ? k : div(k, nt), i = t0 + k - fg * nt;
    return Unit{gu ? kGateUp : kDown, fg, p[4 * i], p[4 * i + 1] & 0xFFFF, p[4 * i + 1] >> 16, p[4 * i + 2]};
  };

  // Tickets: the workgroup draws kChunk consecutive ones at a time and its
  // waves take them from LDS (low half: the next ticket, high half: how many
  // are left, or kRefill while the wave that found none fetches more; that wave
  // is running and waits only for its add to return).
  constexpr uint32_t kRefill = 0xFFFFFFFFu;
  if (wave == 0) {  // the first draw, while the other waves set out
    const int v = draw_dev(a.head + 1, kChunk);
    __hip_atomic_store(&s_pool, (unsigned long long)kChunk << 32 | (uint32_t)v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  }
  __syncthreads();
  const uint32_t pool = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)&s_pool;
  auto claim = [&]() __attribute__((always_inline)) -> int {
    for (;;) {
      const uint64_t s = __hip_atomic_load(&s_pool, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      const uint32_t next = (uint32_t)uni((int)(uint32_t)s), left = (uint32_t)uni((int)(s >> 32));
      if (left == kRefill) {
        __builtin_amdgcn_s_sleep(1);
        continue;
      }
      const uint64_t was = (uint64_t)left << 32 | next;
      const uint64_t now = left > 0 ? (uint64_t)(left - 1) << 32 | (next + 1) : (uint64_t)kRefill << 32;
      if (swap_lds(pool, was, now) != was) continue;
      if (left > 0) return (int)next;
      const int v = draw_dev(a.head + 1, kChunk);
      __hip_atomic_store(&s_pool, (unsigned long long)(kChunk - 1) << 32 | (uint32_t)(v + 1), __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_WORKGROUP);
      return v;
    }
  };

  // Weight load j takes chunks 64 j + lane of a stage: byte 16 c of the first
  // group's run up to chunk 271, then of the second group's, a group on in the
  // matrix.  The instruction's own offset counts for the LDS address, too, so
  // loads 0-3, 4-7 and 8 share a base each, and their lane offsets are
  const int lane16 = 16 * lane;  // 0-3
  const int rest16 = lane < (kRow - 2048) / 16 ? lane16 : kNoLane;  // a row of x, third load: nothing behind its scales
  int wofs4 = 0, wofs5 = 0, wofs8 = 0;  // 4; 5-7; 8 (half of it past the stage: not asked for)
  static_assert(kW == 9, "three bases");

  // ---- issue side.  A stage is the same 512 columns of two neighbouring 16-row
  // groups of one matrix: of w2 (down), or of w1 and then of w3 (gate/up), and
  // the digits that go with those columns, loaded with w1 for both.  Loads
  // return in order, so what a stage waits for must not have been asked for
  // behind what may still be on its way: weights go three stages ahead,
  // activations two, right before the weights of the stage after theirs.
  Unit iu{kNone, 0, 0, 0, 0, 0};  // the unit being issued
  Unit nu = iu;                      // the one after it
  bool drawn = false;                // whether nu has been drawn
  const uint8_t *wb0 = nullptr, *wb1 = nullptr;  // the next stage's weights; gate/up: and those of the stage after it
  int grp2x = 0;             // bytes of a stage's two whole groups, less what lies before the stage
  int act0 = 0, act1 = 0;    // where the stage's activations are, per row of the tile
  int left = 0;              // stages of iu not yet issued (0: nu's are the next)
  int want = 0;              // activations of the stage issued last: rows, + 4 for h; 0: none
  int want0 = 0, want1 = 0;  // where they are
  int inflight = 0, buf_i = 0, abuf_i = 0, pushed = 0;
  bool bad = false;          // a bounded wait ran out

  auto seen = [&](int f) __attribute__((always_inline)) -> uint32_t {
    return (uint32_t)uni((int)__hip_atomic_load(a.flags + f * kFlagStride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
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
    asm volatile("" ::: "memory");  // what the count stands for is loaded behind it
  };
  // (again: the caches' copy turned out to be old)
  auto load_h = [&](uint8_t* dst, int at, bool again) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc((void*)a.h, 0, a.T * a.k * a.hstride, 0x00020000);
    const int so = uni(at);
    const auto l = (__attribute__((address_space(3))) void*)(uintptr_t)dst;
    if (again) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 0, kDevScope);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 1024, kDevScope);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 2048, kDevScope);
    } else {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 1024, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 2048, 0);
    }
  };
  auto load_x = [&](uint8_t* dst, int at) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)a.xd, 0, a.T * nst13 * kRow, 0x00020000);
    const int so = uni(at);
    const auto l = (__attribute__((address_space(3))) void*)(uintptr_t)dst;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, lane16, so, 1024, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, rest16, so, 2048, 0);
  };
  auto prep = [&]() __attribute__((always_inline)) {
    iu = nu;
    drawn = false;
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
    wofs8 = lane < 32 ? wofs5 + 4096 : kNoLane;
    left = gu ? 2 * nst13 : nst2;
    act0 = gu ? t0 * nst13 * kRow : iu.row * a.hstride;
    act1 = gu ? t1 * nst13 * kRow : act0 + a.hstride;
    int* const f = fifo[wave][pushed & 3];
    ++pushed;
    f[0] = iu.kind | iu.fg << 1;  // (every lane, the same)
    f[1] = iu.row | iu.rows << 16;
  };
  // activations of the stage issued last, then the weights of iu's next one
  auto issue = [&]() __attribute__((always_inline)) {
    if (want != 0) {
      uint8_t* const ad = al + abuf_i * kActBytes;
      if (want & 4) {
        load_h(ad, want0, false);
        if (want & 2) load_h(ad + kRowLds, want1, false);
      } else {
        load_x(ad, want0);
        if (want & 2) load_x(ad + kRowLds, want1);
      }
      abuf_i ^= 1;
    }
    want = 0;
    if (left == 0) {
      if (nu.kind >= kSum) return;
      prep();
    }
    uint8_t* const dst = wl + buf_i * kSlot;
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc((void*)wb0, 0, uni(grp2x), 0x00020000);
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
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, l8, 16, wofs8, 0, 0, kNt);
    --left;
    const bool gu = iu.kind == kGateUp;
    const int odd = left & 1;  // gate/up: an even number of stages, w1 where an odd number is left
    want = gu ? (odd ? iu.rows : 0) : iu.rows + 4;
    want0 = act0;
    want1 = act1;
    const int on = gu && odd ? 0 : 1;  // columns go on after w3
    const uint8_t* const next = wb0 + kMatBytes;
    wb0 = gu ? wb1 : next;
    wb1 = next;
    grp2x -= on * kMatBytes;
    act0 += on * kRow;
    act1 += on * kRow;
    ++inflight;
    buf_i = buf_i == kRing - 1 ? 0 : buf_i + 1;
  };

  // ---- publishing
  // flags of finished units by age in stages; a unit's stores lie before the
  // weights asked for in the next stage, which the wait three stages on leaves out
  constexpr int kAges = 3;
  int pub[kAges] = {-1, -1, -1};
  auto publish = [&](int f) __attribute__((always_inline)) {
    if (f >= 0) count_dev(a.flags + f * kFlagStride);
  };
  auto flush = [&]() __attribute__((always_inline)) {
    wait_vm<0>();
#pragma unroll
    for (int i = kAges - 1; i >= 0; --i) {
      publish(pub[i]);
      pub[i] = -1;
    }
  };

  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  f32x4_t acc[2][2] = {{zero, zero}, {zero, zero}};  // [w1 / w3 by turns][16-row group]
  BOperand bop{};
  // LDS offsets of this lane's digits: column 5 r + p is digit p of tile row r;
  // columns from 10 on repeat.
  const int dr = rho >= kDigits && rho < 2 * kDigits ? 1 : 0, dp = rho < 2 * kDigits ? rho - dr * kDigits : 0;
  const int doff0 = dp * kPlane + 16 * (g ^ dp), doff1 = dp * kPlane + 16 * ((4 + g) ^ dp);
  int woff[4], rot0[4], rot1[4];  // per round: this lane's block, the rounds of its operand's two blocks
#pragma unroll
  for (int rnd = 0; rnd < 4; ++rnd) {
    woff[rnd] = block_at<false>(rho, g, rnd, 16) & ~3;
    rot0[rnd] = 128 * ((rnd + (g >> 1)) & 3);
    rot1[rnd] = 128 * ((rnd + 2 + (g >> 1)) & 3);
  }
  const uint32_t sub = 0x05050505u * (uint32_t)dp;

  // One pass of the loop takes a stage out of the ring and asks for a later one;
  // while the ring fills, it only asks.
  int buf_c = 0, abuf_c = 0, popped = 0;
  int s = 0, nst = 0;  // stage of the open unit, its stages
  // the open unit, and this lane's operand pieces in an activation buffer
  int row = 0, rows = 0, fg = 0, cut = 0, off0 = 0, off1 = 0, offs = 0;
  bool down = false;
  for (;;) {
    // the next ticket, once all stages of this unit have been asked for: one
    // drawn at the unit's start kept free waves from work that could begin (77
    // us instead of 70 for one token of 16 experts, D = 3584, I = 3072)
    if (!drawn && left == 0) {
      nu = unit_of(claim());
      drawn = true;
    }
    const bool eat = inflight == kRing || (left == 0 && nu.kind >= kSum && want == 0);
    bool shorter = false;
    uint32_t wd[2][4][5];
    if (eat) {
      if (inflight == 0) break;
      if (s == nst) {
        // ---- the next unit
        const int* const f = fifo[wave][popped & 3];
        ++popped;
        const int f0 = uni(f[0]), f1 = uni(f[1]);
        down = (f0 & 1) != 0;
        row = f1 & 0xFFFF;
        rows = f1 >> 16;
        fg = f0 >> 1;
        s = 0;
        nst = down ? nst2 : 2 * nst13;
        cut = (down ? nfg : nfu) & 15;  // blocks of a last, shorter stage (0: none)
        // column rho's tile row and digit
        const int r = rows == 1 ? 0 : dr * kRowLds;
        off0 = r + doff0;
        off1 = r + doff1;
        offs = r + kDigits * kPlane + 4 * g;
      }
      // The stage has landed once only loads asked for after its own are out:
      // the weights of two stages and, before the newer of them, activations of
      // the next stage (down; counted where that is this unit's).
      if (inflight < kRing) wait_vm<0>();
      else if (!down || s + 1 >= nst) wait_vm<2 * kW>();
      else if (rows == 1) wait_vm<2 * kW + 3>();
      else wait_vm<2 * kW + 6>();
      publish(pub[kAges - 1]);
#pragma unroll
      for (int i = kAges - 1; i > 0; --i) pub[i] = pub[i - 1];
      pub[0] = -1;
      const uint8_t* const st = wl + buf_c * kSlot;
      buf_c = buf_c == kRing - 1 ? 0 : buf_c + 1;
      --inflight;
      shorter = cut != 0 && (down ? s == nst - 1 : s >= nst - 2);
      if (down || (s & 1) == 0) {
        const uint8_t* const ad = al + abuf_c * kActBytes;
        abuf_c ^= 1;
        for (int spins = 0;;) {
          bop.scale = *reinterpret_cast<const uint32_t*>(ad + offs) - sub;
#pragma unroll
          for (int rnd = 0; rnd < 4; ++rnd) {
            bop.q[rnd][0] = *reinterpret_cast<const u32x4_t*>(ad + off0 + rot0[rnd]);
            bop.q[rnd][1] = *reinterpret_cast<const u32x4_t*>(ad + off1 + rot1[rnd]);
          }
          bop.scale = __builtin_amdgcn_alignbit(bop.scale, bop.scale, 8 * g);  // byte rnd: that of round_block's round
          if (shorter) {  // blocks past K: whatever the buffer holds
#pragma unroll
            for (int rnd = 0; rnd < 4; ++rnd) {
              const bool in0 = round_block(rnd, g >> 1) < cut, in1 = round_block(rnd, 2 + (g >> 1)) < cut;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                bop.q[rnd][0][c] = in0 ? bop.q[rnd][0][c] : 0u;
                bop.q[rnd][1][c] = in1 ? bop.q[rnd][1][c] : 0u;
              }
              const uint32_t byte = 0xFFu << (8 * rnd);
              bop.scale = round_block(rnd, g) < cut ? bop.scale : (bop.scale & ~byte) | (0x7F7F7F7Fu & byte);
            }
          }
          if (!down) break;
          // h is here once no piece of it (eight digits, a scale byte) is what
          // the plan left there; else this stage's and the next one's again
          uint32_t least = ~0u;  // 0 where a piece is missing
#pragma unroll
          for (int rnd = 0; rnd < 4; ++rnd)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              least = min(least, min(bop.q[rnd][i][0] ^ kNoDigit, bop.q[rnd][i][2] ^ kNoDigit));
          const uint32_t sc = bop.scale ^ (kNoScale - sub);
          const bool here = (least != 0u) & (((sc - 0x01010101u) & ~sc & 0x80808080u) == 0u);
          if (__all(here)) break;
          if (++spins > kSpinLimit) {
            bad = true;
            break;
          }
          const int at = row * a.hstride + s * kRow;
          for (int j = 0; j < 2; ++j) {
            uint8_t* const aj = al + (abuf_c ^ (1 - j)) * kActBytes;
            if (j == 1 && (inflight == 0 || s + 1 >= nst)) break;
            load_h(aj, at + j * kRow, true);
            if (rows > 1) load_h(aj + kRowLds, at + a.hstride + j * kRow, true);
          }
          __builtin_amdgcn_s_sleep(1);
          wait_vm<0>();
        }
      }
      if (!shorter) {
        stage_read(st, woff, wd);
      } else {
        int at[4];
#pragma unroll
        for (int rnd = 0; rnd < 4; ++rnd) at[rnd] = block_at<true>(rho, g, rnd, cut) & ~3;
        stage_read(st, at, wd);
      }
      // the stage is in registers: its buffers take later ones, whose loads run
      // beside the arithmetic below
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    issue();
    if (!eat) continue;
    // acc[0] takes this stage; in a gate/up unit w1's and w3's sums take turns
    if (!shorter) stage_sums<false>(wd, rho, g, 16, bop, acc[0][0], acc[0][1]);
    else stage_sums<true>(wd, rho, g, cut, bop, acc[0][0], acc[0][1]);
    if (!down)
#pragma unroll
      for (int mi = 0; mi < 2; ++mi) {
        const f32x4_t o = acc[0][mi];
        acc[0][mi] = acc[1][mi];
        acc[1][mi] = o;
      }
    if (++s < nst) continue;

    // lane holds, in column rho, features 4 g + v of each 16-row group; those of
    // columns 0 and 5 hold the tile's rows
    const bool second = (rho == kDigits) & (rows > 1), mine = (rho == 0) | second;
    if (!down) {
      float gt[8], up[8];  // feature 4 g + v of group i at 2 v + i: the digits' byte order
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          gt[2 * v + i] = digit_sum(acc[0][i][v]);
          up[2 * v + i] = digit_sum(acc[1][i][v]);
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
      const uint32_t e = digit_exp(top);
      uint2 dg[kDigits];
      digits8(h, e, dg);
      const __amdgpu_buffer_rsrc_t hb = __builtin_amdgcn_make_buffer_rsrc((void*)a.h, 0, a.T * a.k * a.hstride, 0x00020000);
      const int at = ((row + (second ? 1 : 0)) * a.hstride + (fg >> 4) * kRow) | (mine ? 0 : kNoLane);
      typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int p = 0; p < kDigits; ++p)
        __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{dg[p].x, dg[p].y}, hb, at + p * kPlane + digit_at(fg & 15, g, p), 0, kDevScope);
      __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(e - 3u), hb,
                                           (at + kDigits * kPlane + 4 * (fg & 3) + ((fg & 15) >> 2)) | (g == 0 ? 0 : kNoLane), 0, kDevScope);
    } else {
      f32x4_t sum[2];
#pragma unroll
      for (int mi = 0; mi < 2; ++mi)
#pragma unroll
        for (int v = 0; v < 4; ++v) sum[mi][v] = digit_sum(acc[0][mi][v]);
      const __amdgpu_buffer_rsrc_t yb = __builtin_amdgcn_make_buffer_rsrc((void*)a.y, 0, a.T * a.k * a.D * 4, 0x00020000);
      const int at = (4 * ((row + (second ? 1 : 0)) * a.D + 32 * fg + 4 * g)) | (mine ? 0 : kNoLane);
#pragma unroll
      for (int mi = 0; mi < 2; ++mi) {
        u32x4_t v;
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = bad ? 0x7FC00000u : __float_as_uint(sum[mi][c]);
        __builtin_amdgcn_raw_buffer_store_b128(v, yb, at + 64 * mi, 0, kDevScope);
      }
      pub[0] = fg;
    }
    acc[0][0] = acc[0][1] = acc[1][0] = acc[1][1] = zero;
  }

  // ---- nothing left to stream: count what is finished, then the sums
  flush();
  for (; nu.kind == kSum; nu = unit_of(claim())) {
    wait_for(nu.fg, (uint32_t)n_tiles);
    // eight lanes a token (four features each), eight tokens and 16 slots at a time
    const __amdgpu_buffer_rsrc_t yr = __builtin_amdgcn_make_buffer_rsrc((void*)a.y, 0, a.T * a.k * a.D * 4, 0x00020000);
    const uint32_t f4 = (uint32_t)(32 * nu.fg + 4 * (lane & 7));
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
  size_t ids, w, xd, tiles, slot_row, head, flags, h, y, total;
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
  l.n_flags = (int64_t)(D / 32) * kFlagStride;
  l.hstride = nst2 * kRow;
  l.ids = take(4 * l.n);
  l.w = take(4 * l.n);
  l.xd = take((size_t)T * nst13 * kRow);
  l.tiles = take(16 * l.n);
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
  p.tiles = reinterpret_cast<int4*>(ws + l.tiles);
  p.slot_row = reinterpret_cast<int32_t*>(ws + l.slot_row);
  p.head = reinterpret_cast<int32_t*>(ws + l.head);
  p.flags = reinterpret_cast<uint32_t*>(ws + l.flags);
  p.n_flags = (int)l.n_flags;
  p.h = reinterpret_cast<u32x4_t*>(ws + l.h);
  p.n_h = (int)(l.n * (l.hstride / 16));
  p.x_wgs = (int)((c.T * (c.D / 8) + kPlanThreads - 1) / kPlanThreads);
  const unsigned blocks = 1u + (unsigned)p.x_wgs + (unsigned)((p.n_h + p.n_flags / 4 + kPlanThreads - 1) / kPlanThreads);
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
  a.w1 = c.w1;
  a.w3 = c.w3;
  a.w2 = c.w2;
  a.D = c.D;
  a.I = c.I;
  a.T = c.T;
  a.k = c.k;
  a.tiles = p.tiles;
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
