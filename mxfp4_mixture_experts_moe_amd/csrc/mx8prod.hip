// Products of microscaled 8-bit rows and microscaled 4-bit weights: C[m][n] =
// sum_k A[m][k] * W[n][k], A in E4M3 codes, W in E2M1 codes, both with an E8M0
// scale per 32 elements, on CDNA4's block-scaled matrix instructions.
//
// Exact sums.  The instruction adds the products of a block in a fixed-point
// window: what lies more than 2^14 below the largest product is cut off
// (measured), and E4M3 spans 2^-9 .. 448.  So every fragment of A goes in twice,
// as
//   its elements of magnitude >= 2 (code bit 6 set) and zeros:  products are
//     multiples of 2^-3 up to 2688, 15 bits;
//   the others (< 2) and zeros:  multiples of 2^-10 up to 11.25, 14 bits;
// each of which the window holds whole, and only fp32 additions round.  The split
// is five register operations per four codes (a byte mask out of the sign bits of
// a shifted copy).  It makes the rate that of bf16 products, of which the
// library's reach 1.2 to 1.4 PFLOP/s at 8192^3.
//
// Operands.  For K slots of 32 (a block each), the 4-bit operand's lane group g
// holds block g, 16 bytes as they are stored; the 8-bit operand's holds 16 bytes
// of two blocks: with G lane groups, registers 0-3 bytes 16 (g % 2) .. of block g
// / 2, registers 4-7 the same of block G / 2 + g / 2, that is bytes 16 g and 16 G
// + 16 g of the G blocks.  The scale of a lane group is block g's for both.
//
// Two kernels, as for the 4-bit products (mxprod.hip): few rows, bound by the
// weight bytes, and tiles through a ring of LDS buffers.
#include "mx_common.h"
#include "mx_shape.h"

#include <math.h>

#include <type_traits>

namespace k3moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kFp8 = 0, kFp4 = 4;  // operand types of the scaled matrix instructions: E4M3, E2M1

__device__ __forceinline__ i32x8 operand4(mx_u32x4 q) {
  return i32x8{(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0};
}

// The elements of magnitude >= 2 of a lane's 32 codes, and the others.
struct Split {
  i32x8 hi, lo;
};
__device__ __forceinline__ Split split8(mx_u32x4 p, mx_u32x4 q) {
  Split s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = i < 4 ? p[i] : q[i - 4];
    // bit 6 of bytes 1 and 3 at bits 15 and 31 of x << 1, that of bytes 0 and 2 there of x << 9;
    // selectors 8 to 11 fill a byte with bit 15 or 31 of the second or the first operand
    const uint32_t mask = __builtin_amdgcn_perm(x << 1, x << 9, 0x0B090A08u);
    s.hi[i] = (int)(x & mask);
    s.lo[i] = (int)(x & ~mask);
  }
  return s;
}

// Scale bytes i .. i+3 of a row's nb, those past the end 127 (the value 1).
__device__ __forceinline__ uint32_t load_tail(const uint8_t* row, int i, int nb) {
  uint32_t v = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b = row[min(i + j, nb - 1)];
    v |= (i + j < nb ? b : 127u) << (8 * j);
  }
  return v;
}
__device__ __forceinline__ uint32_t load_u32(const uint8_t* p) {  // any alignment
  uint32_t v;
  __builtin_memcpy(&v, p, 4);
  return v;
}

template <bool kBf16>
__device__ __forceinline__ void store_out(void* out, int64_t i, float v) {
  if constexpr (kBf16)
    static_cast<__bf16*>(out)[i] = (__bf16)v;
  else
    static_cast<float*>(out)[i] = v;
}

// ---------------------------------------------------------------------------
// Few rows: as mx_few_kernel of mxprod.hip (16 weight rows a group, the waves of
// a group split K in pieces of 512, pieces asked for two turns ahead across
// rounds, partial sums through LDS), with the rows of A, 8 bits an element, in
// LDS.  Rows that do not fit together go in chunks, side by side in the grid.
// Bound by the weight bytes: 8 x 33792 x 7168 takes 31 us, 4.2 TB/s of the 5.1 that
// a copy reaches (27 us where the caches still hold part of the weights from the call
// before); of a small product (1 x 3584 x 7168: 6.2 to 7.3 us) by the chain of
// launch, two turns of loads and the sum over the waves; of one with many rows of A
// by their way into LDS, which every workgroup goes before its first product (16 x
// 7168 x 7168 11 to 13 us, of which the weights' bytes are 5.4).
constexpr int kFewWaves = 8;  // at most, per workgroup
constexpr int kFewRows = 16;
constexpr int kFewLds = 80 * 1024;     // two workgroups share a CU
constexpr int kFewLdsAll = 156 * 1024;  // one has it to itself
constexpr int kFewAhead = 2;            // pieces a wave asks for ahead

struct FewArgs {
  const uint8_t *a, *as, *w, *ws;
  int64_t M;
  int N, nb;       // nb = K / 32
  int rows;        // of A per chunk
  int kw, rw;      // waves per group, groups side by side
  int per;         // pieces per wave and group
  int arow, srow;  // LDS bytes per row of codes and of scales
  void* out;
};

// kTail: K is no multiple of 512, so a row's last piece is shorter (and
// scale rows are not 16-byte aligned).
template <bool kBf16, bool kTail, int kLds>
__global__ __launch_bounds__(kFewWaves * 64, kLds > kFewLds ? 2 : 4) void mx8_few_kernel(FewArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
  const int64_t m0 = (int64_t)blockIdx.y * a.rows;
  const int M = (int)(a.M - m0 < a.rows ? a.M - m0 : a.rows);
  uint8_t* const codes = lds;                // [M][arow]
  uint8_t* const scales = lds + M * a.arow;  // [M][srow]
  float* const red = reinterpret_cast<float*>(lds + ((M * (a.arow + a.srow) + 15) & ~15));  // [2][8 waves][256]
  const int tid = threadIdx.x, lane = tid & 63, threads = 64 * a.kw * a.rw;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rho = lane & 15, g = lane >> 4;
  const int nb = a.nb, nss = (nb + 15) >> 4;

  // this wave's turns: pieces s0, s0 + kw, ... of groups g0, g0 + step, ...
  const int gw = __builtin_amdgcn_readfirstlane(wave / a.kw), s0 = wave - gw * a.kw;
  const int ngroups = mx_groups(a.N, 16);
  struct Piece {
    mx_u32x4 q[4], sc;  // sc: 16 scale bytes; kTail: four dwords of one byte, this lane's blocks'
  };
  // Piece ss of group grp, without a branch (a wait for one piece must not become
  // one for all); what lies outside the matrix is outside the buffer: zeros.
  const uint32_t rowb = (uint32_t)nb * 16;
  auto load = [&](int g_, int s_, Piece& d) __attribute__((always_inline)) {
    const int grp = __builtin_amdgcn_readfirstlane(g_), ss = __builtin_amdgcn_readfirstlane(s_);
    const int rows = __builtin_amdgcn_readfirstlane(grp < ngroups && ss < nss ? min(a.N - 16 * grp, 16) : 0);
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc((void*)(a.w + (int64_t)grp * 16 * rowb), 0, rows * rowb, 0x00020000);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)(a.ws + (int64_t)grp * 16 * nb), 0, rows * nb, 0x00020000);
    const uint32_t b = (uint32_t)(16 * ss + g), row = (uint32_t)rho * nb;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = !kTail || b + 4 * i < (uint32_t)nb ? row + b + 4 * i : 0x0FFFFFFFu;
      d.q[i] = __builtin_amdgcn_raw_buffer_load_b128(rw, 16 * at, 0, 0);
      if constexpr (kTail) d.sc[i] = __builtin_amdgcn_raw_buffer_load_b8(rs, at, 0, 0);
    }
    if constexpr (!kTail) d.sc = __builtin_amdgcn_raw_buffer_load_b128(rs, row + 16 * ss, 0, 0);
  };
  const int gstep = (int)gridDim.x * a.rw;
  const int rounds = __builtin_amdgcn_readfirstlane(mx_few_rounds(a.N, a.rw, (int)gridDim.x));  // the same for every wave: the barriers below
  int grp = (int)blockIdx.x * a.rw + gw, done = 0;  // done: turns of this round behind us
  int lgrp = grp, ldone = 0;                        // the same of the next piece to ask for
  Piece ring[kFewAhead];
  auto ask = [&](Piece& d) __attribute__((always_inline)) {
    load(lgrp, s0 + ldone * a.kw, d);
    if (++ldone == a.per) ldone = 0, lgrp += gstep;
  };
  // A, in units of half a block, all rows' in order, kBatch a thread at a time.
  // The first batch is asked for ahead of the weights (loads return in order), one,
  // two, four or eight of them, so that few loads for nothing go before these: 1 x
  // 7168 x 3584 6.3 us, always with eight 7.3.
  constexpr int kBatch = 8;
  const int units = M * nb * 2, turns = __builtin_amdgcn_readfirstlane((units + threads - 1) / threads);
  mx_u32x4 raw[kBatch];
  uint32_t rsc[kBatch];
  int turn0 = 0;  // of the batch
  // row and unit of the row to place next, and what `threads` units further adds
  const int dm = __builtin_amdgcn_readfirstlane(threads / (2 * nb)), dr = threads - dm * 2 * nb;
  int pm = tid / (2 * nb), pr = tid - pm * 2 * nb;
  auto fetch = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if ((b & (b - 1)) == 0 && turn0 + b >= turns) break;
      const int64_t u = m0 * nb * 2 + min((turn0 + b) * threads + tid, units - 1);
      raw[b] = reinterpret_cast<const mx_u32x4*>(a.a)[u];
      rsc[b] = a.as[u >> 1];
    }
  };
  auto stage = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if ((b & (b - 1)) == 0 && turn0 + b >= turns) break;
      if (pm < M) {
        *reinterpret_cast<mx_u32x4*>(codes + pm * a.arow + 16 * pr) = raw[b];
        if ((pr & 1) == 0) scales[pm * a.srow + (pr >> 1)] = (uint8_t)rsc[b];
      }
      pm += dm;
      pr += dr;
      if (pr >= 2 * nb) pr -= 2 * nb, ++pm;
    }
    turn0 += kBatch;
  };
  fetch();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < kFewAhead; ++i) ask(ring[i]);
  asm volatile("" ::: "memory");
  stage();
  while (turn0 < turns) {
    fetch();
    stage();
  }
  if ((nb & 15) != 0)  // scales past K, up to the piece's end
    for (int i = tid; i < M * 16; i += threads)
      if (nb + (i & 15) < 16 * nss) scales[(i >> 4) * a.srow + nb + (i & 15)] = 127;
  __syncthreads();

  const int mrow = min(rho, M - 1);  // columns past M repeat the last row and are never stored
  const uint8_t* const brow = codes + mrow * a.arow;
  const uint8_t* const bsc = scales + mrow * a.srow;
  const int last = 32 * nb - 16;  // last half block of a row
  // byte g of four dwords, as one
  const uint32_t pick = 0x0c0c0400u + 0x0101u * (uint32_t)g;
  auto bytes = [&](mx_u32x4 v) __attribute__((always_inline)) -> uint32_t {
    return __builtin_amdgcn_perm(v[1], v[0], pick) | __builtin_amdgcn_perm(v[3], v[2], pick) << 16;
  };
  f32x4 acc0 = {0.f, 0.f, 0.f, 0.f}, acc1 = acc0;
  int par = 0, rd = 0;
  auto turn = [&](Piece& cur) __attribute__((always_inline)) {
    const int ss = s0 + done * a.kw, sl = min(ss, nss - 1);
    mx_u32x4 bs4;
#pragma unroll
    for (int i = 0; i < 4; ++i) bs4[i] = *reinterpret_cast<const uint32_t*>(bsc + 16 * sl + 4 * i);
    const uint32_t bs = bytes(bs4);
    uint32_t sc;
    if constexpr (kTail)
      sc = (cur.sc[0] | cur.sc[1] << 8) | (cur.sc[2] | cur.sc[3] << 8) << 16;
    else
      sc = bytes(cur.sc);
    // (past K the weights are zeros, and the last half block stands in for A's)
    auto step = [&](auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value;
      const int at = 512 * sl + 128 * i + 16 * g;
      const Split b = split8(*reinterpret_cast<const mx_u32x4*>(brow + min(at, last)),
                             *reinterpret_cast<const mx_u32x4*>(brow + min(at + 64, last)));
      acc0 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand4(cur.q[i]), b.hi, acc0, kFp4, kFp8, i, (int)sc, i, (int)bs);
      acc1 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand4(cur.q[i]), b.lo, acc1, kFp4, kFp8, i, (int)sc, i, (int)bs);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
    ask(cur);
    if (++done < a.per) return;
    done = 0;
    f32x4 sum = acc0 + acc1;
    acc0 = acc1 = f32x4{0.f, 0.f, 0.f, 0.f};
    if (a.kw > 1) {
      float* const slot = red + (par * kFewWaves + wave) * 256;
      *reinterpret_cast<f32x4*>(slot + 4 * lane) = sum;
      __syncthreads();
      if (s0 == 0)
        for (int i = 1; i < a.kw; ++i) sum += *reinterpret_cast<const f32x4*>(slot + 256 * i + 4 * lane);
      par ^= 1;
    }
    if (s0 == 0 && grp < ngroups && rho < M) {
      const int n = 16 * grp + 4 * g;
      const int64_t at = (m0 + rho) * a.N + n;
      if (n <= a.N - 4 && (a.N & 3) == 0) {
        if constexpr (kBf16) {
          typedef __bf16 b4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<b4*>(static_cast<__bf16*>(a.out) + at) = b4{(__bf16)sum[0], (__bf16)sum[1], (__bf16)sum[2], (__bf16)sum[3]};
        } else {
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = sum;
        }
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (n < a.N - v) store_out<kBf16>(a.out, at + v, sum[v]);
      }
    }
    grp += gstep;
    ++rd;
  };
  for (;;) {
#pragma unroll
    for (int i = 0; i < kFewAhead; ++i) {
      turn(ring[i]);
      if (rd >= rounds) return;
    }
  }
}

// ---------------------------------------------------------------------------
// Tiles.  A workgroup owns a BM x BN tile of C; kWm x kWn waves share it, and kSplit
// such sets of waves take the steps of K (128: four blocks, 128 bytes of a row of
// A, 64 of W) in turn, each with sums of its own that are added at the end.  A
// stage is kSplit steps; stages go through a ring of kRing LDS buffers filled by
// direct global -> LDS loads.  Instruction kk (0, 1) of a step takes its blocks 2
// kk and 2 kk + 1.  The 16-byte chunks of an LDS row are permuted by the row so
// that the lanes of a read touch every bank once.
//
// A wave's matrix instructions of one half step run while the operands of the
// next are read and split; the barrier of a stage stands between its two halves,
// when all of it has been read into registers: its buffer is free from there on,
// and the next stage, whose loads the wave has waited for, is there.
//
// Bound, where tiles fill the CUs, by the matrix instructions and the register
// work of the split beside them: 4096 x 7168 x 7168 239 to 266 us by session and data,
// 1.6 to 1.76 PFLOP/s (twice that of products of 8 bits, each going in twice).  That
// is a card at work: after idling its first 20 calls take 313, where a library
// product of 8192^3 in bf16 takes 900 us and then 775.  Where they do not, half of a stage is
// matrix instructions and the rest the way of its 16 or 24 KB into LDS, the barrier
// and the reads behind it: 128 x 7168 x 7168 16.0 us.
//   kStaged (K a multiple of 512): scales, 16 bytes (four steps) of every row, go
//     through LDS, too, one load per wave and four steps;
//   else each lane loads the four scale bytes of its rows for every step, which
//     are not aligned, half a stage ahead.
constexpr int kXcds = 8;

struct TileArgs {
  const uint8_t *a, *as, *w, *ws;
  int M, N, nb;
  void* out;
};

template <int N_>
__device__ __forceinline__ void wait_vm() {
  static_assert(N_ >= 0 && N_ < 64, "vmcnt is 6 bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N_) : "memory");
}
// Barrier of the ring: this wave's LDS reads are done (the buffer they read is
// refilled after it) and its loads of the next stage's buffer have landed.
__device__ __forceinline__ void ring_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <int BM, int BN, int kWm, int kWn, int kSplit, int kRing, bool kStaged, bool kBf16>
__global__ __launch_bounds__(kWm * kWn * kSplit * 64) void mx8_tile_kernel(TileArgs t) {
  constexpr int kSet = kWm * kWn, kWaves = kSet * kSplit;
  constexpr int kTm = BM / (32 * kWm), kTn = BN / (32 * kWn);  // 32-row operand tiles per wave
  constexpr int kBN = (BN + 16 * kSet - 1) / (16 * kSet) * (16 * kSet);  // rows of W in LDS: as many for every wave
  constexpr int kADw = BM * 32, kStepDw = kADw + kBN * 16;  // dwords of a step's rows of A; and of W behind them
  constexpr int kStageDw = kSplit * kStepDw;
  constexpr int kLoadsA = kSplit * BM / (8 * kWaves), kLoadsW = kSplit * kBN / (16 * kWaves), kLoads = kLoadsA + kLoadsW;  // 1 KB each, per wave and stage
  constexpr int kGroup = 4 / kSplit;  // stages that a load of scales lasts
  static_assert((kRing == 2 || kRing == 4) && kSplit <= 2 && kGroup >= kRing - 2, "scales land with the stage that they are for");
  // one array per buffer, so that the compiler sees that a read of one buffer
  // does not depend on the loads in flight into the others
  __shared__ __attribute__((aligned(256))) uint32_t l0[kStageDw], l1[kStageDw], l2[kRing > 2 ? kStageDw : 1],
      l3[kRing > 3 ? kStageDw : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ks = wave / kSet, wm = wave % kSet / kWn, wn = wave % kWn;
  const int r32 = lane & 31, h = lane >> 5;

  // Tile order: the ids an XCD gets (id % 8) are a contiguous run of the
  // logical order, which walks groups of four tile rows column by column.
  const int mt = mx_groups(t.M, BM), nt = mx_groups(t.N, BN);
  const int64_t total = (int64_t)mt * nt;
  int64_t id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (id >= total) return;
  {
    const int64_t q = total / kXcds, r = total % kXcds, x = id % kXcds, j = id / kXcds;
    id = x * q + (x < r ? x : r) + j;
  }
  constexpr int kGm = 4;
  const int64_t grp = id / ((int64_t)kGm * nt), in = id - grp * kGm * nt;
  const int gm = mt - (int)grp * kGm < kGm ? mt - (int)grp * kGm : kGm;
  const int64_t m0 = (grp * kGm + in % gm) * BM;
  const int n0 = (int)(in / gm) * BN;

  const int nb = t.nb;
  const uint32_t arowb = (uint32_t)nb * 32, wrowb = (uint32_t)nb * 16;
  const int mrows = t.M - m0 < BM ? (int)(t.M - m0) : BM;
  const int nrows = t.N - n0 < BN ? t.N - n0 : BN;
  const int nsteps = (nb + 3) >> 2, nstages = (nsteps + kSplit - 1) / kSplit;

  // position of 16-byte chunk c in LDS row r
  auto place_a = [](int c, int r) { return c ^ ((r >> 1) & 7); };
  auto place_w = [](int c, int r) { return c ^ ((r >> 2) & 3); };
  // loads: wave w fills the (w % kSet)-th part of the rows of step w / kSet of a stage
  const int arow0 = wave % kSet * (BM / kSet), wrow0 = wave % kSet * (kBN / kSet);
  uint32_t aoff[kLoadsA], woff[kLoadsW];
#pragma unroll
  for (int j = 0; j < kLoadsA; ++j) {
    const int r = arow0 + 8 * j + lane / 8;
    aoff[j] = (uint32_t)min(r, mrows - 1) * arowb + 16 * place_a(lane % 8, r);
  }
#pragma unroll
  for (int j = 0; j < kLoadsW; ++j) {
    const int r = wrow0 + 16 * j + lane / 4;
    woff[j] = r < BN ? (uint32_t)min(r, nrows - 1) * wrowb + 16 * place_w(lane % 4, r) : 0x80000000u;  // (outside)
  }
  // (steps past K are outside the buffers: zeros that cost no traffic)
  auto issue = [&](int stage, uint32_t* buf, auto fromc, auto toc) {  // the loads from .. to - 1 of a wave's
    constexpr int from = decltype(fromc)::value, to = decltype(toc)::value;
    const int step = stage * kSplit + ks;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)(t.a + m0 * arowb), 0, step < nsteps ? (int)(mrows * arowb) : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc((void*)(t.w + (int64_t)n0 * wrowb), 0, step < nsteps ? (int)(nrows * wrowb) : 0, 0x00020000);
    uint32_t* const da = buf + ks * kStepDw + arow0 * 32;
    uint32_t* const dw = buf + ks * kStepDw + kADw + wrow0 * 16;
    const int sa = __builtin_amdgcn_readfirstlane(128 * step), sw = __builtin_amdgcn_readfirstlane(64 * step);
#pragma unroll
    for (int j = 0; j < kLoadsA; ++j) {
      if (j < from || j >= to) continue;
      const uint32_t vo = aoff[j];  // (an array element passed straight makes the host pass drop the kernel's launch stub)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, da + 256 * j, 16, vo, sa, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kLoadsW; ++j) {
      if (kLoadsA + j < from || kLoadsA + j >= to) continue;
      const uint32_t vo = woff[j];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, dw + 256 * j, 16, vo, sw, 0, 0);
    }
  };

  // Scales.  kStaged: 16 bytes (four steps) of each of the tile's rows through LDS
  constexpr int kScaleA = (BM + 63) / 64, kScaleLoads = kScaleA + (BN + 63) / 64;  // of 64 rows; one per wave (some twice where there are more waves)
  static_assert(kScaleLoads <= kWaves, "every wave does one load of scales");
  __shared__ __attribute__((aligned(256))) uint32_t lsc0[kStaged ? kScaleLoads * 256 : 1], lsc1[kStaged ? kScaleLoads * 256 : 1];  // (of even groups, of odd ones)
  const int sload = wave % kScaleLoads;
  const bool s_a = sload < kScaleA;
  const int slrows = s_a ? mrows : nrows;
  const __amdgpu_buffer_rsrc_t rsc = __builtin_amdgcn_make_buffer_rsrc((void*)(s_a ? t.as + m0 * nb : t.ws + (int64_t)n0 * nb), 0, slrows * nb, 0x00020000);
  const int svoff = min((s_a ? sload : sload - kScaleA) * 64 + lane, slrows - 1) * nb;
  auto issue_scales = [&](int group, uint32_t* buf) {
    uint32_t* dst = buf + sload * 256;
    const int so = 16 * min(group, (nb >> 4) - 1), vo = svoff;  // (past the last: that again, not used)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsc, dst, 16, vo, so, 0, 0);
  };
  // !kStaged: from memory, those past K 127 (the value 1)
  const uint8_t *ap[kTm], *wp[kTn];
  if constexpr (!kStaged) {
#pragma unroll
    for (int i = 0; i < kTm; ++i) ap[i] = t.as + (m0 + min(wm * (BM / kWm) + 32 * i + r32, mrows - 1)) * nb;
#pragma unroll
    for (int i = 0; i < kTn; ++i) wp[i] = t.ws + (int64_t)(n0 + min(wn * (BN / kWn) + 32 * i + r32, nrows - 1)) * nb;
  }
  auto scale4 = [&](const uint8_t* row, int step) -> uint32_t {
    if (nb < 4) return load_tail(row, min(4 * step, nb), nb);
    const int o = min(4 * step, nb - 4);
    return load_u32(row + o);
  };
  // ... and what of the four bytes is past K
  auto trim = [&](uint32_t v, int step) -> uint32_t {
    const int k = nb < 4 ? 0 : min(max(4 * step - (nb - 4), 0), 4);
    return (uint32_t)(((uint64_t)0x7F7F7F7Fu << 32 | v) >> (8 * k));
  };
  // The raw scales of this wave's step of a stage; bytes 0 and 2 of own_bytes() are
  // those of this lane half's blocks of both instructions.
  uint32_t na[kTm], nw[kTn];
  auto read_scales = [&](int stage, const uint32_t* buf) {
    const int step = stage * kSplit + ks;
    if constexpr (kStaged) {
      const uint32_t* const l = buf + (step & 3);
#pragma unroll
      for (int i = 0; i < kTm; ++i) na[i] = l[4 * (wm * (BM / kWm) + 32 * i + r32)];
#pragma unroll
      for (int i = 0; i < kTn; ++i) nw[i] = l[4 * (kScaleA * 64 + wn * (BN / kWn) + 32 * i + r32)];
    } else {
#pragma unroll
      for (int i = 0; i < kTm; ++i) na[i] = scale4(ap[i], step);
#pragma unroll
      for (int i = 0; i < kTn; ++i) nw[i] = scale4(wp[i], step);
    }
  };
  uint32_t ca[kTm], cw[kTn];
  auto take_scales = [&](int stage) {
    auto own_bytes = [&](uint32_t v) {
      if constexpr (!kStaged) v = trim(v, stage * kSplit + ks);
      return h ? v >> 8 : v;
    };
#pragma unroll
    for (int i = 0; i < kTm; ++i) ca[i] = own_bytes(na[i]);
#pragma unroll
    for (int i = 0; i < kTn; ++i) cw[i] = own_bytes(nw[i]);
  };

  f32x16 acc[kTm][kTn];
#pragma unroll
  for (int i = 0; i < kTm; ++i)
#pragma unroll
    for (int j = 0; j < kTn; ++j) acc[i][j] = f32x16{};

  const uint32_t arow = (uint32_t)ks * kStepDw * 4 + (uint32_t)(wm * (BM / kWm) + r32) * 128;
  const uint32_t wrow = (uint32_t)(ks * kStepDw + kADw) * 4 + (uint32_t)(wn * (BN / kWn) + r32) * 64;
  // Operands of an instruction: as read, and split.
  struct Raw {
    mx_u32x4 a[kTm][2], w[kTn];
  };
  auto read = [&](const uint32_t* buf, auto kc, Raw& n) {
    constexpr int kk = decltype(kc)::value;
    const uint8_t* const l = reinterpret_cast<const uint8_t*>(buf);
    const uint32_t p0 = 16u * (uint32_t)place_a(4 * kk + h, r32), p1 = 16u * (uint32_t)place_a(4 * kk + 2 + h, r32);
    const uint32_t pw = 16u * (uint32_t)place_w(2 * kk + h, r32);
#pragma unroll
    for (int i = 0; i < kTm; ++i) {
      n.a[i][0] = *reinterpret_cast<const mx_u32x4*>(l + arow + 32 * 128 * i + p0);
      n.a[i][1] = *reinterpret_cast<const mx_u32x4*>(l + arow + 32 * 128 * i + p1);
    }
#pragma unroll
    for (int i = 0; i < kTn; ++i) n.w[i] = *reinterpret_cast<const mx_u32x4*>(l + wrow + 32 * 64 * i + pw);
  };
  Split fa[kTm];
  mx_u32x4 fw[kTn];
  // (blocks of A past K are zeroed: what lies there is another row's, or NaN codes)
  auto split = [&](Raw& n, auto kc, int stage) {
    constexpr int kk = decltype(kc)::value;
    if constexpr (!kStaged) {
      const int b0 = 4 * (stage * kSplit + ks) + 2 * kk;
#pragma unroll
      for (int i = 0; i < kTm; ++i) {
        if (b0 >= nb) n.a[i][0] = mx_u32x4{0u, 0u, 0u, 0u};
        if (b0 + 1 >= nb) n.a[i][1] = mx_u32x4{0u, 0u, 0u, 0u};
      }
    }
#pragma unroll
    for (int i = 0; i < kTm; ++i) fa[i] = split8(n.a[i][0], n.a[i][1]);
#pragma unroll
    for (int i = 0; i < kTn; ++i) fw[i] = n.w[i];
  };
  auto multiply = [&](auto kc) {
    constexpr int kk = decltype(kc)::value;
#pragma unroll
    for (int i = 0; i < kTm; ++i)
#pragma unroll
      for (int j = 0; j < kTn; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[i].hi, operand4(fw[j]), acc[i][j], kFp8, kFp4, 2 * kk, (int)ca[i], 2 * kk, (int)cw[j]);
#pragma unroll
    for (int i = 0; i < kTm; ++i)
#pragma unroll
      for (int j = 0; j < kTn; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[i].lo, operand4(fw[j]), acc[i][j], kFp8, kFp4, 2 * kk, (int)ca[i], 2 * kk, (int)cw[j]);
  };
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;

  // Order of a half step: the reads, which the compiler would move to where their
  // data are used, then the matrix instructions with the register work, and the
  // loads of a later stage, between them (two first, while the reads are on their
  // way). 128 x 7168 x 7168 took 19.4 us without any order, 18.5 with it; 2048 x 7168
  // x 7168 in tiles of 128 149 and 146; waves of more than 192 columns have no
  // registers for it (spills).
  auto ordered = [&](auto loads, auto&& reads, auto&& work) {
    reads();
    if constexpr (kTm == 1 && kTn < 7) {
      __builtin_amdgcn_sched_barrier(0);
      work();
      constexpr int kMfma = 2 * kTm * kTn, kGaps = kMfma > 2 ? kMfma - 2 : 1;
      __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
#pragma unroll
      for (int i = 0; i < kGaps; ++i) {
        if (decltype(loads)::value) __builtin_amdgcn_sched_group_barrier(0x10, (decltype(loads)::value + kGaps - 1) / kGaps, 0);
        __builtin_amdgcn_sched_group_barrier(0x2, (42 * kTm + kGaps - 1) / kGaps, 0);
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      }
      // (split before the branch that may follow, not behind it)
      if constexpr (kStaged) {
#pragma unroll
        for (int i = 0; i < kTm; ++i) asm volatile("" : "+v"(fa[i].hi), "+v"(fa[i].lo));
      }
      __builtin_amdgcn_sched_barrier(0);
    } else {
      work();
    }
  };

  // One stage, of which the first half step's operands are in registers: `prev`,
  // `cur`, `next` the buffers of the stage before, its own and the next stage's.
  // Between the halves the loads in flight are those of kRing - 1 stages (and up to
  // two sets of scales); the oldest has to have landed, and with it, or before it,
  // the scales that it needs.
  // Into a buffer that is free goes the stage kRing further.  With four buffers its
  // loads are spread over this half step and the first of the next stage: the waves
  // would wait for each other's, all at once behind the barrier (128 x 7168 x 7168
  // 17.7 us, spread 16.0).  With two, they have to go out at once, and other
  // workgroups fill the CU meanwhile (1003 x 4000 x 4128 40 us, spread 48).
  using L0 = std::integral_constant<int, 0>;
  using LA = std::integral_constant<int, kLoads>;
  constexpr bool kSpread = kRing > 2;
  using LH = std::integral_constant<int, (kSpread ? kLoads / 2 : kLoads)>;  // those of a stage's second half
  using LR = std::integral_constant<int, kLoads - LH::value>;               // and of the first half of the next
  auto stage = [&](auto uc, int q, uint32_t* prev, uint32_t* cur, uint32_t* next) {
    constexpr int u = decltype(uc)::value;  // q modulo 4 where groups have two stages, 8 where they have four
    constexpr bool kLast = u % kGroup == kGroup - 1;  // of its group
    uint32_t* const sn = (u + 1) / kGroup % 2 ? lsc1 : lsc0;  // the next stage's scales
    Raw n;
    ordered(LR{}, [&] { read(cur, C1{}, n); }, [&] { multiply(C0{}); split(n, C1{}, q); issue(q - 1 + kRing, prev, LH{}, LA{}); });
    wait_vm<(kRing - 2) * kLoads>();
    ring_barrier();
    read_scales(q + 1, sn);
    asm volatile("" ::: "memory");
    if constexpr (kStaged && kLast) issue_scales((q + 1) / kGroup + 1, sn == lsc0 ? lsc1 : lsc0);
    asm volatile("" ::: "memory");
    if constexpr (kSpread) {
      ordered(LH{}, [&] { read(next, C0{}, n); }, [&] { multiply(C1{}); split(n, C0{}, q + 1); issue(q + kRing, cur, L0{}, LH{}); });
    } else {
      issue(q + kRing, cur, L0{}, LA{});
      asm volatile("" ::: "memory");  // the loads go out before the reads below
      ordered(L0{}, [&] { read(next, C0{}, n); }, [&] { multiply(C1{}); split(n, C0{}, q + 1); });
    }
    take_scales(q + 1);
  };
  {
    Raw n;
    if constexpr (kStaged) issue_scales(0, lsc0);
    asm volatile("" ::: "memory");
    issue(0, l0, L0{}, LA{});
    if constexpr (kStaged) issue_scales(1, lsc1);
    if constexpr (kRing == 2) issue(1, l1, L0{}, LH{});
    if constexpr (kRing > 2) {
      issue(1, l1, L0{}, LA{});
      issue(2, l2, L0{}, LA{});
      issue(3, l3, L0{}, LH{});
    }
    wait_vm<(kRing - 2) * kLoads + LH::value>();
    ring_barrier();
    read_scales(0, lsc0);
    take_scales(0);
    read(l0, C0{}, n);
    split(n, C0{}, 0);
  }
  // (kStaged: whole groups; no branch around a load, so that their number in flight is known everywhere)
  auto four = [&](auto uc, int q) {  // stages q .. q + 3, false: that was all
    constexpr int u = decltype(uc)::value;
    stage(std::integral_constant<int, u>{}, q, kRing > 2 ? l3 : l1, l0, l1);
    if (!kStaged && q + 1 == nstages) return false;
    stage(std::integral_constant<int, u + 1>{}, q + 1, l0, l1, kRing > 2 ? l2 : l0);
    if ((!kStaged || kGroup == 2) && q + 2 == nstages) return false;
    stage(std::integral_constant<int, u + 2>{}, q + 2, l1, kRing > 2 ? l2 : l0, kRing > 2 ? l3 : l1);
    if (!kStaged && q + 3 == nstages) return false;
    stage(std::integral_constant<int, u + 3>{}, q + 3, kRing > 2 ? l2 : l0, kRing > 2 ? l3 : l1, l0);
    return q + 4 < nstages;
  };
  if constexpr (kStaged && kGroup == 4) {
    for (int q = 0;; q += 8)
      if (!four(C0{}, q) || !four(std::integral_constant<int, 4>{}, q + 4)) break;
  } else {
    for (int q = 0; four(C0{}, q); q += 4) {}
  }
  wait_vm<0>();  // no load into LDS outlives the workgroup

  if constexpr (kSplit == 2) {  // the second set's sums through LDS, an operand tile at a time
    static_assert(kSet * 1024 <= kStageDw, "the set's operand tiles fit a buffer");
    float* const red = reinterpret_cast<float*>(l0) + (wave % kSet) * 1024 + 4 * lane;
#pragma unroll
    for (int i = 0; i < kTm; ++i)
#pragma unroll
      for (int j = 0; j < kTn; ++j) {
        __syncthreads();
        if (ks == 1)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            *reinterpret_cast<f32x4*>(red + 256 * v) = f32x4{acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]};
        __syncthreads();
        if (ks == 0)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(red + 256 * v);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][4 * v + e] += x[e];
          }
      }
    if (ks == 1) return;
  }

  // lane holds column n = lane % 32, rows 8 * (v / 4) + 4 * h + v % 4; a whole tile's need no test each
  const int64_t o0 = (m0 + wm * (BM / kWm) + 4 * h) * (int64_t)t.N + n0 + wn * (BN / kWn) + r32;
  auto store = [&](auto whole) {
#pragma unroll
    for (int i = 0; i < kTm; ++i)
#pragma unroll
      for (int j = 0; j < kTn; ++j) {
        if (!decltype(whole)::value && wn * (BN / kWn) + 32 * j + r32 >= nrows) continue;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int m = 32 * i + 8 * (v >> 2) + (v & 3);
          if (decltype(whole)::value || wm * (BM / kWm) + 4 * h + m < mrows) store_out<kBf16>(t.out, o0 + (int64_t)m * t.N + 32 * j, acc[i][j][v]);
        }
      }
  };
  if (mrows == BM && nrows == BN) store(std::true_type{});
  else store(std::false_type{});
}

// LDS bytes of the few-row kernel: rows of codes (an odd number of 16-byte
// units, so 16 rows start in different banks), rows of scales, partial sums.
int few_arow(int nb) { return 32 * nb + 16; }
int few_srow(int nb) { return (nb + 15) / 16 * 16 + 4; }
constexpr int kFewRed = 12 + 2 * kFewWaves * 256 * (int)sizeof(float);
// Rows of A that fit `lds` bytes together, at most 16.
int few_rows(int nb, int lds) {
  const int r = (lds - kFewRed) / (few_arow(nb) + few_srow(nb));
  return r < kFewRows ? r : kFewRows;
}

template <int BM, int BN, int kWm, int kWn, int kSplit, int kRing>
hipError_t launch_tiles(const TileArgs& t, bool bf16, hipStream_t s) {
  const MxTileGrid g = mx_tile_grid(t.M, t.N, BM, BN);
  const dim3 grid(g.x, g.y), block(kWm * kWn * kSplit * 64);
  auto go = [&](auto st, auto b) {
    hipLaunchKernelGGL((mx8_tile_kernel<BM, BN, kWm, kWn, kSplit, kRing, decltype(st)::value, decltype(b)::value>), grid, block, 0, s, t);
  };
  const bool staged = t.nb % 16 == 0;
  if (staged && bf16) go(std::true_type{}, std::true_type{});
  else if (staged) go(std::true_type{}, std::false_type{});
  else if constexpr (BN <= 192) {  // (the registers of the largest do not hold the scales of ragged rows, too)
    if (bf16) go(std::false_type{}, std::true_type{});
    else go(std::false_type{}, std::false_type{});
  }
  return hipGetLastError();
}

// most: rows of a chunk; half: two workgroups share a CU.
hipError_t launch_few(FewArgs a, int most, bool half, bool bf16, hipStream_t s) {
  const int64_t chunks = (a.M + most - 1) / most;
  a.rows = (int)((a.M + chunks - 1) / chunks);
  a.arow = few_arow(a.nb);
  a.srow = few_srow(a.nb);
  const int cus = device_cu_count();
  const dim3 grid((unsigned)mx_few_grid(a.N, a.rw, half ? cus : (cus + 1) / 2).wgs, (unsigned)chunks), block((unsigned)(64 * a.kw * a.rw));
  auto go = [&](auto b, auto t, auto l) {
    hipLaunchKernelGGL((mx8_few_kernel<decltype(b)::value, decltype(t)::value, decltype(l)::value>), grid, block, 0, s, a);
  };
  using Half = std::integral_constant<int, kFewLds>;
  using All = std::integral_constant<int, kFewLdsAll>;
  const bool tail = a.nb % 16 != 0;
  auto type = [&](auto t, auto l) {
    if (bf16) go(std::true_type{}, t, l);
    else go(std::false_type{}, t, l);
  };
  if (half && tail) type(std::true_type{}, Half{});
  else if (half) type(std::false_type{}, Half{});
  else if (tail) type(std::true_type{}, All{});
  else type(std::false_type{}, All{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx8_product(const uint8_t* a, const uint8_t* as, const uint8_t* w, const uint8_t* ws, int64_t M,
                              int N, int K, bool out_bf16, void* out, hipStream_t s) {
  const int nb = K / 32, nss = (nb + 15) / 16;
  FewArgs f{};
  f.a = a;
  f.as = as;
  f.w = w;
  f.ws = ws;
  f.M = M;
  f.N = N;
  f.nb = nb;
  f.per = (nss + kFewWaves - 1) / kFewWaves;
  f.kw = (nss + f.per - 1) / f.per;
  f.rw = kFewWaves / f.kw;
  f.out = out;
  const int fit = few_rows(nb, kFewLds), fit_all = few_rows(nb, kFewLdsAll);
  const int64_t cus = device_cu_count(), wgs = (mx_groups(N, 16) + f.rw - 1) / f.rw;
  // Few rows: two workgroups a CU where all rows fit half of its LDS, else one, in
  // chunks of what fits, of a long K as mx8_few_in_chunks says.  More, of K beyond a tile's first few stages: where the
  // workgroups of every chunk are resident at once (32 x 3584 x 3584 7.9 us, in
  // tiles 11; 64 x 2048 x 2048 5.3, not 7.6; 77 x 1003 x 4128 11, not 17; 256 x 2048 x
  // 512 5.1 by either; beyond, 64 x 3584 x 3584 12.7 instead of 10.3 in tiles).
  if (M <= kFewRows && fit >= M) return launch_few(f, kFewRows, true, out_bf16, s);
  if (M <= kFewRows && fit_all >= 1 && mx8_few_in_chunks(N, (M + fit_all - 1) / fit_all, nb % 16 == 0, (int)cus))
    return launch_few(f, fit_all, false, out_bf16, s);
  if (K > 512 && fit >= 4 && (M + fit - 1) / fit * wgs <= 2 * cus) return launch_few(f, fit, true, out_bf16, s);
  const TileArgs t{a, as, w, ws, (int)M, N, nb, out};
  // Tiles of 32 x 64 where there are no more of them than CUs (a stage brings a CU 16
  // KB, not the 24 of 64 x 64; 32 x 7168 x 3584 8.0 us, not 10.5, 64 x 7168 x 3584
  // 8.1, not 9.4), and for up to 32 rows (with two buffers, as there are several on
  // a CU: 32 x 33792 x 7168 30 to 34 us, 39 in tiles of 64).
  const int64_t narrow = mx_tile_grid(t.M, N, 32, 64).total;
  if (narrow <= cus) return launch_tiles<32, 64, 1, 2, 2, 4>(t, out_bf16, s);
  if (M <= 32) return launch_tiles<32, 64, 1, 2, 2, 2>(t, out_bf16, s);
  // Else the tile whose workgroups take the least time together, n of them on the CU
  // with the most, in units of 17.7 us at K = 7168 (of a short K more is a tile's fixed
  // part, which the costs do not hold: 1536 x 7168 x 512 with f32 output takes 17.3 us in
  // tiles of 256 x 192, in those of 128 15.8).  One tile of 64 with a CU to
  // itself takes 16 us (with four buffers, which leave no room for another); where
  // there are more of those, two buffers: 2 take 27 us, 3 39, 4 50, 9 115, 14 178;
  // one of 128 41 (2 69 to 82, 3 108, 4 141, 7 264).  One of 256 rows, one to a CU:
  // 97 to 101 us with 192 columns, 107 to 120 with 224, 120 to 134 with 256 (more
  // where all CUs have one), so that 7168 columns are 28, 32 or 38 tiles and the
  // last round is full or not: 1536 x 7168 x 7168 101 us by 192 (128: 108, 224: 109),
  // 4096 x 7168 x 7168 239 by 224 (256: 251, 128: 264), 4096 x 4096 x 7168 134 by 256
  // (128: 152, 192: 194).  384 x 7168 x 7168 takes tiles of 64 (39 us, not 42), 512 x
  // 7168 x 7168 of 128 (41, not 51).
  auto each = [&](int rows, int columns) { return (double)((mx_tile_grid(t.M, N, rows, columns).total + cus - 1) / cus); };
  const double n64 = each(64, 64), n128 = each(128, 128);
  const double c64 = n64 <= 1 ? 0.9 : 0.15 + 0.7 * n64, c128 = n128 <= 1 ? 2.3 : 0.2 + 2.05 * n128;
  const double c192 = 5.65 * each(256, 192), c224 = 6.7 * each(256, 224), c256 = 7.2 * each(256, 256);
  const double small = c64 < c128 ? c64 : c128;
  if (nb % 16 == 0 && c224 < small && c224 <= c192 && c224 <= c256) return launch_tiles<256, 224, 8, 1, 1, 2>(t, out_bf16, s);
  if (nb % 16 == 0 && c256 < small && c256 <= c192) return launch_tiles<256, 256, 8, 1, 1, 2>(t, out_bf16, s);
  if (c192 < small) return launch_tiles<256, 192, 8, 1, 1, 2>(t, out_bf16, s);
  if (c128 < c64) return launch_tiles<128, 128, 4, 1, 1, 2>(t, out_bf16, s);
  if (n64 <= 1) return launch_tiles<64, 64, 2, 1, 2, 4>(t, out_bf16, s);
  return launch_tiles<64, 64, 2, 1, 2, 2>(t, out_bf16, s);
}

}  // namespace k3moe
