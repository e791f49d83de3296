// Products of microscaled 4-bit matrices: C[m][n] = sum_k A[m][k] * W[n][k], A
// and W given as packed E2M1 codes and E8M0 block scales (compressed-tensors
// layout), on CDNA4's block-scaled matrix instructions: one instruction takes
// 16 bytes (a block of 32 codes) and one scale byte of every operand row per
// lane, multiplies the 32 products of a block by both scales and sums in fp32.
//
// The instruction's own k order does not matter as long as both operands use
// the same one, so a lane always takes whole 16-byte blocks as they are
// stored, and a lane's blocks are chosen next to each other in memory.
//
// Two kernels:
//   few rows (M <= 16): the weights are read once, straight from memory into
//     the operand registers, with the rows of A (quantised on the way from
//     float rows by the linear layer) in LDS; bound by the weight bytes (8 x
//     33792 x 7168: 24 us, 5.4 TB/s; 1 x 3584 x 7168: 5.8 us, of which 3 are
//     the launch and the way of A through LDS);
//   tiles: square output tiles, both operands staged through a ring of LDS
//     buffers by direct global -> LDS loads.  Large products are bound by loads
//     and matrix instructions that overlap in part only (4096 x 4096 x 7168: 69
//     to 71 us, 3.4 PFLOP/s; 55 without the loads, 46 without the matrix
//     instructions; 4096 x 7168 x 7168: 114 us, the matrix cores busy 0.51 of the
//     CUs' time), small ones by load latency (128 x 7168 x 3584: 7.8-8.3 us).
#include "mx_common.h"
#include "mx_shape.h"

#include <type_traits>

namespace k3moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kFp4 = 4;  // operand type of the scaled matrix instructions: E2M1

__device__ __forceinline__ i32x8 operand(mx_u32x4 q) {
  return i32x8{(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0};
}

// Scale bytes at p (any alignment).
__device__ __forceinline__ uint2 load_u64(const uint8_t* p) {
  uint2 v;
  __builtin_memcpy(&v, p, 8);
  return v;
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

template <bool kBf16>
__device__ __forceinline__ void store_out(void* out, int64_t i, float v) {
  if constexpr (kBf16)
    static_cast<__bf16*>(out)[i] = (__bf16)v;
  else
    static_cast<float*>(out)[i] = v;
}

// ---------------------------------------------------------------------------
// Few rows.  A workgroup takes groups of 16 weight rows; the waves of a group
// split K in pieces of 512 (16 blocks: 256 bytes of every row), and lane (row
// rho, quarter g) of a wave loads blocks g, 4 + g, 8 + g and 12 + g of its row's
// piece (each load takes 64 bytes of a row in four lanes) and the piece's 16
// scale bytes, which feed four 16x16x128 instructions.  kw waves share a group,
// as many as give each the same number of pieces with at most eight waves;
// 8 / kw groups run side by side; the kw partial sums meet in LDS.  The
// workgroups are persistent, so rows of A are staged (and quantised) once each,
// and the pieces of the next two turns are on their way across rounds (three
// ahead: 23.9 us instead of 23.3 for 1 x 33792 x 7168).  A row's 128-byte lines
// are each met by two loads, so the loads carry no streaming hint: with it the
// lines came twice (31.8 us).  More
// than 16 rows of A (packed) go 16 at a time, side by side in the grid.
constexpr int kFewWaves = 8;  // at most, per workgroup
constexpr int kFewRows = 16;
constexpr int kFewLds = 80 * 1024;  // two workgroups share a CU
// The linear layer quantises rows in every workgroup up to this many elements,
// by a launch of its own beyond (about 3 us: 8 x 3584, 3.4 us more than the
// packed product in the kernel; 8 x 7168, 4.4; 4 x 7168, 0.9; 16 x 7168, 9).
constexpr int64_t kFewFused = 32768;
constexpr int kFewAhead = 2;  // pieces a wave asks for ahead

struct FewArgs {
  const uint8_t* x;  // float rows [M, K] (kX >= 0), or packed codes [M, K/2]
  const uint8_t* xs; // scales of packed rows
  const uint8_t* w;
  const uint8_t* ws;
  int64_t M;
  int N, nb;         // nb = K / 32
  int kw, rw;        // waves per group, groups side by side
  int per;           // pieces per wave and group
  int saturate;
  int arow, srow;    // LDS bytes per row of codes and of scales
  void* out;
};

// kTail: K is no multiple of 512, so a row's last piece is shorter (and
// scale rows are not 16-byte aligned).
template <int kX, bool kBf16, bool kTail>
__global__ __launch_bounds__(kFewWaves * 64, 4) void mx_few_kernel(FewArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kFewLds];
  const int64_t m0 = (int64_t)blockIdx.y * kFewRows;
  const int M = (int)(a.M - m0 < kFewRows ? a.M - m0 : kFewRows);
  uint8_t* const codes = lds;                    // [M][arow]
  uint8_t* const scales = lds + M * a.arow;      // [M][srow]
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
  // Piece ss of group grp, without a branch: one around the loads would make the
  // wait for a piece a wait for all that was asked for since.  What lies outside
  // (groups past the last, rows past N, pieces and blocks past K) is outside the
  // buffer: zeros that cost no traffic.
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
  int grp = (int)blockIdx.x * a.rw + gw, done = 0;   // done: turns of this round behind us
  int lgrp = grp, ldone = 0;                         // the same of the next piece to ask for
  Piece ring[kFewAhead];
  auto ask = [&](Piece& d) __attribute__((always_inline)) {
    load(lgrp, s0 + ldone * a.kw, d);
    if (++ldone == a.per) ldone = 0, lgrp += gstep;
  };
  // A, a unit per thread and turn, kBatch turns at a time.  Float rows: units of
  // eight elements (four lanes hold a block), a row at a time, which spares a
  // division per unit; packed ones: blocks, all rows' in order.  The first batch
  // is asked for ahead of the weights (loads return in order), the rest behind
  // them.
  constexpr bool kFlat = kX < 0;
  constexpr int kBatch = kFlat || kX == K3MOE_DTYPE_F32 ? 4 : 8, kRaw = kX == K3MOE_DTYPE_F32 ? 2 : 1;
  const int rows = kFlat ? 1 : M, units = kFlat ? M * nb : 4 * nb;  // of a row
  const int turns = __builtin_amdgcn_readfirstlane((units + threads - 1) / threads);
  mx_u32x4 raw[kBatch][kRaw];
  uint32_t rsc[kBatch];
  int fm = 0, ft = 0, sm = 0, st = 0;  // row and turn to fetch and to stage next
  auto fetch = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int u = min(ft * threads + tid, kFlat ? units - 1 : units - 4 + (tid & 3));
      const int64_t at = kFlat ? m0 * nb + u : (m0 + min(fm, rows - 1)) * units + u;
#pragma unroll
      for (int h = 0; h < kRaw; ++h) raw[b][h] = reinterpret_cast<const mx_u32x4*>(a.x)[at * kRaw + h];
      if constexpr (kFlat) rsc[b] = a.xs[at];
      if (++ft == turns) ft = 0, ++fm;
    }
  };
  auto stage = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (sm >= rows) break;
      const int u = st * threads + tid;
      if constexpr (kFlat) {
        const int m = u / nb, r = u - m * nb;
        if (u < units) {
          *reinterpret_cast<mx_u32x4*>(codes + m * a.arow + 16 * r) = raw[b][0];
          scales[m * a.srow + r] = (uint8_t)rsc[b];
        }
      } else {
        uint32_t e;
        const uint32_t c = mx_quant8<kX>(raw[b], a.saturate != 0, e);
        if (u < units) {
          *reinterpret_cast<uint32_t*>(codes + sm * a.arow + 4 * u) = c;
          if ((tid & 3) == 0) scales[sm * a.srow + (u >> 2)] = (uint8_t)e;
        }
      }
      if (++st == turns) st = 0, ++sm;
    }
  };
  fetch();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < kFewAhead; ++i) ask(ring[i]);
  asm volatile("" ::: "memory");
  stage();
  while (sm < rows) {
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
  // byte g of four dwords, as one
  const uint32_t pick = 0x0c0c0400u + 0x0101u * (uint32_t)g;
  auto bytes = [&](mx_u32x4 v) __attribute__((always_inline)) -> uint32_t {
    return __builtin_amdgcn_perm(v[1], v[0], pick) | __builtin_amdgcn_perm(v[3], v[2], pick) << 16;
  };
  f32x4 acc0 = {0.f, 0.f, 0.f, 0.f}, acc1 = acc0;
  int par = 0, rd = 0;
  auto turn = [&](Piece& cur) __attribute__((always_inline)) {
    const int ss = s0 + done * a.kw, sl = min(ss, nss - 1);
    mx_u32x4 b[4], bs4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[i] = *reinterpret_cast<const mx_u32x4*>(brow + 16 * min(16 * sl + 4 * i + g, nb - 1));
      bs4[i] = *reinterpret_cast<const uint32_t*>(bsc + 16 * sl + 4 * i);
    }
    const uint32_t bs = bytes(bs4);
    uint32_t sc;
    if constexpr (kTail)
      sc = (cur.sc[0] | cur.sc[1] << 8) | (cur.sc[2] | cur.sc[3] << 8) << 16;
    else
      sc = bytes(cur.sc);
    acc0 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(cur.q[0]), operand(b[0]), acc0, kFp4, kFp4, 0, (int)sc, 0, (int)bs);
    acc1 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(cur.q[1]), operand(b[1]), acc1, kFp4, kFp4, 1, (int)sc, 1, (int)bs);
    acc0 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(cur.q[2]), operand(b[2]), acc0, kFp4, kFp4, 2, (int)sc, 2, (int)bs);
    acc1 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(cur.q[3]), operand(b[3]), acc1, kFp4, kFp4, 3, (int)sc, 3, (int)bs);
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
// Tiles.  A workgroup (2 x 2 waves, 4 x 2 for the larger tiles) owns a B x B
// tile of C; K goes in steps of 128 (four blocks: 64 bytes of every row), in
// stages of one or two steps, through a ring of LDS buffers filled by direct
// global -> LDS loads.  Lane (row r = lane % 32, half h) of a 32x32x64
// instruction kk of a step takes its block 2h + kk.  The 16-byte blocks of an
// LDS row are permuted by the row (place()), so that the 16-lane groups of a
// read touch every bank once (no conflicts counted).
//   kStaged (K a multiple of 512): stages of two steps, so a row's piece is a
//     whole 128-byte line (33 x 33792 x 7168: 28 us, with lines in two halves
//     31; 1024 x 7168 x 3584: 25 and 28), a ring of four, for the larger tiles
//     of two (128 KB, or 64 for two workgroups on a CU); scales, 16 bytes (four
//     steps) of every row, go through LDS, too, one load per wave and four steps.
//   else: stages of one step, a ring of four, and each lane loads eight scale
//     bytes (two steps) of its rows, which are not aligned.  That is a load of 32
//     lines for every operand tile and wave: 89 us instead of 71 for 4096 x 4096
//     x 7168.
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
// refilled after it) and its loads of the next step's buffer have landed.
__device__ __forceinline__ void ring_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <int B, int kWaves, bool kStaged, bool kBf16>
__global__ __launch_bounds__(kWaves * 64) void mx_tile_kernel(TileArgs t) {
  constexpr int kWm = kWaves / 2;         // waves along M; two along N
  constexpr int kTm = B / (32 * kWm), kTn = B / 64;  // 32-row operand tiles per wave
  constexpr int kS = kStaged ? 2 : 1;     // steps of a stage
  constexpr int kRow = 64 * kS;           // bytes of a row of a stage
  constexpr int kRing = kStaged && B >= 128 ? 2 : 4;
  constexpr int kStageDw = 2 * B * kRow / 4;  // B rows of A, B rows of W
  constexpr int kLoadRows = 1024 / kRow;  // of a 1 KB load
  constexpr int kLoads = 2 * B / (kLoadRows * kWaves);  // per wave and stage
  // one array per buffer, so that the compiler sees that a read of one buffer
  // does not depend on the loads in flight into the others
  __shared__ __attribute__((aligned(256))) uint32_t l0[kStageDw], l1[kStageDw], l2[kRing > 2 ? kStageDw : 1],
      l3[kRing > 2 ? kStageDw : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r32 = lane & 31, h = lane >> 5;

  // Tile order: the ids an XCD gets (id % 8) are a contiguous run of the
  // logical order, which walks groups of four tile rows column by column.
  const int mt = mx_groups(t.M, B), nt = mx_groups(t.N, B);
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
  const int64_t m0 = (grp * kGm + in % gm) * B;
  const int n0 = (int)(in / gm) * B;

  const int nb = t.nb;
  const uint32_t rowb = (uint32_t)nb * 16;
  const int mrows = t.M - m0 < B ? (int)(t.M - m0) : B;
  const int nrows = t.N - n0 < B ? t.N - n0 : B;
  const int nsteps = (nb + 3) >> 2;

  // loads: wave w fills LDS rows 2B / kWaves * w ..
  const bool from_a = wave < kWaves / 2;
  const int lrow0 = wave % (kWaves / 2) * (2 * B / kWaves);  // first row within A or W
  const uint8_t* const src = from_a ? t.a + m0 * rowb : t.w + (int64_t)n0 * rowb;
  const int srows = from_a ? mrows : nrows;
  // position of 16-byte chunk c in LDS row r
  auto place = [](int c, int r) { return kS == 2 ? c ^ ((r >> 1) & 7) : c ^ ((r >> 2) & 3); };
  uint32_t voff[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int r = lrow0 + kLoadRows * j + lane / (kRow / 16);
    voff[j] = (uint32_t)min(r, srows - 1) * rowb + 16 * place(lane % (kRow / 16), r);
  }
  // (steps past K are outside the buffer: zeros that cost no traffic)
  auto issue = [&](int step, uint32_t* buf) {
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc((void*)src, 0, step < nsteps ? (int)(srows * rowb) : 0, 0x00020000);
    uint32_t* dst = buf + (2 * B / kWaves) * wave * (kRow / 4);
    const int so = 64 * step;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const uint32_t vo = voff[j];  // (an array element passed straight makes the host pass drop the kernel's launch stub)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, dst + 256 * j, 16, vo, so, 0, 0);
    }
  };

  // scales of this lane's rows
  const uint8_t* ap[kTm];
  const uint8_t* wp[kTn];
#pragma unroll
  for (int i = 0; i < kTm; ++i) ap[i] = t.as + (m0 + min(wm * (B / kWm) + 32 * i + r32, mrows - 1)) * nb;
#pragma unroll
  for (int i = 0; i < kTn; ++i) wp[i] = t.ws + (int64_t)(n0 + min(wn * (B / 2) + 32 * i + r32, nrows - 1)) * nb;
  uint2 sa[kTm], sw[kTn];  // eight scale bytes of the next pair of steps (kStaged: of this one)
  auto load_scales = [&](int pair) {
#pragma unroll
    for (int i = 0; i < kTm; ++i) sa[i] = load_u64(ap[i] + 8 * pair);
#pragma unroll
    for (int i = 0; i < kTn; ++i) sw[i] = load_u64(wp[i] + 8 * pair);
  };
  // kStaged: 16 bytes (four steps) of each of the tile's rows through LDS
  constexpr int kScaleLoads = 2 * B / 64;  // of 64 rows; one per wave (some twice where there are more waves)
  __shared__ __attribute__((aligned(256))) uint32_t lsc[kStaged ? 2 * 2 * B * 4 : 1];
  const int sload = wave % kScaleLoads;
  const bool s_a = sload < kScaleLoads / 2;
  const int slrows = s_a ? mrows : nrows;
  const __amdgpu_buffer_rsrc_t rsc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(s_a ? t.as + m0 * nb : t.ws + (int64_t)n0 * nb), 0, slrows * nb, 0x00020000);
  const int svoff = min(sload % (kScaleLoads / 2) * 64 + lane, slrows - 1) * nb;
  auto issue_scales = [&](int group) {
    uint32_t* dst = lsc + (group & 1) * 2 * B * 4 + sload * 256;
    const int so = 16 * min(group, (nb >> 4) - 1), vo = svoff;  // (past the last: that again, not used)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsc, dst, 16, vo, so, 0, 0);
  };
  mx_u32x4 ga[kTm], gw[kTn];
  const uint32_t ssel = h ? 0x07060302u : 0x05040100u;  // bytes 2h, 2h+1 of both steps
  uint32_t ca[kTm], cw[kTn];

  f32x16 acc[kTm][kTn];
#pragma unroll
  for (int i = 0; i < kTm; ++i)
#pragma unroll
    for (int j = 0; j < kTn; ++j) acc[i][j] = f32x16{};

  uint32_t pos[2 * kS];  // of the chunk of each instruction of a stage
#pragma unroll
  for (int i = 0; i < 2 * kS; ++i) pos[i] = 16u * (uint32_t)place(4 * (i >> 1) + 2 * h + (i & 1), r32);
  const uint32_t arow = (uint32_t)(wm * (B / kWm) + r32) * kRow, wrow = (uint32_t)(B + wn * (B / 2) + r32) * kRow;
  // Instruction kk (0, 1: the first step's, 2, 3: the second's) of a stage held
  // in `buf`; scale byte `sel` of ca / cw.  keep: false zeroes this lane's block
  // of A (blocks past K).
  auto part = [&](const uint32_t* buf, auto kc, auto selc, bool keep) {
    constexpr int kk = decltype(kc)::value, sel = decltype(selc)::value;
    const uint8_t* const l = reinterpret_cast<const uint8_t*>(buf);
    mx_u32x4 fa[kTm], fw[kTn];
#pragma unroll
    for (int i = 0; i < kTm; ++i) fa[i] = *reinterpret_cast<const mx_u32x4*>(l + arow + 32 * kRow * i + pos[kk]);
#pragma unroll
    for (int i = 0; i < kTn; ++i) fw[i] = *reinterpret_cast<const mx_u32x4*>(l + wrow + 32 * kRow * i + pos[kk]);
    if (!keep)
#pragma unroll
      for (int i = 0; i < kTm; ++i) fa[i] = mx_u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < kTm; ++i)
#pragma unroll
      for (int j = 0; j < kTn; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fa[i]), operand(fw[j]), acc[i][j], kFp4, kFp4,
                                                                    sel, (int)ca[i], sel, (int)cw[j]);
  };
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
  using C3 = std::integral_constant<int, 3>;

  // Whole groups of four steps, a stage of kS of them at a time.  Every stage
  // issues the loads of kRing - 1 stages on, the first of a group (kStaged; else
  // every second one) the scales of the next steps but those, without a branch,
  // so the number of loads in flight is the same everywhere: when a stage
  // starts, the loads after its own are those of kRing - 2 stages and up to one
  // set of scales.
  const int full = nb >> 4;
  const int last_pair = 2 * full - 1;
  auto stage = [&](auto uc, int q, uint32_t* cur, uint32_t* refill) {
    constexpr int u = decltype(uc)::value;  // the stage's first step in its group
    if constexpr (kStaged)
      wait_vm<(kRing - 2) * kLoads + (kRing > 2 && u != 0 ? 1 : 0)>();
    else
      wait_vm<2 * kLoads + kTm + kTn>();
    ring_barrier();
    if constexpr (kStaged && u == 0) {
      const uint32_t* const l = lsc + ((q >> 2) & 1) * 2 * B * 4;
#pragma unroll
      for (int i = 0; i < kTm; ++i) ga[i] = *reinterpret_cast<const mx_u32x4*>(l + 4 * (wm * (B / kWm) + 32 * i + r32));
#pragma unroll
      for (int i = 0; i < kTn; ++i) gw[i] = *reinterpret_cast<const mx_u32x4*>(l + 4 * (B + wn * (B / 2) + 32 * i + r32));
      asm volatile("" ::: "memory");
      issue_scales((q >> 2) + 1);
      asm volatile("" ::: "memory");
    }
    if constexpr (kStaged && u % 2 == 0) {
#pragma unroll
      for (int i = 0; i < kTm; ++i) ca[i] = __builtin_amdgcn_perm(ga[i][u + 1], ga[i][u], ssel);
#pragma unroll
      for (int i = 0; i < kTn; ++i) cw[i] = __builtin_amdgcn_perm(gw[i][u + 1], gw[i][u], ssel);
    } else if constexpr (u % 2 == 0) {
#pragma unroll
      for (int i = 0; i < kTm; ++i) ca[i] = __builtin_amdgcn_perm(sa[i].y, sa[i].x, ssel);
#pragma unroll
      for (int i = 0; i < kTn; ++i) cw[i] = __builtin_amdgcn_perm(sw[i].y, sw[i].x, ssel);
      load_scales(min((q >> 1) + 1, last_pair));
      asm volatile("" ::: "memory");
    }
    issue(q + (kRing - 1) * kS, refill);
    asm volatile("" ::: "memory");  // the loads go out before the reads below
    part(cur, C0{}, std::integral_constant<int, 2 * (u % 2)>{}, true);
    part(cur, C1{}, std::integral_constant<int, 2 * (u % 2) + 1>{}, true);
    if constexpr (kS == 2) {
      part(cur, C2{}, C2{}, true);
      part(cur, C3{}, C3{}, true);
    }
  };
  if constexpr (kStaged) issue_scales(0);
  asm volatile("" ::: "memory");
  issue(0, l0);
  if (kRing > 2) issue(kS, l1);
  if (!kStaged && full > 0) load_scales(0);
  asm volatile("" ::: "memory");
  if (kRing > 2) issue(2 * kS, l2);
  if constexpr (kRing == 2) {
    for (int q = 0; q < 4 * full; q += 4) {
      stage(C0{}, q, l0, l1);
      stage(C2{}, q + 2, l1, l0);
    }
  } else if constexpr (kS == 1) {
    for (int q = 0; q < 4 * full; q += 4) {
      stage(C0{}, q, l0, l3);
      stage(C1{}, q + 1, l1, l0);
      stage(C2{}, q + 2, l2, l1);
      stage(C3{}, q + 3, l3, l2);
    }
  } else {
    for (int q = 0; q < 4 * full; q += 8) {
      stage(C0{}, q, l0, l3);
      stage(C2{}, q + 2, l1, l0);
      if (q + 4 == 4 * full) break;
      stage(C0{}, q + 4, l2, l1);
      stage(C2{}, q + 6, l3, l2);
    }
  }

  // The rest of K, up to four steps: three of them are already on their way.
  const int rest = kStaged ? 0 : nsteps - 4 * full;
  if (!kStaged && rest > 3) {
    // the last reads of l3 are done in every wave once all have passed here
    ring_barrier();
    issue(4 * full + 3, l3);
  }
  wait_vm<0>();  // also: no load into LDS outlives the workgroup
  ring_barrier();
  for (int u = 0; u < rest; ++u) {
    const int b0 = 4 * (4 * full + u);
    const uint32_t* const buf = u == 0 ? l0 : u == 1 ? l1 : u == 2 ? l2 : l3;
#pragma unroll
    for (int i = 0; i < kTm; ++i) ca[i] = load_tail(ap[i], b0 + 2 * h, nb);
#pragma unroll
    for (int i = 0; i < kTn; ++i) cw[i] = load_tail(wp[i], b0 + 2 * h, nb);
    part(buf, C0{}, C0{}, b0 + 2 * h < nb);
    part(buf, C1{}, C1{}, b0 + 2 * h + 1 < nb);
  }

  // lane holds column n = lane % 32, rows 8 * (v / 4) + 4 * h + v % 4
#pragma unroll
  for (int i = 0; i < kTm; ++i)
#pragma unroll
    for (int j = 0; j < kTn; ++j) {
      const int n = wn * (B / 2) + 32 * j + r32;
      if (n >= nrows) continue;
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int m = wm * (B / kWm) + 32 * i + 8 * (v >> 2) + 4 * h + (v & 3);
        if (m < mrows) store_out<kBf16>(t.out, (m0 + m) * (int64_t)t.N + n0 + n, acc[i][j][v]);
      }
    }
}

// LDS bytes of the few-row kernel: rows of codes (an odd number of 16-byte
// units, so 16 rows start in different banks), rows of scales, partial sums.
int few_arow(int nb) { return 16 * (nb | 1); }
int few_srow(int nb) { return (nb + 15) / 16 * 16 + 4; }
size_t few_lds(int64_t M, int nb) { return (size_t)(M < kFewRows ? M : kFewRows) * (few_arow(nb) + few_srow(nb)) + 12 + 2 * kFewWaves * 256 * sizeof(float); }

template <int kX>
hipError_t launch_few(const FewArgs& a, bool bf16, hipStream_t s) {
  const unsigned chunks = (unsigned)((a.M + kFewRows - 1) / kFewRows);
  const dim3 grid((unsigned)mx_few_grid(a.N, a.rw, device_cu_count()).wgs, chunks), block((unsigned)(64 * a.kw * a.rw));
  auto go = [&](auto b, auto t) { hipLaunchKernelGGL((mx_few_kernel<kX, decltype(b)::value, decltype(t)::value>), grid, block, 0, s, a); };
  const bool tail = a.nb % 16 != 0;
  if (bf16 && tail) go(std::true_type{}, std::true_type{});
  else if (bf16) go(std::true_type{}, std::false_type{});
  else if (tail) go(std::false_type{}, std::true_type{});
  else go(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

template <int B, int kWaves>
hipError_t launch_square(const TileArgs& t, bool bf16, hipStream_t s) {
  const MxTileGrid g = mx_tile_grid(t.M, t.N, B);
  const dim3 grid(g.x, g.y), block(kWaves * 64);
  auto go = [&](auto st, auto b) {
    hipLaunchKernelGGL((mx_tile_kernel<B, kWaves, decltype(st)::value, decltype(b)::value>), grid, block, 0, s, t);
  };
  const bool staged = t.nb % 16 == 0;
  if (staged && bf16) go(std::true_type{}, std::true_type{});
  else if (staged) go(std::true_type{}, std::false_type{});
  else if (bf16) go(std::false_type{}, std::true_type{});
  else go(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

}  // namespace

// Waves per group and groups side by side of the few-row kernel.
static void few_split(int nb, int& per, int& kw, int& rw) {
  const int nss = (nb + 15) / 16;
  per = (nss + kFewWaves - 1) / kFewWaves;
  kw = (nss + per - 1) / per;
  rw = kFewWaves / kw;
}

bool mx_few_fused(int64_t M, int64_t K) {
  return M <= kFewRows && M * K <= kFewFused && few_lds(M, (int)(K / 32)) <= kFewLds;
}

hipError_t launch_mx_few(const void* x, int x_dtype, const uint8_t* xs, const uint8_t* w, const uint8_t* ws, int64_t M,
                         int N, int K, int saturate, bool out_bf16, void* out, hipStream_t s) {
  FewArgs a{};
  a.x = static_cast<const uint8_t*>(x);
  a.xs = xs;
  a.w = w;
  a.ws = ws;
  a.M = M;
  a.N = N;
  a.nb = K / 32;
  few_split(a.nb, a.per, a.kw, a.rw);
  a.saturate = saturate;
  a.arow = few_arow(a.nb);
  a.srow = few_srow(a.nb);
  a.out = out;
  if (xs) return launch_few<-1>(a, out_bf16, s);
  if (x_dtype == K3MOE_DTYPE_F32) return launch_few<K3MOE_DTYPE_F32>(a, out_bf16, s);
  if (x_dtype == K3MOE_DTYPE_BF16) return launch_few<K3MOE_DTYPE_BF16>(a, out_bf16, s);
  return launch_few<K3MOE_DTYPE_F16>(a, out_bf16, s);
}

// Few rows: all that fit the kernel.  More, with a long K: where the groups of
// every 16 rows are resident at once (77 x 1003 x 4128: 32 tiles of 64 x 64, 13.0
// us, or 315 workgroups of the few-row kernel, 7.7; 128 x 1024 x 1024, short,
// 4.3 or 6.3).
hipError_t launch_mx_product(const uint8_t* a, const uint8_t* as, const uint8_t* w, const uint8_t* ws, int64_t M, int N,
                             int K, bool out_bf16, void* out, hipStream_t s) {
  int per, kw, rw;
  few_split(K / 32, per, kw, rw);
  const int64_t cus = device_cu_count(), wgs = (mx_groups(N, 16) + rw - 1) / rw;
  if (few_lds(M, K / 32) <= kFewLds && (M <= kFewRows || (K >= 4096 && (M + kFewRows - 1) / kFewRows * wgs <= 2 * cus)))
    return launch_mx_few(a, -1, as, w, ws, M, N, K, 0, out_bf16, out, s);
  TileArgs t{};
  t.a = a;
  t.as = as;
  t.w = w;
  t.ws = ws;
  t.M = (int)M;
  t.N = N;
  t.nb = K / 32;
  t.out = out;
  auto tiles = [&](int B) { return mx_tile_grid(t.M, N, B).total; };
  // the largest tile that gives every CU one and that either side more than half
  // fills (64 x 33792 x 7168: 64-row tiles 34 us, half-empty ones of 128 39;
  // 2048 x 2048 x 4096: 128, 18 us, 64, 26)
  const int64_t side = M < N ? M : N;
  if (side > 128 && tiles(256) >= cus) return launch_square<256, 8>(t, out_bf16, s);
  if (side > 64 && tiles(128) >= cus) return launch_square<128, 8>(t, out_bf16, s);
  return launch_square<64, 4>(t, out_bf16, s);
}

}  // namespace k3moe
