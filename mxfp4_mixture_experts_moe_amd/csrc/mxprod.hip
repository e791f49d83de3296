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
//     float rows by the linear layer) in LDS; bound by the weight bytes;
//   tiles: square output tiles, both operands staged through a ring of LDS
//     buffers by direct global -> LDS loads; bound by the matrix cores for
//     large products and by load latency for small ones.
#include "mx_common.h"

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
__device__ __forceinline__ uint32_t load_u32(const uint8_t* p) {
  uint32_t v;
  __builtin_memcpy(&v, p, 4);
  return v;
}
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
// Few rows.  A workgroup of eight waves takes groups of 16 weight rows; the
// waves of a group split K in pieces of 512 (16 blocks: 256 bytes of every
// row), lane (row rho, quarter g) of a wave loads its row's blocks 4g .. 4g+3
// of the piece (64 bytes, four lanes 256 in order) and their four scale bytes
// (one dword), which feed four 16x16x128 instructions.  kw waves share a group
// (as many as K has pieces, at most eight), 8 / kw groups run side by side; the
// kw partial sums meet in LDS.  The workgroups are persistent: rows of A are
// staged (and quantised) once each.
constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / 64;
constexpr int kFewRows = 16;
constexpr int kFewLds = 80 * 1024;  // two workgroups share a CU

struct FewArgs {
  const uint8_t* x;  // float rows [M, K] (kX >= 0), or packed codes [M, K/2]
  const uint8_t* xs; // scales of packed rows
  const uint8_t* w;
  const uint8_t* ws;
  int M, N, nb;      // nb = K / 32
  int kw;            // waves per group
  int saturate;
  int arow, srow;    // LDS bytes per row of codes and of scales
  void* out;
};

template <int kX, bool kBf16>
__global__ __launch_bounds__(kFewThreads, 4) void mx_few_kernel(FewArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kFewLds];
  uint8_t* const codes = lds;                      // [M][arow]
  uint8_t* const scales = lds + a.M * a.arow;      // [M][srow]
  float* const red = reinterpret_cast<float*>(lds + ((a.M * (a.arow + a.srow) + 15) & ~15));  // [2][8 waves][256]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rho = lane & 15, g = lane >> 4;
  const int nb = a.nb, nss = (nb + 15) >> 4;

  // this wave's items: pieces s0, s0 + kw, ... of groups g0, g0 + step, ...
  const int rw = kFewWaves / a.kw, s0 = wave % a.kw, gw = wave / a.kw;
  const int ngroups = (a.N + 15) >> 4;
  const int64_t rowb = (int64_t)nb * 16;
  auto load = [&](int grp, int ss, mx_u32x4 (&q)[4], uint32_t& sc) {
    const int64_t row = min(16 * grp + rho, a.N - 1);
    const uint8_t* p = a.w + row * rowb;
    const uint8_t* ps = a.ws + row * nb;
    if (16 * ss + 16 <= nb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = __builtin_nontemporal_load(reinterpret_cast<const mx_u32x4*>(p + 256 * ss + 64 * g) + i);
      sc = load_u32(ps + 16 * ss + 4 * g);
    } else {  // the last piece: blocks past K are zeros of scale 1
      const int n = nb - 16 * ss - 4 * g;
      sc = load_tail(ps, 16 * ss + 4 * g, nb);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[i] = mx_u32x4{0u, 0u, 0u, 0u};
        if (i < n) q[i] = *(reinterpret_cast<const mx_u32x4*>(p + 256 * ss + 64 * g) + i);
      }
    }
  };
  const int gstep = (int)gridDim.x * rw;
  int grp = (int)blockIdx.x * rw + gw, ss = s0;
  mx_u32x4 q[4], qn[4];
  uint32_t sc = 0, scn = 0;
  load(min(grp, ngroups - 1), ss, q, sc);  // in flight while A is staged

  const int units = a.M * nb * 4;  // eight elements each; four lanes hold a block
  for (int u0 = 0; u0 < units; u0 += kFewThreads) {
    const int u = u0 + tid;
    const int uc = u < units ? u : units - 4 + (tid & 3);
    const int m = uc / (nb * 4), r = uc - m * (nb * 4);
    if constexpr (kX >= 0) {
      float v[8];
      mx_load8<kX>(a.x + (int64_t)uc * (kX == K3MOE_DTYPE_F32 ? 32 : 16), v);
      const uint32_t e = mx_scale_byte(mx_block_top(v), a.saturate != 0);
      const uint32_t c = mx_codes(v, e);
      if (u < units) {
        *reinterpret_cast<uint32_t*>(codes + m * a.arow + 4 * r) = c;
        if ((tid & 3) == 0) scales[m * a.srow + (r >> 2)] = (uint8_t)e;
      }
    } else if (u < units) {
      *reinterpret_cast<uint32_t*>(codes + m * a.arow + 4 * r) = reinterpret_cast<const uint32_t*>(a.x)[u];
      if ((tid & 3) == 0) scales[m * a.srow + (r >> 2)] = a.xs[u >> 2];
    }
  }
  if ((nb & 15) != 0)  // scales past K, up to the piece's end
    for (int i = tid; i < a.M * 16; i += kFewThreads)
      if (nb + (i & 15) < 16 * nss) scales[(i >> 4) * a.srow + nb + (i & 15)] = 127;
  __syncthreads();

  const int mrow = min(rho, a.M - 1);  // columns past M repeat the last row and are never stored
  const uint8_t* const brow = codes + mrow * a.arow;
  const uint8_t* const bsc = scales + mrow * a.srow;
  int par = 0;
  const int rounds = (ngroups + gstep - 1) / gstep;  // the same for every wave: the barriers below
  for (int rd = 0; rd < rounds; ++rd, grp += gstep) {
    f32x4 acc0 = {0.f, 0.f, 0.f, 0.f}, acc1 = acc0;
    for (; ss < nss; ss += a.kw) {
      const bool more = ss + a.kw < nss;
      const int gn = more ? grp : grp + gstep;
      load(min(gn, ngroups - 1), more ? ss + a.kw : s0, qn, scn);
      const uint32_t bs = *reinterpret_cast<const uint32_t*>(bsc + 16 * ss + 4 * g);
      mx_u32x4 b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = *reinterpret_cast<const mx_u32x4*>(brow + 16 * min(16 * ss + 4 * g + i, nb - 1));
      acc0 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(q[0]), operand(b[0]), acc0, kFp4, kFp4, 0, (int)sc, 0, (int)bs);
      acc1 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(q[1]), operand(b[1]), acc1, kFp4, kFp4, 1, (int)sc, 1, (int)bs);
      acc0 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(q[2]), operand(b[2]), acc0, kFp4, kFp4, 2, (int)sc, 2, (int)bs);
      acc1 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(q[3]), operand(b[3]), acc1, kFp4, kFp4, 3, (int)sc, 3, (int)bs);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = qn[i];
      sc = scn;
    }
    ss = s0;
    f32x4 sum = acc0 + acc1;
    if (a.kw > 1) {
      float* const slot = red + (par * kFewWaves + wave) * 256;
      *reinterpret_cast<f32x4*>(slot + 4 * lane) = sum;
      __syncthreads();
      if (s0 == 0)
        for (int i = 1; i < a.kw; ++i) sum += *reinterpret_cast<const f32x4*>(slot + 256 * i + 4 * lane);
      par ^= 1;
    }
    if (s0 == 0 && grp < ngroups && rho < a.M) {
      const int n = 16 * grp + 4 * g;
      const int64_t at = (int64_t)rho * a.N + n;
      if (n + 4 <= a.N && (a.N & 3) == 0) {
        if constexpr (kBf16) {
          typedef __bf16 b4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<b4*>(static_cast<__bf16*>(a.out) + at) = b4{(__bf16)sum[0], (__bf16)sum[1], (__bf16)sum[2], (__bf16)sum[3]};
        } else {
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = sum;
        }
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (n + v < a.N) store_out<kBf16>(a.out, at + v, sum[v]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Tiles.  A workgroup of four waves (2 x 2) owns a B x B tile of C; K goes in
// steps of 128 (four blocks: 64 bytes of every row) through a ring of four
// LDS buffers filled by direct global -> LDS loads, three steps ahead.  Lane
// (row r = lane % 32, half h) of a 32x32x64 instruction kk takes block 2h + kk
// of the step.  The 16-byte block c of LDS row r sits at position
// c ^ ((r >> 2) & 3) of the row's 64 bytes, so the 16-lane groups of a read
// touch every bank once.  Scales go straight to registers, eight bytes (two
// steps) of a row at a time.
constexpr int kTileThreads = 256;
constexpr int kXcds = 8;

struct TileArgs {
  const uint8_t *a, *as, *w, *ws;
  int64_t M;
  int N, nb;
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

template <int B, bool kBf16>
__global__ __launch_bounds__(kTileThreads) void mx_tile_kernel(TileArgs t) {
  constexpr int kT = B / 64;              // 32-row operand tiles per wave and side
  constexpr int kStageDw = 2 * B * 16;    // dwords of a stage: B rows of A, B rows of W, 64 bytes each
  constexpr int kLoads = 2 * B / 64;      // 1 KB loads per wave and stage
  // one array per buffer, so that the compiler sees that a read of one buffer
  // does not depend on the loads in flight into the others
  __shared__ __attribute__((aligned(256))) uint32_t l0[kStageDw], l1[kStageDw], l2[kStageDw], l3[kStageDw];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r32 = lane & 31, h = lane >> 5;

  // Tile order: the ids an XCD gets (id % 8) are a contiguous run of the
  // logical order, which walks groups of four tile rows column by column.
  const int mt = (int)((t.M + B - 1) / B), nt = (t.N + B - 1) / B;
  const int64_t total = (int64_t)mt * nt;
  int64_t id = blockIdx.x;
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

  // loads: wave w fills LDS rows 2B/4 * w ..; a 1 KB load holds 16 rows
  const bool from_a = wave < 2;
  const int lrow0 = (wave & 1) * (B / 2);  // first row within A or W
  const uint8_t* const src = from_a ? t.a + m0 * rowb : t.w + (int64_t)n0 * rowb;
  const int srows = from_a ? mrows : nrows;
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)src, 0, (int)(srows * rowb), 0x00020000);
  uint32_t voff[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int r = lrow0 + 16 * j + (lane >> 2);
    const int c = (lane & 3) ^ ((r >> 2) & 3);
    voff[j] = (uint32_t)min(r, srows - 1) * rowb + 16 * c;
  }
  auto issue = [&](int step, uint32_t* buf) {
    uint32_t* dst = buf + (B / 2) * wave * 16;
    const int so = 64 * step;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const uint32_t vo = voff[j];  // (an array element passed straight makes the host pass drop the kernel's launch stub)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, dst + 256 * j, 16, vo, so, 0, 0);
    }
  };

  // scales of this lane's rows
  const uint8_t* ap[kT];
  const uint8_t* wp[kT];
#pragma unroll
  for (int i = 0; i < kT; ++i) {
    ap[i] = t.as + (m0 + min(wm * (B / 2) + 32 * i + r32, mrows - 1)) * nb;
    wp[i] = t.ws + (int64_t)(n0 + min(wn * (B / 2) + 32 * i + r32, nrows - 1)) * nb;
  }
  uint2 sa[kT], sw[kT];  // eight scale bytes of the next pair of steps
  auto load_scales = [&](int pair) {
#pragma unroll
    for (int i = 0; i < kT; ++i) {
      sa[i] = load_u64(ap[i] + 8 * pair);
      sw[i] = load_u64(wp[i] + 8 * pair);
    }
  };
  const uint32_t ssel = h ? 0x07060302u : 0x05040100u;  // bytes 2h, 2h+1 of both steps
  uint32_t ca[kT], cw[kT];

  f32x16 acc[kT][kT];
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int j = 0; j < kT; ++j) acc[i][j] = f32x16{};

  const uint32_t pos[2] = {16u * (uint32_t)((2 * h) ^ ((lane >> 2) & 3)), 16u * (uint32_t)((2 * h + 1) ^ ((lane >> 2) & 3))};
  const uint32_t arow = (uint32_t)(wm * (B / 2) + r32) * 64, wrow = (uint32_t)(B + wn * (B / 2) + r32) * 64;
  // Instruction kk (0, 1) of a step held in `buf`; scale byte `sel` of ca / cw.
  // keep: false zeroes this lane's block of A (blocks past K).
  auto part = [&](const uint32_t* buf, auto kc, auto selc, bool keep) {
    constexpr int kk = decltype(kc)::value, sel = decltype(selc)::value;
    const uint8_t* const l = reinterpret_cast<const uint8_t*>(buf);
    mx_u32x4 fa[kT], fw[kT];
#pragma unroll
    for (int i = 0; i < kT; ++i) {
      fa[i] = *reinterpret_cast<const mx_u32x4*>(l + arow + 2048 * i + pos[kk]);
      fw[i] = *reinterpret_cast<const mx_u32x4*>(l + wrow + 2048 * i + pos[kk]);
    }
    if (!keep)
#pragma unroll
      for (int i = 0; i < kT; ++i) fa[i] = mx_u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < kT; ++i)
#pragma unroll
      for (int j = 0; j < kT; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fa[i]), operand(fw[j]), acc[i][j], kFp4, kFp4,
                                                                    sel, (int)ca[i], sel, (int)cw[j]);
  };
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
  using C3 = std::integral_constant<int, 3>;

  // Whole groups of four steps.  Every step issues the loads of three steps on
  // (past K they read other bytes of the tile's rows or nothing; no step uses
  // them), every second one the scales of the next pair, without a branch, so
  // the number of loads in flight is the same everywhere: when step q starts,
  // the loads after its own are those of steps q+1 and q+2 and one set of
  // scales.
  const int full = nb >> 4;
  const int last_pair = 2 * full - 1;
  auto step = [&](auto uc, int q, uint32_t* cur, uint32_t* refill) {
    constexpr int u = decltype(uc)::value;
    wait_vm<2 * kLoads + 2 * kT>();
    ring_barrier();
    if constexpr (u % 2 == 0) {
#pragma unroll
      for (int i = 0; i < kT; ++i) {
        ca[i] = __builtin_amdgcn_perm(sa[i].y, sa[i].x, ssel);
        cw[i] = __builtin_amdgcn_perm(sw[i].y, sw[i].x, ssel);
      }
      load_scales(min((q >> 1) + 1, last_pair));
      asm volatile("" ::: "memory");
    }
    issue(q + 3, refill);
    part(cur, C0{}, std::integral_constant<int, 2 * (u % 2)>{}, true);
    part(cur, C1{}, std::integral_constant<int, 2 * (u % 2) + 1>{}, true);
  };
  issue(0, l0);
  issue(1, l1);
  if (full > 0) load_scales(0);
  asm volatile("" ::: "memory");
  issue(2, l2);
  for (int q = 0; q < 4 * full; q += 4) {
    step(C0{}, q, l0, l3);
    step(C1{}, q + 1, l1, l0);
    step(C2{}, q + 2, l2, l1);
    step(C3{}, q + 3, l3, l2);
  }

  // The rest of K, up to four steps: three of them are already on their way.
  const int rest = nsteps - 4 * full;
  if (rest > 3) {
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
    for (int i = 0; i < kT; ++i) {
      ca[i] = load_tail(ap[i], b0 + 2 * h, nb);
      cw[i] = load_tail(wp[i], b0 + 2 * h, nb);
    }
    part(buf, C0{}, C0{}, b0 + 2 * h < nb);
    part(buf, C1{}, C1{}, b0 + 2 * h + 1 < nb);
  }

  // lane holds column n = lane % 32, rows 8 * (v / 4) + 4 * h + v % 4
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int j = 0; j < kT; ++j) {
      const int n = wn * (B / 2) + 32 * j + r32;
      if (n >= nrows) continue;
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int m = wm * (B / 2) + 32 * i + 8 * (v >> 2) + 4 * h + (v & 3);
        if (m < mrows) store_out<kBf16>(t.out, (m0 + m) * (int64_t)t.N + n0 + n, acc[i][j][v]);
      }
    }
}

// LDS bytes of the few-row kernel: rows of codes (an odd number of 16-byte
// units, so 16 rows start in different banks), rows of scales, partial sums.
int few_arow(int nb) { return 16 * (nb | 1); }
int few_srow(int nb) { return (nb + 15) / 16 * 16 + 4; }
size_t few_lds(int64_t M, int nb) { return (size_t)M * (few_arow(nb) + few_srow(nb)) + 12 + 2 * kFewWaves * 256 * sizeof(float); }

template <int kX>
hipError_t launch_few(const FewArgs& a, bool bf16, hipStream_t s) {
  const int ngroups = (a.N + 15) / 16, rw = kFewWaves / a.kw;
  const int64_t wgs = (ngroups + rw - 1) / rw;
  const int64_t most = 2 * device_cu_count();
  const dim3 grid((unsigned)(wgs < most ? wgs : most)), block(kFewThreads);
  if (bf16)
    hipLaunchKernelGGL((mx_few_kernel<kX, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((mx_few_kernel<kX, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <int B>
hipError_t launch_square(const TileArgs& t, bool bf16, hipStream_t s) {
  const int64_t total = ((t.M + B - 1) / B) * ((t.N + B - 1) / B);
  const dim3 grid((unsigned)total), block(kTileThreads);
  if (bf16)
    hipLaunchKernelGGL((mx_tile_kernel<B, true>), grid, block, 0, s, t);
  else
    hipLaunchKernelGGL((mx_tile_kernel<B, false>), grid, block, 0, s, t);
  return hipGetLastError();
}

}  // namespace

bool mx_few_supported(int64_t M, int nb) { return M <= kFewRows && few_lds(M, nb) <= kFewLds; }

hipError_t launch_mx_few(const void* x, int x_dtype, const uint8_t* xs, const uint8_t* w, const uint8_t* ws, int64_t M,
                         int N, int K, int saturate, bool out_bf16, void* out, hipStream_t s) {
  FewArgs a{};
  a.x = static_cast<const uint8_t*>(x);
  a.xs = xs;
  a.w = w;
  a.ws = ws;
  a.M = (int)M;
  a.N = N;
  a.nb = K / 32;
  const int nss = (a.nb + 15) / 16;
  a.kw = nss >= 8 ? 8 : nss >= 4 ? 4 : nss >= 2 ? 2 : 1;
  a.saturate = saturate;
  a.arow = few_arow(a.nb);
  a.srow = few_srow(a.nb);
  a.out = out;
  if (xs) return launch_few<-1>(a, out_bf16, s);
  if (x_dtype == K3MOE_DTYPE_F32) return launch_few<K3MOE_DTYPE_F32>(a, out_bf16, s);
  if (x_dtype == K3MOE_DTYPE_BF16) return launch_few<K3MOE_DTYPE_BF16>(a, out_bf16, s);
  return launch_few<K3MOE_DTYPE_F16>(a, out_bf16, s);
}

hipError_t launch_mx_tiles(const uint8_t* a, const uint8_t* as, const uint8_t* w, const uint8_t* ws, int64_t M, int N,
                           int K, bool out_bf16, void* out, hipStream_t s) {
  TileArgs t{};
  t.a = a;
  t.as = as;
  t.w = w;
  t.ws = ws;
  t.M = M;
  t.N = N;
  t.nb = K / 32;
  t.out = out;
  const int64_t cus = device_cu_count();
  auto tiles = [&](int64_t B) { return ((M + B - 1) / B) * ((N + B - 1) / B); };
  if (tiles(256) >= cus) return launch_square<256>(t, out_bf16, s);
  if (tiles(128) >= cus) return launch_square<128>(t, out_bf16, s);
  return launch_square<64>(t, out_bf16, s);
}

}  // namespace k3moe
