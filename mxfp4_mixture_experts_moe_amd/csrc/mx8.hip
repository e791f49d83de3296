// Microscaled 8-bit rows: rounding, decode, and the residual's addition with a
// root-mean-square norm whose output is rounded the same way.
//
// Scale rule as in quant.hip (OCP Microscaling Formats specification 1.0,
// section 6.3) with E4M3 elements.  A lane owns eight consecutive elements and
// four neighbouring lanes hold one block, as there.  Bound by the bytes:
// 16384 x 7168 bf16 are rounded in 64 us, 5.6 TB/s, and decoded in 50 to 57.
#include "mx8_common.h"

#include <type_traits>

namespace k3moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 2;  // groups of eight elements per thread and round

template <int kType>
__global__ __launch_bounds__(kThreads) void quantize8_kernel(const uint8_t* __restrict__ x, int64_t n8, int saturate,
                                                             uint2* __restrict__ codes, uint8_t* __restrict__ scale) {
  constexpr int kRaw = kType == K3MOE_DTYPE_F32 ? 2 : 1;
  // n8 is a multiple of 4, so the four lanes of a block are in or out together
  for (int64_t b = (int64_t)blockIdx.x * (kThreads * kPer); b < n8; b += (int64_t)gridDim.x * (kThreads * kPer)) {
    mx_u32x4 raw[kPer][kRaw];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int64_t i = b + u * kThreads + threadIdx.x;
      const int64_t j = i < n8 ? i : n8 - 4 + (threadIdx.x & 3);
#pragma unroll
      for (int h = 0; h < kRaw; ++h) raw[u][h] = reinterpret_cast<const mx_u32x4*>(x)[j * kRaw + h];
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int64_t i = b + u * kThreads + threadIdx.x;
      float v[8];
      mx8_floats<kType>(raw[u], v);
      const uint32_t e = mx8_scale_byte(mx_block_top(v), saturate != 0);
      const float s = mx8_inverse(e == 255u ? 127u : e);
      uint2 c;
      c.x = mx8_codes4(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
      c.y = mx8_codes4(v[4] * s, v[5] * s, v[6] * s, v[7] * s);
      if (e == 255u) c = uint2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
      if (i < n8) {
        codes[i] = c;
        if ((threadIdx.x & 3) == 0) scale[i >> 2] = (uint8_t)e;
      }
    }
  }
}

// A lane's unit fills one 16-byte store: eight bf16 elements or four fp32 ones.
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void unpack8_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scale, int64_t units,
                                                           mx_u32x4* __restrict__ out) {
  typedef std::conditional_t<kBf16, uint2, uint32_t> Codes;
  constexpr int kShift = kBf16 ? 2 : 3;  // units of a block
  for (int64_t b = (int64_t)blockIdx.x * (kThreads * kPer); b < units; b += (int64_t)gridDim.x * (kThreads * kPer)) {
    Codes q[kPer];
    uint32_t e[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int64_t i = b + u * kThreads + threadIdx.x;
      const int64_t j = i < units ? i : units - 1;
      q[u] = reinterpret_cast<const Codes*>(codes)[j];
      e[u] = scale[j >> kShift];
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int64_t i = b + u * kThreads + threadIdx.x;
      if (i >= units) continue;
      const float s = e[u] == 255u ? __uint_as_float(0x7FC00000u) : mx_scale_f32(e[u]);
      typedef float f2 __attribute__((ext_vector_type(2)));
      mx_u32x4 r;
      if constexpr (kBf16) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t d = c < 2 ? q[u].x : q[u].y;
          const f2 p = c & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)d, true) : __builtin_amdgcn_cvt_pk_f32_fp8((int)d, false);
          const __bf16 lo = (__bf16)(p[0] * s), hi = (__bf16)(p[1] * s);
          r[c] = (uint32_t)__builtin_bit_cast(uint16_t, lo) | (uint32_t)__builtin_bit_cast(uint16_t, hi) << 16;
        }
      } else {
        const f2 p = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[u], false), t = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[u], true);
        r = mx_u32x4{__float_as_uint(p[0] * s), __float_as_uint(p[1] * s), __float_as_uint(t[0] * s), __float_as_uint(t[1] * s)};
      }
      __builtin_nontemporal_store(r, out + i);
    }
  }
}

unsigned copy_grid(int64_t units) {
  const int64_t g = (units + kThreads * kPer - 1) / (kThreads * kPer);
  const int64_t most = (int64_t)1 << 20;
  return (unsigned)(g < most ? g : most);
}

// ---------------------------------------------------------------------------
// Residual, norm and rounding.
//
// y = v / sqrt(mean(v^2) + eps) * gamma with v = x + residual, and the codes of
// y.  An element next to the border between two codes goes one way or the other
// with the last bits of y, and an fp32 sum's order moves those; so the sum of
// squares is fp64, and so is y wherever it matters: an fp32 y, off by at most
// kOff of itself, is rounded from both ends of that interval, and where the two
// differ in any element of a wave's units (or the block's scale does), the wave
// takes these units again in fp64.  That is 0.6% of the units for codes alone,
// about 12% with y in bf16, too; y in the finer types is fp64 always.
// What the rounding needs of an fp64 y is kept in 32 bits: sign-free upper word,
// shifted by one, and whether the lower word holds anything ("key").
//
// A row stays in the registers of its threads between the sum and the rounding.
//
// Bound by the bytes where rows are many: 16384 x 7168 bf16 with residual and sum,
// 826 MB, 177 to 182 us, 4.5 to 4.7 TB/s (fp64 throughout and rows read twice: 368
// us), with y, 1.06 GB, 217; f16 177 and, y in fp64, 240; f32 282 and 369 (5.4
// TB/s).  (On a card that has been idle the first 25 ms are slower, 202 instead of
// 177.)  One row of 7168 takes 4.4 to 5 us, the chain of loads, sum over the
// workgroup, root, division and rounding.

constexpr int64_t kMaxGroups = 1 << 20;  // workgroups of a launch (a grid dimension has fewer than 2^32 threads)

struct NormArgs {
  const uint8_t *x, *residual, *gamma;
  int gamma_type;
  int64_t R;
  int units;  // of eight elements, a row
  int team;   // lanes of a row where several share a wave
  double eps, inv_k;
  int saturate;
  uint8_t *sum, *y;
  uint2* codes;
  uint8_t* scale;
};

// d as sign-free key: bits 31..1 the upper word's lower 31, bit 0: the lower word is not 0.
__device__ __forceinline__ uint32_t key_of(double d) {
  const uint64_t b = (uint64_t)__double_as_longlong(d);
  return (uint32_t)(b >> 32) << 1 | ((uint32_t)b != 0u ? 1u : 0u);
}
__device__ __forceinline__ uint32_t sign_of(double d) { return (uint32_t)((uint64_t)__double_as_longlong(d) >> 32) & 0x80000000u; }

// E8M0 byte from the largest key of a block: the exponent field of fp64 is key >> 21.
__device__ __forceinline__ uint32_t scale_byte_of_key(uint32_t top, bool saturate) {
  const uint32_t E = top >> 21;
  uint32_t e = E > 904u ? E - 904u : 0u;  // (E - 1023) - 8 + 127
  if (!saturate && E >= 904u && (top & 0x1FFFFFu) > 0x180000u) ++e;
  return e > 254u ? 255u : e;
}

// y / 2^(e - 127) as fp32 with 20 mantissa bits and a last one that stands for
// all the rest (rounded to odd), which rounds to E4M3 as y itself does.  Below
// fp32's normal range: 0, as all that is far below E4M3's smallest step.
__device__ __forceinline__ float scaled_odd(double y, uint32_t e) {
  const uint32_t k = key_of(y);
  const int t = (int)((k >> 1) - ((769u + e) << 20));  // exponent E - 1023 + 127 - e, biased by 127
  const uint32_t m = t < (1 << 20) ? 0u : ((uint32_t)t << 3 | (k & 1u));
  return __uint_as_float(m | sign_of(y));
}

// fp64 rounded once to a 16-bit type: by way of an fp32 number rounded to odd
// inside fp32's normal range, and directly outside.  bf16 has numbers below that
// range, n steps of 2^-133 whose bits are n: the sum with 1.5 * 2^-81, where fp64 has
// these steps, ends in n.  (fp32's own steps there, 2^-149, would round a first time,
// and that onto ties.)
template <int kType>
__device__ __forceinline__ uint16_t round16(double d) {
  const uint32_t k = key_of(d), hi = k >> 1;
  const float plain = (float)d;
  const bool inside = (kType == K3MOE_DTYPE_BF16 || hi >= 0x38100000u) && hi < 0x47F00000u;
  const float f = inside ? __uint_as_float((hi - 0x38000000u) << 3 | (k & 1u) | sign_of(d)) : plain;
  if constexpr (kType == K3MOE_DTYPE_BF16) {
    const uint32_t n = (uint32_t)(uint64_t)__double_as_longlong(fabs(d) + 0x1.8p-81) | sign_of(d) >> 16;
    return hi < 0x38100000u ? (uint16_t)n : __builtin_bit_cast(uint16_t, (__bf16)f);
  } else {
    return __builtin_bit_cast(uint16_t, (_Float16)f);
  }
}
template <int kType>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (kType == K3MOE_DTYPE_BF16) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, b2{(__bf16)a, (__bf16)b});
  } else {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, h2{(_Float16)a, (_Float16)b});
  }
}

template <int kType>
struct Raw {
  mx_u32x4 q[kType == K3MOE_DTYPE_F32 ? 2 : 1];
};
template <int kType>
__device__ __forceinline__ Raw<kType> load_raw(const uint8_t* p, int64_t unit) {
  constexpr int kRaw = kType == K3MOE_DTYPE_F32 ? 2 : 1;
  Raw<kType> r;
#pragma unroll
  for (int h = 0; h < kRaw; ++h) r.q[h] = reinterpret_cast<const mx_u32x4*>(p)[unit * kRaw + h];
  return r;
}
template <int kType>
__device__ __forceinline__ void store_raw(uint8_t* p, int64_t unit, const Raw<kType>& r) {
  constexpr int kRaw = kType == K3MOE_DTYPE_F32 ? 2 : 1;
#pragma unroll
  for (int h = 0; h < kRaw; ++h) reinterpret_cast<mx_u32x4*>(p)[unit * kRaw + h] = r.q[h];
}

// Gamma of a unit, as loaded (a 16-bit type leaves the second half alone), and as fp32.
struct GammaRaw {
  mx_u32x4 q[2];
};
__device__ __forceinline__ GammaRaw load_gamma(const NormArgs& a, int col) {
  GammaRaw g{};
  if (!a.gamma) return g;
  if (a.gamma_type == K3MOE_DTYPE_F32) {
    g.q[0] = reinterpret_cast<const mx_u32x4*>(a.gamma)[2 * col];
    g.q[1] = reinterpret_cast<const mx_u32x4*>(a.gamma)[2 * col + 1];
  } else {
    g.q[0] = reinterpret_cast<const mx_u32x4*>(a.gamma)[col];
  }
  return g;
}
__device__ __forceinline__ void gamma_floats(const NormArgs& a, const GammaRaw& g, float (&f)[8]) {
  const mx_u32x4 half[1] = {g.q[0]};
  if (!a.gamma) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.0f;
  } else if (a.gamma_type == K3MOE_DTYPE_F32) {
    mx8_floats<K3MOE_DTYPE_F32>(g.q, f);
  } else if (a.gamma_type == K3MOE_DTYPE_BF16) {
    mx8_floats<K3MOE_DTYPE_BF16>(half, f);
  } else {
    mx8_floats<K3MOE_DTYPE_F16>(half, f);
  }
}

// What a row's threads know: `unit` counts over the matrix.
template <int kType>
struct Unit {
  Raw<kType> x, r;
  GammaRaw g;
};

// Sum of the squares of a unit's v, exact products of fp64 sums.
template <int kType>
__device__ __forceinline__ double squares(const Unit<kType>& w, bool res, double ss) {
  float x[8], r[8];
  mx8_floats<kType>(w.x.q, x);
  if (res) {
    mx8_floats<kType>(w.r.q, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double v = (double)x[i] + (double)r[i];
      ss = fma(v, v, ss);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma((double)x[i], (double)x[i], ss);
  }
  return ss;
}

// y and its codes in fp64 (c and e: the unit's codes and its block's scale byte; y: the rounded y, where it is wanted).
template <int kType>
__device__ __forceinline__ void exact_unit(const NormArgs& a, const Unit<kType>& w, bool res, double rstd, uint2& c, uint32_t& e, Raw<kType>& yr) {
  float x[8], r[8], g[8];
  mx8_floats<kType>(w.x.q, x);
  mx8_floats<kType>(w.r.q, r);
  gamma_floats(a, w.g, g);
  double y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double v = res ? (double)x[i] + (double)r[i] : (double)x[i];
    y[i] = v * rstd * (double)g[i];
  }
  if (a.y) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (kType == K3MOE_DTYPE_F32)
        yr.q[i >> 2][i & 3] = __float_as_uint((float)y[i]);
      else if (i % 2 == 0) {
        uint32_t p = (uint32_t)round16<kType>(y[i]) | (uint32_t)round16<kType>(y[i + 1]) << 16;
        if constexpr (kType == K3MOE_DTYPE_BF16) asm volatile("" : "+v"(p));  // (a pair at a time: all eight at once spill)
        yr.q[0][i / 2] = p;
      }
    }
  }
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, key_of(y[i]));
  e = scale_byte_of_key(mx_quad_max(top), a.saturate != 0);
  c = uint2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
  if (e != 255u) {
    c.x = mx8_codes4(scaled_odd(y[0], e), scaled_odd(y[1], e), scaled_odd(y[2], e), scaled_odd(y[3], e));
    c.y = mx8_codes4(scaled_odd(y[4], e), scaled_odd(y[5], e), scaled_odd(y[6], e), scaled_odd(y[7], e));
  }
}

// An fp32 y = (v rounded * rstd rounded) * gamma carries four roundings of 2^-24,
// and its product with 1 -+ kOff one more.  That takes results in fp32's normal
// range; below it, a rounding of v * rstd to fp32's subnormals moves y by at most
// 2^-150 gamma, 2^-36 of the unit of a block of scale byte 32 or more with |gamma|
// < 2^19, which is less than the sixth 2^-24 is of anything that does not round to 0.
constexpr float kOff = 6.0f / (1 << 24);

// The same from fp32 intervals; false: an element (of this lane) needs fp64.
template <int kType, bool kY>
__device__ __forceinline__ bool quick_unit(const NormArgs& a, const Unit<kType>& w, bool res, float rstd, uint2& c, uint32_t& e, Raw<kType>& yr) {
  float v[8], g[8], y[8];
  mx8_floats<kType>(w.x.q, v);
  if (res) {
    float r[8];
    mx8_floats<kType>(w.r.q, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  gamma_floats(a, w.g, g);
  uint32_t top = 0u, gtop = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = v[i] * rstd * g[i];
    top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    gtop = max(gtop, __float_as_uint(g[i]) & 0x7FFFFFFFu);
  }
  const bool sat = a.saturate != 0;
  const float ftop = __uint_as_float(mx_quad_max(top));
  e = mx8_scale_byte(__float_as_uint(ftop * (1.0f + kOff)), sat);
  bool sure = e == mx8_scale_byte(__float_as_uint(ftop * (1.0f - kOff)), sat) && e - 32u < 192u && gtop < (127u + 19u) << 23 && rstd > 0x1p-100f;
  const float s = mx8_inverse(e == 255u ? 127u : e), sl = s * (1.0f - kOff), sh = s * (1.0f + kOff);
  c.x = mx8_codes4(y[0] * sl, y[1] * sl, y[2] * sl, y[3] * sl);
  c.y = mx8_codes4(y[4] * sl, y[5] * sl, y[6] * sl, y[7] * sl);
  sure &= c.x == mx8_codes4(y[0] * sh, y[1] * sh, y[2] * sh, y[3] * sh);
  sure &= c.y == mx8_codes4(y[4] * sh, y[5] * sh, y[6] * sh, y[7] * sh);
  if constexpr (kY) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = y[2 * i], q = y[2 * i + 1];
      yr.q[0][i] = pack16<kType>(p * (1.0f - kOff), q * (1.0f - kOff));
      sure &= yr.q[0][i] == pack16<kType>(p * (1.0f + kOff), q * (1.0f + kOff));
      // below 2^-106 the result, or v * rstd under a gamma of up to 2^19, may lie below fp32's
      // normal range, where roundings are not relative any more
      sure &= (__float_as_uint(p) & 0x7FFFFFFFu) >= (127u - 106u) << 23 || v[2 * i] == 0.0f;
      sure &= (__float_as_uint(q) & 0x7FFFFFFFu) >= (127u - 106u) << 23 || v[2 * i + 1] == 0.0f;
    }
  }
  return sure;
}

// Writes what a unit gives.  kMode 0: codes only, 1: y in bf16, too, 2: fp64 throughout.
template <int kType, int kMode>
__device__ __forceinline__ void finish(const NormArgs& a, const Unit<kType>& w, int64_t unit, bool live, bool res, double rstd) {
  uint2 c;
  uint32_t e;
  Raw<kType> yr;
  bool sure = false;
  if constexpr (kMode != 2) sure = quick_unit<kType, kMode == 1>(a, w, res, (float)rstd, c, e, yr);
  if (kMode == 2 || __builtin_amdgcn_ballot_w64(live && !sure) != 0) exact_unit<kType>(a, w, res, rstd, c, e, yr);
  if (!live) return;
  if (a.sum) {
    // v rounded once.  Two 16-bit numbers whose fp32 sum is not exact lie so far
    // apart that it rounds to the type as the exact one does.
    float x[8], r[8];
    mx8_floats<kType>(w.x.q, x);
    mx8_floats<kType>(w.r.q, r);
    Raw<kType> t;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (res) x[i] += r[i];
      if constexpr (kType == K3MOE_DTYPE_F32)
        t.q[i >> 2][i & 3] = __float_as_uint(x[i]);
      else if (i % 2 == 1)
        t.q[0][i / 2] = pack16<kType>(x[i - 1], x[i]);
    }
    store_raw<kType>(a.sum, unit, t);
  }
  if (kMode != 0 && a.y) store_raw<kType>(a.y, unit, yr);
  if (a.codes) {
    a.codes[unit] = c;
    if ((threadIdx.x & 3) == 0) a.scale[unit >> 2] = (uint8_t)e;
  }
}

template <int kType>
__device__ __forceinline__ Unit<kType> load_unit(const NormArgs& a, int64_t row0, int u, bool res, bool gamma) {
  Unit<kType> w;
  w.x = load_raw<kType>(a.x, row0 + u);
  w.r = res ? load_raw<kType>(a.residual, row0 + u) : w.x;
  if (gamma) w.g = load_gamma(a, u);
  return w;
}

// Rows of up to 512 elements: `team` lanes (a power of two) each, several to a wave.
template <int kType, int kMode>
__global__ __launch_bounds__(256) void norm_short_kernel(NormArgs a) {
  const bool res = a.residual != nullptr;
  const int lane = threadIdx.x & 63, u = lane % a.team, per_wave = 64 / a.team;
  const int64_t step = (int64_t)gridDim.x * 4 * per_wave;
  for (int64_t row0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * per_wave; row0 < a.R; row0 += step) {
    const int64_t row = row0 + lane / a.team;
    const bool live = row < a.R && u < a.units;
    const int64_t first = (row < a.R ? row : a.R - 1) * a.units;
    const Unit<kType> w = load_unit<kType>(a, first, u < a.units ? u : (u & 3), res, true);
    double ss = live ? squares<kType>(w, res, 0.0) : 0.0;
    for (int m = 1; m < a.team; m <<= 1) ss += __shfl_xor(ss, m, 64);
    finish<kType, kMode>(a, w, first + u, live, res, 1.0 / sqrt(ss * a.inv_k + a.eps));
  }
}

// The sum of a row's squares over a workgroup, in every thread.
__device__ __forceinline__ double row_sum(double ss, double (&part)[16]) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) ss += __shfl_xor(ss, m, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
  __syncthreads();
  double t = 0.0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) t += part[w];
  return t;
}

// Longer rows: a workgroup each, kU units of a thread in its registers (kU 0:
// rows beyond the registers of 1024 threads, which are read twice).
template <int kType, int kMode, int kU>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a) {
  __shared__ double part[16];
  const bool res = a.residual != nullptr;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
    const int64_t first = row * a.units;
    if constexpr (kU > 0) {
      Unit<kType> w[kU];
      double ss = 0.0;
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int u = threadIdx.x + i * blockDim.x;
        w[i] = load_unit<kType>(a, first, u < a.units ? u : (u & 3), res, kU == 1);
      }
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if ((int)(threadIdx.x + i * blockDim.x) < a.units) ss = squares<kType>(w[i], res, ss);
      const double rstd = 1.0 / sqrt(row_sum(ss, part) * a.inv_k + a.eps);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int u = threadIdx.x + i * blockDim.x;
        if (kU > 1) w[i].g = load_gamma(a, u < a.units ? u : (u & 3));  // (from the caches, and not held meanwhile)
        finish<kType, kMode>(a, w[i], first + u, u < a.units, res, rstd);
      }
    } else {
      double ss = 0.0;
      for (int u = threadIdx.x; u < a.units; u += blockDim.x) ss = squares<kType>(load_unit<kType>(a, first, u, res, false), res, ss);
      const double rstd = 1.0 / sqrt(row_sum(ss, part) * a.inv_k + a.eps);
      for (int u = threadIdx.x; u < a.units; u += blockDim.x)
        finish<kType, kMode>(a, load_unit<kType>(a, first, u, res, true), first + u, true, res, rstd);
    }
    __syncthreads();  // part[] is free again
  }
}

template <int kType, int kMode>
void norm_launch(NormArgs a, hipStream_t s) {
  if (a.units <= 64) {
    a.team = 4;
    while (a.team < a.units) a.team *= 2;
    const int64_t rows = 4 * (64 / a.team), wgs = (a.R + rows - 1) / rows;
    hipLaunchKernelGGL((norm_short_kernel<kType, kMode>), dim3((unsigned)(wgs < kMaxGroups ? wgs : kMaxGroups)), dim3(256), 0, s, a);
    return;
  }
  // Few rows: as many threads as there are units.  Rows for every CU: more units
  // a thread, so that several small workgroups, each at its own stage, share a CU
  // (16384 x 7168 bf16, one, two or four units a thread: 286, 205, 178 us).
  constexpr int kMost = kType == K3MOE_DTYPE_F32 ? 2 : 4;
  const int want = a.R <= device_cu_count() ? 1 : (a.units + 63) / 64;
  int per = 1;
  while (per < kMost && (per < want || a.units > 1024 * per)) per *= 2;
  const dim3 grid((unsigned)(a.R < kMaxGroups ? a.R : kMaxGroups));
  if (a.units > 1024 * kMost) {
    hipLaunchKernelGGL((norm_kernel<kType, kMode, 0>), grid, dim3(1024), 0, s, a);
    return;
  }
  const dim3 block((unsigned)((a.units + 64 * per - 1) / (64 * per) * 64));
  if (per == 1) hipLaunchKernelGGL((norm_kernel<kType, kMode, 1>), grid, block, 0, s, a);
  else if (per == 2) hipLaunchKernelGGL((norm_kernel<kType, kMode, 2>), grid, block, 0, s, a);
  else if constexpr (kMost == 4) hipLaunchKernelGGL((norm_kernel<kType, kMode, 4>), grid, block, 0, s, a);
}

template <int kType>
void norm_mode(const NormArgs& a, hipStream_t s) {
  if (!a.y) norm_launch<kType, 0>(a, s);
  else if constexpr (kType == K3MOE_DTYPE_BF16) norm_launch<kType, 1>(a, s);
  else norm_launch<kType, 2>(a, s);
}

}  // namespace

hipError_t launch_quantize8(const void* x, int x_dtype, int64_t n, int saturate, uint8_t* codes, uint8_t* scale,
                            hipStream_t s) {
  const int64_t n8 = n / 8;
  const dim3 grid(copy_grid(n8)), block(kThreads);
  const auto xp = static_cast<const uint8_t*>(x);
  const auto cp = reinterpret_cast<uint2*>(codes);
  if (x_dtype == K3MOE_DTYPE_F32)
    hipLaunchKernelGGL(quantize8_kernel<K3MOE_DTYPE_F32>, grid, block, 0, s, xp, n8, saturate, cp, scale);
  else if (x_dtype == K3MOE_DTYPE_BF16)
    hipLaunchKernelGGL(quantize8_kernel<K3MOE_DTYPE_BF16>, grid, block, 0, s, xp, n8, saturate, cp, scale);
  else
    hipLaunchKernelGGL(quantize8_kernel<K3MOE_DTYPE_F16>, grid, block, 0, s, xp, n8, saturate, cp, scale);
  return hipGetLastError();
}

hipError_t launch_unpack8(const uint8_t* codes, const uint8_t* scale, int64_t n, int out_bf16, void* out,
                          hipStream_t s) {
  const int64_t units = n / (out_bf16 ? 8 : 4);
  const dim3 grid(copy_grid(units)), block(kThreads);
  const auto o = static_cast<mx_u32x4*>(out);
  if (out_bf16)
    hipLaunchKernelGGL(unpack8_kernel<true>, grid, block, 0, s, codes, scale, units, o);
  else
    hipLaunchKernelGGL(unpack8_kernel<false>, grid, block, 0, s, codes, scale, units, o);
  return hipGetLastError();
}

hipError_t launch_norm8(const NormCall& c, hipStream_t s) {
  NormArgs a{};
  a.x = static_cast<const uint8_t*>(c.x);
  a.residual = static_cast<const uint8_t*>(c.residual);
  a.gamma = static_cast<const uint8_t*>(c.gamma);
  a.R = c.R;
  a.gamma_type = c.gamma_dtype;
  a.units = (int)(c.K / 8);
  a.eps = c.eps;
  a.inv_k = 1.0 / (double)c.K;
  a.saturate = c.saturate;
  a.sum = static_cast<uint8_t*>(c.sum);
  a.y = static_cast<uint8_t*>(c.y);
  a.codes = reinterpret_cast<uint2*>(c.codes);
  a.scale = c.scale;
  if (c.x_dtype == K3MOE_DTYPE_F32) norm_mode<K3MOE_DTYPE_F32>(a, s);
  else if (c.x_dtype == K3MOE_DTYPE_BF16) norm_mode<K3MOE_DTYPE_BF16>(a, s);
  else norm_mode<K3MOE_DTYPE_F16>(a, s);
  return hipGetLastError();
}

}  // namespace k3moe
