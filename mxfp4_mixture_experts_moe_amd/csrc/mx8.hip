// Microscaled 8-bit rows: rounding, decode, and the residual's addition with a
// root-mean-square norm whose output is rounded the same way.
//
// Scale rule as in quant.hip (OCP Microscaling Formats specification 1.0,
// section 6.3) with E4M3 elements.  A lane owns eight consecutive elements and
// four neighbouring lanes hold one block, as there.
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
// y.  An element that lies next to the border between two codes goes one way or
// the other with the last bits of y, and an fp32 sum's order moves those; so
// everything up to the rounding is fp64 (as many operations per clock here as
// fp32, and the kernel moves 5 to 8 bytes an element).  What the rounding needs of
// an fp64 y is kept in 32 bits: sign-free upper word, shifted by one, and whether
// the lower word holds anything ("key").

constexpr int64_t kMaxRows = 1 << 20;  // workgroups of a launch (a grid dimension has fewer than 2^32 threads)

struct NormArgs {
  const uint8_t *x, *residual, *gamma;
  int64_t R;
  int units;  // of eight elements, a row
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
// inside fp32's normal range, and directly outside.
template <int kType>
__device__ __forceinline__ uint16_t round16(double d) {
  const uint32_t k = key_of(d), hi = k >> 1;
  const float plain = (float)d;
  const bool normal = hi - 0x38100000u < 0x47F00000u - 0x38100000u;
  const float f = normal ? __uint_as_float((hi - 0x38000000u) << 3 | (k & 1u) | sign_of(d)) : plain;
  if constexpr (kType == K3MOE_DTYPE_BF16)
    return __builtin_bit_cast(uint16_t, (__bf16)f);
  else
    return __builtin_bit_cast(uint16_t, (_Float16)f);
}

template <int kType>
__device__ __forceinline__ void store8(uint8_t* out, int64_t unit, const double (&d)[8]) {
  if constexpr (kType == K3MOE_DTYPE_F32) {
    mx_u32x4 r[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i >> 2][i & 3] = __float_as_uint((float)d[i]);
    reinterpret_cast<mx_u32x4*>(out)[2 * unit] = r[0];
    reinterpret_cast<mx_u32x4*>(out)[2 * unit + 1] = r[1];
  } else {
    mx_u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (uint32_t)round16<kType>(d[2 * i]) | (uint32_t)round16<kType>(d[2 * i + 1]) << 16;
    reinterpret_cast<mx_u32x4*>(out)[unit] = r;
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

// v of a unit; kRes: with a residual.
template <int kType>
__device__ __forceinline__ void values(const Raw<kType>& x, const Raw<kType>& r, bool res, double (&v)[8]) {
  float a[8], b[8];
  mx8_floats<kType>(x.q, a);
  mx8_floats<kType>(r.q, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = res ? (double)a[i] + (double)b[i] : (double)a[i];
}

// Writes what a unit of eight elements gives: `unit` counts over the matrix, `col` within the row.
template <int kType, int kGamma>
__device__ __forceinline__ void finish(const NormArgs& a, int64_t unit, int col, const double (&v)[8], double rstd) {
  if (a.sum) store8<kType>(a.sum, unit, v);  // (fp32: the fp64 sum of two fp32 numbers rounds as the exact one does)
  double y[8];
  if (a.gamma) {
    const Raw<kGamma> g = load_raw<kGamma>(a.gamma, col);
    float gf[8];
    mx8_floats<kGamma>(g.q, gf);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = v[i] * rstd * (double)gf[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = v[i] * rstd;
  }
  if (a.y) store8<kType>(a.y, unit, y);
  if (a.codes) {
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, key_of(y[i]));
    const uint32_t e = scale_byte_of_key(mx_quad_max(top), a.saturate != 0);
    uint2 c = uint2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
    if (e != 255u) {
      c.x = mx8_codes4(scaled_odd(y[0], e), scaled_odd(y[1], e), scaled_odd(y[2], e), scaled_odd(y[3], e));
      c.y = mx8_codes4(scaled_odd(y[4], e), scaled_odd(y[5], e), scaled_odd(y[6], e), scaled_odd(y[7], e));
    }
    a.codes[unit] = c;
    if ((threadIdx.x & 3) == 0) a.scale[unit >> 2] = (uint8_t)e;
  }
}

// A team of 64 * waves threads per row reads the row, sums the squares, reads it
// again (from the caches) and writes.
template <int kType, int kGamma>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a) {
  __shared__ double part[16];
  const bool res = a.residual != nullptr;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
    const int64_t u0 = row * a.units;
    double ss = 0.0;
    for (int u = threadIdx.x; u < a.units; u += blockDim.x) {
      const Raw<kType> x = load_raw<kType>(a.x, u0 + u);
      const Raw<kType> r = res ? load_raw<kType>(a.residual, u0 + u) : x;
      double v[8];
      values<kType>(x, r, res, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fma(v[i], v[i], ss);
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) ss += __shfl_xor(ss, m, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
    __syncthreads();
    double t = 0.0;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) t += part[w];
    const double rstd = 1.0 / sqrt(t * a.inv_k + a.eps);
    for (int u = threadIdx.x; u < a.units; u += blockDim.x) {
      const Raw<kType> x = load_raw<kType>(a.x, u0 + u);
      const Raw<kType> r = res ? load_raw<kType>(a.residual, u0 + u) : x;
      double v[8];
      values<kType>(x, r, res, v);
      finish<kType, kGamma>(a, u0 + u, u, v, rstd);
    }
    __syncthreads();  // part[] is free again
  }
}

template <int kType, int kGamma>
void norm_launch(const NormArgs& a, hipStream_t s) {
  int waves = (a.units + 63) / 64;
  waves = waves > 16 ? 16 : waves;
  hipLaunchKernelGGL((norm_kernel<kType, kGamma>), dim3((unsigned)(a.R < kMaxRows ? a.R : kMaxRows)), dim3(64 * waves), 0, s, a);
}

template <int kType>
void norm_gamma(const NormArgs& a, int gamma_dtype, hipStream_t s) {
  if (gamma_dtype == K3MOE_DTYPE_F32) norm_launch<kType, K3MOE_DTYPE_F32>(a, s);
  else if (gamma_dtype == K3MOE_DTYPE_BF16) norm_launch<kType, K3MOE_DTYPE_BF16>(a, s);
  else norm_launch<kType, K3MOE_DTYPE_F16>(a, s);
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
  a.units = (int)(c.K / 8);
  a.eps = c.eps;
  a.inv_k = 1.0 / (double)c.K;
  a.saturate = c.saturate;
  a.sum = static_cast<uint8_t*>(c.sum);
  a.y = static_cast<uint8_t*>(c.y);
  a.codes = reinterpret_cast<uint2*>(c.codes);
  a.scale = c.scale;
  if (c.x_dtype == K3MOE_DTYPE_F32) norm_gamma<K3MOE_DTYPE_F32>(a, c.gamma_dtype, s);
  else if (c.x_dtype == K3MOE_DTYPE_BF16) norm_gamma<K3MOE_DTYPE_BF16>(a, c.gamma_dtype, s);
  else norm_gamma<K3MOE_DTYPE_F16>(a, c.gamma_dtype, s);
  return hipGetLastError();
}

}  // namespace k3moe
