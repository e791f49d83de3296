// Microscaled 4-bit quantisation of float rows into the compressed-tensors
// layout (packed codes, one E8M0 byte per 32 elements: the layout mxfp4_repack
// reads) and the decode of that layout.
//
// Scale rule: the OCP Microscaling Formats specification, version 1.0 (2023),
// section 6.3: shared exponent = floor(log2(max |v|)) minus the element type's
// largest exponent (2 for E2M1), elements rounded to nearest even and clamped
// to the largest value (saturate), or the same with the scale one step larger
// where the block's largest element would be clamped.
//
// Both kernels are copies with a conversion on the way: bound by the bytes
// they read and write (16384 x 7168 bf16: quantise 48-52 us, 5.7-6.2 TB/s;
// decode to bf16 43 us, 6.9 TB/s; a plain copy of 1 GiB runs at 5.1 TB/s).  8 x
// 7168 takes 2-3 us either way, a launch.  A lane owns eight consecutive
// elements (one dword of codes), so a bf16 row is read 16 bytes a lane in order
// and four neighbouring lanes hold one block: its maximum takes two quad
// permutes, no LDS.
#include "mx_common.h"

#include <type_traits>

namespace k3moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 2;  // groups of eight elements per thread and round (4: 54 us instead of 52, 8: 58, for 16384 x 7168 bf16)

template <int kType>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const uint8_t* __restrict__ x, int64_t n8, int saturate,
                                                            uint32_t* __restrict__ packed, uint8_t* __restrict__ scale) {
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
      uint32_t e;
      const uint32_t c = mx_quant8<kType>(raw[u], saturate != 0, e);
      if (i < n8) {
        packed[i] = c;
        if ((threadIdx.x & 3) == 0) scale[i >> 2] = (uint8_t)e;
      }
    }
  }
}

// A lane's unit is what fills one 16-byte store: eight bf16 elements (a dword of
// codes) or four fp32 ones (half a dword), so that a wave writes whole lines;
// they go past the caches (43 us instead of 49 for 16384 x 7168 to bf16).
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void unpack_kernel(const uint8_t* __restrict__ packed,
                                                          const uint8_t* __restrict__ scale, int64_t units,
                                                          mx_u32x4* __restrict__ out) {
  typedef std::conditional_t<kBf16, uint32_t, uint16_t> Codes;
  constexpr int kShift = kBf16 ? 2 : 3;  // units of a block
  for (int64_t b = (int64_t)blockIdx.x * (kThreads * kPer); b < units; b += (int64_t)gridDim.x * (kThreads * kPer)) {
    uint32_t q[kPer], e[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int64_t i = b + u * kThreads + threadIdx.x;
      const int64_t j = i < units ? i : units - 1;
      q[u] = reinterpret_cast<const Codes*>(packed)[j];
      e[u] = scale[j >> kShift];
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int64_t i = b + u * kThreads + threadIdx.x;
      if (i >= units) continue;
      const float s = mx_scale_f32(e[u] == 255u ? 127u : e[u]);
      typedef float f2 __attribute__((ext_vector_type(2)));
      f2 p[kBf16 ? 4 : 2];
      p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, 0);
      p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, 1);
      if constexpr (kBf16) {
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, 2);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, 3);
      }
      if (e[u] == 255u) {
        const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int c = 0; c < (kBf16 ? 4 : 2); ++c) p[c] = f2{nan, nan};
      }
      mx_u32x4 r;
      if constexpr (kBf16) {  // every value of finite scale is exact in bf16: its upper half is the number
#pragma unroll
        for (int c = 0; c < 4; ++c) r[c] = __builtin_amdgcn_perm(__float_as_uint(p[c][1]), __float_as_uint(p[c][0]), 0x07060302u);
      } else {
        r = mx_u32x4{__float_as_uint(p[0][0]), __float_as_uint(p[0][1]), __float_as_uint(p[1][0]), __float_as_uint(p[1][1])};
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

}  // namespace

hipError_t launch_quantize(const void* x, int x_dtype, int64_t n, int saturate, uint8_t* packed, uint8_t* scale,
                           hipStream_t s) {
  const int64_t n8 = n / 8;
  const dim3 grid(copy_grid(n8)), block(kThreads);
  const auto xp = static_cast<const uint8_t*>(x);
  const auto pp = reinterpret_cast<uint32_t*>(packed);
  if (x_dtype == K3MOE_DTYPE_F32)
    hipLaunchKernelGGL(quantize_kernel<K3MOE_DTYPE_F32>, grid, block, 0, s, xp, n8, saturate, pp, scale);
  else if (x_dtype == K3MOE_DTYPE_BF16)
    hipLaunchKernelGGL(quantize_kernel<K3MOE_DTYPE_BF16>, grid, block, 0, s, xp, n8, saturate, pp, scale);
  else
    hipLaunchKernelGGL(quantize_kernel<K3MOE_DTYPE_F16>, grid, block, 0, s, xp, n8, saturate, pp, scale);
  return hipGetLastError();
}

hipError_t launch_unpack(const uint8_t* packed, const uint8_t* scale, int64_t n, int out_bf16, void* out,
                         hipStream_t s) {
  const int64_t units = n / (out_bf16 ? 8 : 4);
  const dim3 grid(copy_grid(units)), block(kThreads);
  const auto o = static_cast<mx_u32x4*>(out);
  if (out_bf16)
    hipLaunchKernelGGL(unpack_kernel<true>, grid, block, 0, s, packed, scale, units, o);
  else
    hipLaunchKernelGGL(unpack_kernel<false>, grid, block, 0, s, packed, scale, units, o);
  return hipGetLastError();
}

}  // namespace k3moe
