// Rounding to microscaled 8 bits (E4M3 codes, one E8M0 scale per 32 elements),
// shared by the rounding kernel and the norm.
#pragma once

#include "mx_common.h"

namespace k3moe {

// E8M0 byte of a block from its largest |v| as sign-free fp32 bits, as
// mx_scale_byte with E4M3's largest exponent 8: floor(log2 m) - 8 + 127 = E - 8.
// Without saturation the scale doubles where m exceeds 448 * 2^(E-135), that is
// where the mantissa exceeds that of 1.75.
__device__ __forceinline__ uint32_t mx8_scale_byte(uint32_t top, bool saturate) {
  const uint32_t E = top >> 23;
  uint32_t e = E > 8u ? E - 8u : 0u;
  if (!saturate && E >= 8u && (top & 0x7FFFFFu) > 0x600000u) ++e;
  return E == 255u ? 255u : e;
}

// 2^(127 - e) for e <= 253: what v is multiplied by before its code is taken.
__device__ __forceinline__ float mx8_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// The codes of four scaled values, clamped to +-448 (the conversion rounds to
// nearest even, subnormals included).
__device__ __forceinline__ uint32_t mx8_codes4(float a, float b, float c, float d) {
  auto clamp = [](float v) { return __builtin_amdgcn_fmed3f(v, -448.0f, 448.0f); };
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(clamp(a), clamp(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp(c), clamp(d), r, true);
}

// Eight elements as loaded (16 bytes of 16-bit types, 32 of fp32) as fp32.
template <int kType, int kRaw>
__device__ __forceinline__ void mx8_floats(const mx_u32x4 (&raw)[kRaw], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (kType == K3MOE_DTYPE_F32) {
      const uint32_t b = raw[i >> 2][i & 3];
      v[i] = __uint_as_float(b);
    } else {
      const uint32_t d = raw[0][i >> 1];
      if constexpr (kType == K3MOE_DTYPE_BF16) {
        v[i] = __uint_as_float(i & 1 ? d & 0xFFFF0000u : d << 16);
      } else {
        const uint16_t h = (uint16_t)(i & 1 ? d >> 16 : d);
        v[i] = (float)__builtin_bit_cast(_Float16, h);
      }
    }
  }
}

}  // namespace k3moe
