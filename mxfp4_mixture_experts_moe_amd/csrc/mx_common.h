// Rounding of fp32 values to microscaled 4 bits, shared by the quantisation
// kernel and the linear layer that quantises its rows itself.
#pragma once

#include "k3moe_internal.h"

namespace k3moe {

typedef uint32_t mx_u32x4 __attribute__((ext_vector_type(4)));

// The value 2^(e - 127) of an E8M0 byte e <= 254 as fp32 (e = 0: the subnormal 2^-127).
__device__ __forceinline__ float mx_scale_f32(uint32_t e) { return __uint_as_float(e ? (e << 23) : 0x00400000u); }

// E8M0 byte of a 32-element block from the largest |v| of the block, given as
// fp32 bits without the sign (they order like the magnitudes; an infinity or a
// NaN is largest).  With E = the exponent field, floor(log2 m) = E - 127, so
// floor(log2 m) - 2 + 127 = E - 2, clamped to 0 (subnormal and tiny blocks,
// and the all-zero block).  Without saturation the scale doubles where m
// exceeds 6 * 2^(E-129), that is where the mantissa exceeds that of 1.5.
// 255 (NaN) marks a block that holds a non-finite value.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top, bool saturate) {
  const uint32_t E = top >> 23;
  uint32_t e = E > 2u ? E - 2u : 0u;
  if (!saturate && E >= 2u && (top & 0x7FFFFFu) > 0x400000u) ++e;
  return E == 255u ? 255u : e;
}

// The eight codes of v[0..7] (element i in nibble i) for a block of scale byte
// e: nearest E2M1 value of v * 2^(127 - e), ties to the even code, beyond 6
// clamped, sign kept.  The conversion instruction divides by its scale operand
// and rounds exactly so for every exponent, 2^-127 included.  Blocks of byte
// 255 get the code 7 throughout: a decoder that takes 255 for NaN gives NaN,
// one that computes 2^(e - 128) gives an infinity, none gives a plain number.
__device__ __forceinline__ uint32_t mx_codes(const float (&v)[8], uint32_t e) {
  const float s = mx_scale_f32(e == 255u ? 127u : e);
  uint32_t r = 0u;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], s, 3);
  return e == 255u ? 0x77777777u : r;
}

// Largest of the four lanes 4q .. 4q+3: two quad permutes.
__device__ __forceinline__ uint32_t mx_quad_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));  // lane ^ 1
  return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));  // lane ^ 2
}
// Largest |v| of the four lanes 4q .. 4q+3 (a block of 32 elements, eight a
// lane), as sign-free bits.
__device__ __forceinline__ uint32_t mx_block_top(const float (&v)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return mx_quad_max(m);
}

// Codes and scale byte (e) of a lane's eight elements of a block of four lanes,
// as loaded (16 bytes of 16-bit elements, 32 of fp32).  16-bit elements stay
// packed: their magnitudes order like their bits, too, and the conversion takes
// them as they are, with the same rounding.
template <int kType, int kRaw>
__device__ __forceinline__ uint32_t mx_quant8(const mx_u32x4 (&raw)[kRaw], bool saturate, uint32_t& e) {
  if constexpr (kType == K3MOE_DTYPE_F32) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t bits = raw[i >> 2][i & 3];
      v[i] = __uint_as_float(bits);
    }
    e = mx_scale_byte(mx_block_top(v), saturate);
    return mx_codes(v, e);
  } else {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    const uint32_t d[4] = {raw[0][0], raw[0][1], raw[0][2], raw[0][3]};
    u16x2 m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = __builtin_bit_cast(u16x2, d[i] & 0x7FFF7FFFu);
    m[0] = __builtin_elementwise_max(__builtin_elementwise_max(m[0], m[1]), __builtin_elementwise_max(m[2], m[3]));
    const uint32_t m2 = __builtin_bit_cast(uint32_t, m[0]);
    const uint32_t top = mx_quad_max(max(m2 & 0xFFFFu, m2 >> 16));
    uint32_t r = 0u;
    if constexpr (kType == K3MOE_DTYPE_BF16) {
      typedef __bf16 b2 __attribute__((ext_vector_type(2)));
      e = mx_scale_byte(top << 16, saturate);
      const float s = mx_scale_f32(e == 255u ? 127u : e);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(b2, d[0]), s, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(b2, d[1]), s, 1);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(b2, d[2]), s, 2);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(b2, d[3]), s, 3);
    } else {
      typedef _Float16 h2 __attribute__((ext_vector_type(2)));
      const uint16_t t16 = (uint16_t)top;
      e = mx_scale_byte(__float_as_uint((float)__builtin_bit_cast(_Float16, t16)), saturate);
      const float s = mx_scale_f32(e == 255u ? 127u : e);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2, d[0]), s, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2, d[1]), s, 1);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2, d[2]), s, 2);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2, d[3]), s, 3);
    }
    return e == 255u ? 0x77777777u : r;
  }
}

}  // namespace k3moe
