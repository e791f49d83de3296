// Device helpers of the weight-streaming kernels (decode-sized batches): the
// decode of staged MXFP4 blocks into bf16 operands, and waits for loads in
// flight.
#pragma once

#include "k3moe_internal.h"

namespace k3moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float e8m0_to_f32(uint32_t e) { return __uint_as_float(e ? (e << 23) : 0x00400000u); }

__device__ __forceinline__ bf16x8_t decode_dword(uint32_t q, float sf) {
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sf, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sf, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sf, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sf, 3));
  return __builtin_bit_cast(bf16x8_t, r);
}

__device__ __forceinline__ uint32_t f32_to_bf16_bits(float f) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);
}

// Block (4*rnd + g) of a staged row: four bf16x8 operands (P-order
// positions 8i..8i+7, i = 0..3) from the five dwords d[0..4] (LDS dwords
// 17*rnd + 4*g .. +4 of the row).  The block starts at byte g of d[0], so its
// exponent is byte g and its qs dword i is bytes g+1+4i .. g+4+4i, picked out
// of two neighbouring dwords with v_perm.
__device__ __forceinline__ void decode_dwords(const uint32_t (&d)[5], int g, uint32_t qsel, bf16x8_t op[4]) {
  const float sf = e8m0_to_f32(__builtin_amdgcn_ubfe(d[0], 8 * g, 8));
  op[0] = decode_dword(__builtin_amdgcn_perm(d[1], d[0], qsel), sf);
  op[1] = decode_dword(__builtin_amdgcn_perm(d[2], d[1], qsel), sf);
  op[2] = decode_dword(__builtin_amdgcn_perm(d[3], d[2], qsel), sf);
  op[3] = decode_dword(__builtin_amdgcn_perm(d[4], d[3], qsel), sf);
}

// Tile list and token map are read through the constant address space so that
// the wave-uniform reads become scalar loads: a vector load would have to be
// waited for with the global -> LDS loads still in flight ahead of it.
template <typename T_>
__device__ __forceinline__ const __attribute__((address_space(4))) T_* as_const(const T_* p) {
  return reinterpret_cast<const __attribute__((address_space(4))) T_*>(reinterpret_cast<uintptr_t>(p));
}

// s_waitcnt vmcnt(N): at most N of this wave's vector-memory operations
// outstanding.  Loads complete in issue order, so after the wait every load
// issued before the newest N has landed (in LDS, for the global -> LDS loads).
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// The same with N = kBase + b, b (0..16) known only at run time.
template <int kBase>
__device__ __forceinline__ void wait_vm_plus(int b) {
  switch (b) {
#define K3_CASE(v) \
  case v: wait_vm<kBase + v>(); break;
    K3_CASE(0) K3_CASE(1) K3_CASE(2) K3_CASE(3) K3_CASE(4) K3_CASE(5) K3_CASE(6) K3_CASE(7) K3_CASE(8)
    K3_CASE(9) K3_CASE(10) K3_CASE(11) K3_CASE(12) K3_CASE(13) K3_CASE(14) K3_CASE(15) K3_CASE(16)
#undef K3_CASE
    default: wait_vm<0>(); break;
  }
}

}  // namespace
}  // namespace k3moe
