// 4-bit codes to 16-bit values, and the operand types of the 16-bit matrix instructions (w4.hip, w4_gemm.hip).
#pragma once

#include "rows.h"

namespace mx {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Two FP8 bytes (E4M3, half H of w) times 2^9 as 16-bit values: the bytes 0 .. 15 are
// the subnormals and the first binade, code * 2^-9, so this is the code itself (with bit 7
// as its sign).
template <int DT, bool H>
__device__ __forceinline__ uint32_t int_pair(uint32_t w) {
  if constexpr (DT == DT_BF16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.0f, H));
  else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 512.0f, H));
}
template <int DT, int SEL>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t w, float scale) {
  if constexpr (DT == DT_BF16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
  else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, SEL));
}

// Eight E2M1 codes (a dword, the low nibble first) times a power of two, in their order.
template <int DT>
__device__ __forceinline__ u32v4 expand_fp4(uint32_t d, float scale) {
  return u32v4{fp4_pair<DT, 0>(d, scale), fp4_pair<DT, 1>(d, scale), fp4_pair<DT, 2>(d, scale), fp4_pair<DT, 3>(d, scale)};
}

// Four codes 0 .. 15 in the bytes of q minus z (replicated), as sign and magnitude: q - z
// + 128 has bit 7 where it is not negative; a negative one is complemented and one
// added, which leaves bit 7 set.
__device__ __forceinline__ uint32_t sign_magnitude(uint32_t q, uint32_t z) {
  const uint32_t v = (q | 0x80808080u) - z;
  const uint32_t neg = ~v & 0x80808080u, one = neg >> 7;
  return (v ^ ((neg - one) | 0x80808080u)) + one;
}

// Eight codes 0 .. 15.
template <int DT>
__device__ __forceinline__ u32v4 expand_code(uint32_t d) {
  const uint32_t lo = d & 0x0F0F0F0Fu, hi = (d >> 4) & 0x0F0F0F0Fu;
  const uint32_t a = __builtin_amdgcn_perm(hi, lo, 0x05010400u), b = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
  return u32v4{int_pair<DT, false>(a), int_pair<DT, true>(a), int_pair<DT, false>(b), int_pair<DT, true>(b)};
}

// A zero point 0 .. 15 as expand_int takes it: four bytes, or two fp16.
template <int DT>
__device__ __forceinline__ uint32_t zero_bits(uint32_t z) {
  if constexpr (DT == DT_F16) return pack2<DT_F16>((float)z, (float)z);
  else return z * 0x01010101u;
}

// Eight codes 0 .. 15 minus their zero point, exact.
template <int DT>
__device__ __forceinline__ u32v4 expand_int(uint32_t d, uint32_t zero) {
  const uint32_t lo = d & 0x0F0F0F0Fu, hi = (d >> 4) & 0x0F0F0F0Fu;
  uint32_t a = __builtin_amdgcn_perm(hi, lo, 0x05010400u), b = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
  if constexpr (DT == DT_BF16) {
    a = sign_magnitude(a, zero);
    b = sign_magnitude(b, zero);
  }
  uint32_t r[4] = {int_pair<DT, false>(a), int_pair<DT, true>(a), int_pair<DT, false>(b), int_pair<DT, true>(b)};
  if constexpr (DT == DT_F16) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, r[i]) - __builtin_bit_cast(f16x2, zero));
  }
  return u32v4{r[0], r[1], r[2], r[3]};
}

__device__ __forceinline__ float e8m0(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7FC00000u) : ldexpf(1.0f, (int)b - 127);
}

}  // namespace mx
