// Row-wise helpers of the operators around the experts (moe_rows.hip,
// block_norm.hip, lora.hip): elements of the three activation types as fp32,
// a few at a time, and sums over the lanes of a workgroup.
#pragma once

#include "mx_device.h"
#include "mx_internal.h"

namespace mx {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32v2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32v4 __attribute__((ext_vector_type(4)));

template <int DT> constexpr int dt_size = DT == DT_F32 ? 4 : 2;

// Two fp32 -> two 16-bit elements in a dword, round to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == DT_BF16) return bf16x2_rne(lo, hi);
  else return __builtin_bit_cast(uint32_t, f16x2{(_Float16)lo, (_Float16)hi});
}
template <int DT>
__device__ __forceinline__ float lo_f32(uint32_t w) {
  if constexpr (DT == DT_BF16) return __uint_as_float(w << 16);
  else return (float)__builtin_bit_cast(f16x2, w)[0];
}
template <int DT>
__device__ __forceinline__ float hi_f32(uint32_t w) {
  if constexpr (DT == DT_BF16) return __uint_as_float(w & 0xFFFF0000u);
  else return (float)__builtin_bit_cast(f16x2, w)[1];
}

// N consecutive elements as they lie in memory. N is 1 (any element address)
// or fills whole 16-byte pieces (16-byte aligned address), except N = 4 of a
// 16-bit type: one 8-byte piece.
template <int DT, int N>
struct Raw {
  static constexpr int BYTES = N * dt_size<DT>;
  static constexpr int WORDS = BYTES < 4 ? 1 : BYTES / 4;
  uint32_t w[WORDS];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0u;
  }
  // NT: a streaming access, for data that nothing reads again soon.
  template <bool NT = false>
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const char* p = (const char*)base + i * dt_size<DT>;
    if constexpr (BYTES == 2) {
      w[0] = NT ? __builtin_nontemporal_load((const uint16_t*)p) : *(const uint16_t*)p;
    } else if constexpr (BYTES == 4) {
      w[0] = NT ? __builtin_nontemporal_load((const uint32_t*)p) : *(const uint32_t*)p;
    } else if constexpr (BYTES == 8) {
      const u32v2 v = NT ? __builtin_nontemporal_load((const u32v2*)p) : *(const u32v2*)p;
      w[0] = v[0]; w[1] = v[1];
    } else {
#pragma unroll
      for (int j = 0; j < BYTES / 16; ++j) {
        const u32v4 v = NT ? __builtin_nontemporal_load((const u32v4*)p + j) : ((const u32v4*)p)[j];
#pragma unroll
        for (int q = 0; q < 4; ++q) w[4 * j + q] = v[q];
      }
    }
  }
  template <bool NT = false>
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    char* p = (char*)base + i * dt_size<DT>;
    if constexpr (BYTES == 2) {
      if (NT) __builtin_nontemporal_store((uint16_t)w[0], (uint16_t*)p);
      else *(uint16_t*)p = (uint16_t)w[0];
    } else if constexpr (BYTES == 4) {
      if (NT) __builtin_nontemporal_store(w[0], (uint32_t*)p);
      else *(uint32_t*)p = w[0];
    } else if constexpr (BYTES == 8) {
      const u32v2 v = {w[0], w[1]};
      if (NT) __builtin_nontemporal_store(v, (u32v2*)p);
      else *(u32v2*)p = v;
    } else {
#pragma unroll
      for (int j = 0; j < BYTES / 16; ++j) {
        const u32v4 v = {w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]};
        if (NT) __builtin_nontemporal_store(v, (u32v4*)p + j);
        else ((u32v4*)p)[j] = v;
      }
    }
  }
  __device__ __forceinline__ float get(int i) const {   // i a compile-time constant after unrolling
    if constexpr (DT == DT_F32) return __uint_as_float(w[i]);
    else return (i & 1) ? hi_f32<DT>(w[i >> 1]) : lo_f32<DT>(w[i >> 1]);
  }
  __device__ __forceinline__ void set(const float* f) {
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (N == 1) {
      w[0] = pack2<DT>(f[0], 0.0f) & 0xFFFFu;
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) w[i] = pack2<DT>(f[2 * i], f[2 * i + 1]);
    }
  }
};

// Sum over the 64 lanes, in every lane (xor butterfly: the same order always).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Sums of N values over the `waves` waves of the workgroup, in every thread.
// red: LDS, N * 16 floats, used alternately by the caller (two areas) so that
// one barrier per sum is enough.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red, int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * 16 + wave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.0f;
    for (int w = 0; w < waves; ++w) s += red[i * 16 + w];
    v[i] = s;
  }
}

}  // namespace mx
