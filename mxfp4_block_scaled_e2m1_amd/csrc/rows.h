// Row-wise helpers of the operators around the experts (moe_rows.hip,
// block_norm.hip, lora.hip): elements of the three activation types as fp32,
// a few at a time, and sums over the lanes of a workgroup.
#pragma once

#include <type_traits>

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

// The element at 64-bit index i: the start of a row, uniform over a wave where i
// is, so that a lane's own 32-bit offset into the row is all it has to hold.
template <int DT>
__device__ __forceinline__ const char* at(const void* p, int64_t i) { return (const char*)p + i * dt_size<DT>; }
template <int DT>
__device__ __forceinline__ char* at(void* p, int64_t i) { return (char*)p + i * dt_size<DT>; }

// The same vector at any element's address: the hardware and its ABI take
// unaligned global accesses, so a row that does not start on 16 bytes still moves 16
// bytes a lane. 4096 rows of bf16, post-norm and channel gate, us per call in a
// graph: 4096 columns 25.9, their gradient 47.7; 4097 columns 40.8 and 75.6 (element
// by element 194 and 680).
typedef uint32_t u32v4_any __attribute__((ext_vector_type(4), aligned(2)));

// N consecutive elements as they lie in memory, at element i of a row: one
// element, or whole 16-byte pieces. AL: the address is a multiple of 16.
// NT: a streaming access, for data that nothing reads again soon.
template <int DT, int N>
struct Raw {
  static constexpr int BYTES = N * dt_size<DT>;
  static constexpr int WORDS = BYTES < 4 ? 1 : BYTES / 4;
  static_assert(N == 1 || BYTES % 16 == 0, "one element or whole pieces");
  uint32_t w[WORDS];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0u;
  }
  // Keeps the packed words where they are: without this the compiler unpacks a
  // loop-invariant row of weights to fp32 ahead of the loop, in twice the registers.
  __device__ __forceinline__ void pin() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) asm volatile("" : "+v"(w[i]));
  }
  template <bool NT = false, bool AL = true>
  __device__ __forceinline__ void load(const void* row, uint32_t i) {
    typedef std::conditional_t<AL, u32v4, u32v4_any> vec;
    const char* p = (const char*)row + i * (uint32_t)dt_size<DT>;
    if constexpr (BYTES == 2) {
      w[0] = NT ? __builtin_nontemporal_load((const uint16_t*)p) : *(const uint16_t*)p;
    } else if constexpr (BYTES == 4) {
      w[0] = NT ? __builtin_nontemporal_load((const uint32_t*)p) : *(const uint32_t*)p;
    } else {
#pragma unroll
      for (int j = 0; j < BYTES / 16; ++j) {
        const u32v4 v = NT ? __builtin_nontemporal_load((const vec*)p + j) : ((const vec*)p)[j];
#pragma unroll
        for (int q = 0; q < 4; ++q) w[4 * j + q] = v[q];
      }
    }
  }
  template <bool NT = false, bool AL = true>
  __device__ __forceinline__ void store(void* row, uint32_t i) const {
    typedef std::conditional_t<AL, u32v4, u32v4_any> vec;
    char* p = (char*)row + i * (uint32_t)dt_size<DT>;
    if constexpr (BYTES == 2) {
      if (NT) __builtin_nontemporal_store((uint16_t)w[0], (uint16_t*)p);
      else *(uint16_t*)p = (uint16_t)w[0];
    } else if constexpr (BYTES == 4) {
      if (NT) __builtin_nontemporal_store(w[0], (uint32_t*)p);
      else *(uint32_t*)p = w[0];
    } else {
#pragma unroll
      for (int j = 0; j < BYTES / 16; ++j) {
        const u32v4 v = {w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]};
        if (NT) __builtin_nontemporal_store((vec)v, (vec*)p + j);
        else ((vec*)p)[j] = v;
      }
    }
  }
  // The piece at column c < H of a row of H >= N elements. A row's last piece may
  // reach past its end (!AL): then the row's last N elements are loaded, and
  // settle(), which has to wait for them, turns them into what the piece has
  // (zeros behind); a store writes these one by one.
  template <bool NT = false, bool AL = true>
  __device__ __forceinline__ void load_row(const void* row, uint32_t c, uint32_t H) {
    load<NT, AL>(row, AL ? c : min(c, H - N));
  }
  template <bool AL>
  __device__ __forceinline__ void settle(uint32_t c, uint32_t H) {
    if constexpr (!AL) {
      if (c + N > H) drop(c + N - H);
    }
  }
  // The first n < N elements leave, zeros come in behind.
  __device__ __forceinline__ void drop(uint32_t n) {
    const uint32_t words = dt_size<DT> == 2 ? n >> 1 : n;
#pragma unroll
    for (int b = 1; b < WORDS; b *= 2)
      if (words & b) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = i + b < WORDS ? w[i + b] : 0u;
      }
    if (dt_size<DT> == 2 && (n & 1)) {
#pragma unroll
      for (int i = 0; i < WORDS; ++i) w[i] = (w[i] >> 16) | (i + 1 < WORDS ? w[i + 1] << 16 : 0u);
    }
  }
  template <bool NT = false, bool AL = true>
  __device__ __forceinline__ void store_row(void* row, uint32_t c, uint32_t H) const {
    if (AL || c + N <= H) {
      store<NT, AL>(row, c);
      return;
    }
#pragma unroll
    for (int j = 0; j < N - 1; ++j)
      if (c + j < H) {
        Raw<DT, 1> e;
        e.w[0] = w[j * dt_size<DT> / 4] >> (j * dt_size<DT> % 4 * 8);
        e.store(row, c + j);
      }
  }
  __device__ __forceinline__ void fill(float x) {
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = x;
    set(f);
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

// v plus v of the lanes that a DPP control names (0 where there is none).
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, ROWS, 0xF, false));
}
// Sum over each row of 16 lanes, in the row's last lane.
__device__ __forceinline__ float row_sum(float v) {
  v = dpp_add<0x111>(v);   // row_shr 1, 2, 4, 8
  v = dpp_add<0x112>(v);
  v = dpp_add<0x114>(v);
  return dpp_add<0x118>(v);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
// Sum over the 64 lanes, uniform over the wave, by DPP adds (lane shuffles go
// through LDS and cost a norm row several times as much).
__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum(v);
  v = dpp_add<0x142, 0xA>(v);   // row_bcast 15: rows 1 and 3 add the row before
  v = dpp_add<0x143, 0xC>(v);   // row_bcast 31: rows 2 and 3 add the first half
  return lane_value(v, 63);
}

// Sums of N values over a group of `waves` (at most 16) waves of the workgroup,
// uniform over the group; `wave` is the thread's wave in its group. All groups
// of the workgroup call this together. red: the group's LDS, N * 16 floats, used
// alternately by the caller (two areas) so that one barrier per sum is enough.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red, int waves, int lane, int wave) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * 16 + wave] = v[i];
  }
  __syncthreads();
  // a row of 16 lanes per value, a lane per wave
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const bool has = (lane & 15) < waves && (lane >> 4) < N - i;
    const float s = row_sum(has ? red[i * 16 + lane] : 0.0f);
#pragma unroll
    for (int j = 0; j < 4 && i + j < N; ++j) v[i + j] = lane_value(s, 16 * j + 15);
  }
}

}  // namespace mx
