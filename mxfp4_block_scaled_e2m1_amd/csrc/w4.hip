// Linear layer of unquantised activations with 4-bit weights and group scales:
//   y[t, n] = sum_g scale[n, g] * sum_{c in group g} x[t, c] * (code[n, c] - zero[n, g])
// MXFP4: E2M1 codes, one E8M0 byte per 32 columns, no zero. INT4: codes 0 .. 15, a scale
// of the activations' type and a zero point (8 without) per 32, 64 or 128 columns.
//
// The codes become 16-bit values exactly and enter V_MFMA_F32_16X16X32 as they are; the
// scale multiplies the fp32 sum of 32 columns. So no weight is rounded, and every scale
// that fp32 holds does its work (an MXFP4 scale is far outside fp16, and scale * code of
// INT4 needs 15 bits where bf16 has 8). A zero point z subtracts z times the sum of the
// 32 activations, which one more MFMA with ones gives in the lanes that need it.
#include <algorithm>

#include "w4_expand.h"

namespace mx {

namespace {

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32v4 a, u32v4 b, f32x4 c) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <int DT>
constexpr uint32_t ONES = DT == DT_BF16 ? 0x3F803F80u : 0x3C003C00u;

// Eight codes (a dword, the low nibble first) as 16-bit values in their order.
template <int DT, bool INT>
__device__ __forceinline__ u32v4 expand(uint32_t d) {
  if constexpr (INT) {
    const uint32_t lo = d & 0x0F0F0F0Fu, hi = (d >> 4) & 0x0F0F0F0Fu;
    const uint32_t a = __builtin_amdgcn_perm(hi, lo, 0x05010400u), b = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
    return u32v4{int_pair<DT, false>(a), int_pair<DT, true>(a), int_pair<DT, false>(b), int_pair<DT, true>(b)};
  } else {
    return expand_fp4<DT>(d, 1.0f);
  }
}

// 4 x 4 transposition between the four rows of 16 lanes and four registers: afterwards
// register i of lane row q is what register q of lane row i was.
__device__ __forceinline__ void transpose4(uint32_t (&d)[4]) {
  auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
  auto e = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto f = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  d[0] = e[0]; d[1] = e[1]; d[2] = f[0]; d[3] = f[1];
}

// Scale of a row's 32 columns at block `blk` (columns 32 blk ..).
template <int DT, bool INT>
__device__ __forceinline__ float scale_of(const void* row, int blk, int group_log2) {
  if constexpr (INT) return Raw<DT, 1>{{((const uint16_t*)row)[blk >> (group_log2 - 5)]}}.get(0);
  else return e8m0(((const uint8_t*)row)[blk]);
}

constexpr int W4_WAVES = 8;

// A workgroup has 16 NT weight rows and 16 MT tokens; its waves share K in steps of 128
// columns. Lane (r = lane % 16, q = lane / 16) loads 16 code bytes of row r: columns 32 q
// .. of the step. Four swaps turn them so that MFMA i has the step's columns 32 i .. 32 i +
// 31 and no others, eight of them in each lane: one group's scale is then the lane's own.
template <int DT, bool INT, int NT, int MT>
__global__ __launch_bounds__(64 * W4_WAVES) void k_w4(W4Args a) {
  __shared__ float part[W4_WAVES / 2][NT * MT][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * NT, t0 = (int64_t)blockIdx.y * 16 * MT;
  const int blocks = (int)(a.K / 32), steps = (blocks + 3) / 4;
  const uint8_t* w[NT];
  const uint8_t* sc[NT];
  const uint8_t* zp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t n = min(n0 + 16 * i + r, a.N - 1);
    w[i] = a.w + n * (a.K / 2);
    sc[i] = (const uint8_t*)a.scales + n * (a.K >> a.group_log2) * (INT ? 2 : 1);
    zp[i] = a.zeros + n * (a.K >> a.group_log2);
  }
  const char* x[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) x[i] = at<DT>(a.x, min(t0 + 16 * i + r, a.M - 1) * a.ldx);
  f32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = wave; s < steps; s += W4_WAVES) {
    uint32_t d[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int blk = 4 * s + q < blocks ? 4 * s + q : 4 * s;      // the row's last step may be short
      const u32v4 v = *(const u32v4*)(w[i] + (int64_t)blk * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[i][j] = v[j];
      transpose4(d[i]);
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int blk = 4 * s + b;
      if (blk >= blocks) break;
      u32v4 xv[MT];
#pragma unroll
      for (int j = 0; j < MT; ++j) xv[j] = *(const u32v4*)(x[j] + ((int64_t)blk * 32 + 8 * q) * 2);
      f32x4 sum[MT];
      if constexpr (INT) {
#pragma unroll
        for (int j = 0; j < MT; ++j)
          sum[j] = mfma<DT>(xv[j], u32v4{ONES<DT>, ONES<DT>, ONES<DT>, ONES<DT>}, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const u32v4 wv = expand<DT, INT>(d[i][b]);
        const float scale = scale_of<DT, INT>(sc[i], blk, a.group_log2);
        float zero = 0.0f;
        if constexpr (INT) zero = a.zeros != nullptr ? (float)zp[i][blk >> (a.group_log2 - 5)] : 8.0f;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const f32x4 p = mfma<DT>(xv[j], wv, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][j][e] = fmaf(scale, INT ? fmaf(-zero, sum[j][e], p[e]) : p[e], acc[i][j][e]);
        }
      }
    }
  }
  // the waves' sums, in a tree of fixed order
#pragma unroll
  for (int half = W4_WAVES / 2; half > 0; half >>= 1) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[wave - half][i * MT + j][e][lane] = acc[i][j][e];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] += part[wave][i * MT + j][e][lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
  // lane (r, q) has tokens 4 q + e of weight row r
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t t = t0 + 16 * j + 4 * q + e, n = n0 + 16 * i + r;
        if (t < a.M && n < a.N) {
          Raw<DT, 1> o;
          o.set(&((const float*)&acc[i][j])[e]);
          o.store(at<DT>(a.y, t * a.ldy), (uint32_t)n);
        }
      }
}

}  // namespace

hipError_t launch_w4(const W4Args& a, hipStream_t s) {
  if (a.M > W4_FEW) return launch_w4_gemm(a, s);
  const auto go = [&](auto d, auto in) {
    constexpr int D = decltype(d)::value;
    constexpr bool I = decltype(in)::value;
    const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.M + 63) / 64));
    if (a.M <= 16)
      k_w4<D, I, 1, 1><<<dim3(grid.x, 1), 64 * W4_WAVES, 0, s>>>(a);
    else
      k_w4<D, I, 1, 4><<<grid, 64 * W4_WAVES, 0, s>>>(a);
  };
  if (a.dt == DT_BF16) {
    if (a.int4) go(DtC<DT_BF16>(), std::true_type());
    else go(DtC<DT_BF16>(), std::false_type());
  } else {
    if (a.int4) go(DtC<DT_F16>(), std::true_type());
    else go(DtC<DT_F16>(), std::false_type());
  }
  return hipGetLastError();
}

}  // namespace mx
