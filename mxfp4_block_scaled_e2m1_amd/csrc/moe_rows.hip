// Rows to the experts and back: the caller-visible form of the permute and the
// weighted combine that the routed MLP fuses, with the gradient.
//
// With row(t, j) the row of slot j of token t in expert order (-1: the slot's
// expert is on another rank; see route.hip for the sort):
//   permute          xs[row(t, j)] = x[t]
//   unpermute        y[t]  = sum_j w[t, j] ys[row(t, j)]      (w = 1 without weights)
//   unpermute grad   dys[row(t, j)] = w[t, j] dy[t],  dw[t, j] = <dy[t], ys[row(t, j)]>
// and the gradient of the permute is the unweighted unpermute of dxs.
//
// All of them move rows of `hidden` elements and do next to no arithmetic: HBM
// bandwidth bounds them. Each kernel is token-major, so that a token's own row
// is read (or written) once and its k rows once each; a wave owns 64 pieces of
// 16 bytes of one token, which makes the slot's row and weight uniform over the
// wave (scalar loads, and a skipped slot costs no vector load). Rows that no
// slot names are neither read nor written. No atomics: the sums run in slot
// order, so results do not vary between runs. The k-fold side is read and
// written with streaming accesses. 4096 tokens x 8 slots x 7168 bf16: permute
// 104.8 -> 93 us with them (529 MB, 5.7 TB/s), unpermute 103.6 -> 89.7 us
// (5.9 TB/s), gradient 202 -> 182 us (999 MB, 5.5 TB/s); a copy reaches
// 5.4 to 5.7 TB/s on this card.
#include <algorithm>
#include <type_traits>

#include "rows.h"

namespace mx {

namespace {

constexpr int MR_WAVES = 4;          // waves per workgroup of the wave-per-segment kernels
constexpr int SLOT_BATCH = 8;        // slots whose rows are in flight together

// The wave's first (token, segment) unit; the others follow a grid apart.
__device__ __forceinline__ int64_t first_unit() {
  return (int64_t)blockIdx.x * MR_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// One wave per (token, segment of 64 pieces). DT: a type of the elements' size.
// Streaming stores only of whole lines (2048 x 8 x 4097 bf16: 46 us with, 40 without).
template <int DT, int N, bool AL>
__global__ __launch_bounds__(64 * MR_WAVES) void k_permute(const void* __restrict__ x, int64_t T, int k, int H,
                                                           int segs, const int32_t* __restrict__ slot_row,
                                                           int64_t rows, void* __restrict__ xs) {
  for (int64_t unit = first_unit(); unit < T * segs; unit += (int64_t)gridDim.x * MR_WAVES) {
    const int64_t t = unit / segs;
    const int c = ((int)(unit - t * segs) * 64 + (threadIdx.x & 63)) * N;
    if (c >= H) continue;
    Raw<DT, N> v;
    v.template load_row<false, AL>(at<DT>(x, t * H), c, H);
    v.template settle<AL>(c, H);
    for (int j = 0; j < k; ++j) {
      const int r = slot_row[t * k + j];
      if ((unsigned)r < (unsigned)rows) v.template store_row<AL, AL>(at<DT>(xs, (int64_t)r * H), c, H);
    }
  }
}

template <int DT, int N, bool AL>
__global__ __launch_bounds__(64 * MR_WAVES) void k_unpermute(const void* __restrict__ ys, int64_t rows,
                                                             const int32_t* __restrict__ slot_row,
                                                             const float* __restrict__ w, int64_t T, int k, int H,
                                                             int segs, void* __restrict__ y) {
  for (int64_t unit = first_unit(); unit < T * segs; unit += (int64_t)gridDim.x * MR_WAVES) {
    const int64_t t = unit / segs;
    const int c = ((int)(unit - t * segs) * 64 + (threadIdx.x & 63)) * N;
    if (c >= H) continue;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += SLOT_BATCH) {
      Raw<DT, N> v[SLOT_BATCH];
      float wt[SLOT_BATCH];
#pragma unroll
      for (int q = 0; q < SLOT_BATCH; ++q) {
        const int r = j0 + q < k ? slot_row[t * k + j0 + q] : -1;
        wt[q] = 0.0f;
        v[q].zero();
        if ((unsigned)r < (unsigned)rows) {
          wt[q] = w != nullptr ? w[t * k + j0 + q] : 1.0f;
          v[q].template load_row<true, AL>(at<DT>(ys, (int64_t)r * H), c, H);
        }
      }
#pragma unroll
      for (int q = 0; q < SLOT_BATCH; ++q) {
        v[q].template settle<AL>(c, H);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(wt[q], v[q].get(i), acc[i]);
      }
    }
    Raw<DT, N> o;
    o.set(acc);
    o.template store_row<true, AL>(at<DT>(y, t * H), c, H);
  }
}

// One workgroup per token: its dy pieces stay in registers while the rows of
// up to SLOT_BATCH slots stream by; the dot products are summed over the lanes
// and waves at the end.
template <int DT, int N, bool AL>
__global__ __launch_bounds__(1024) void k_unpermute_grad(const void* __restrict__ dy, const void* __restrict__ ys,
                                                         int64_t rows, const int32_t* __restrict__ slot_row,
                                                         const float* __restrict__ w, int64_t T, int k, int H,
                                                         void* __restrict__ dys, float* __restrict__ dw) {
  __shared__ float red[SLOT_BATCH * 16];
  const int waves = blockDim.x >> 6;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    for (int j0 = 0; j0 < k; j0 += SLOT_BATCH) {
      int row[SLOT_BATCH];
      float wt[SLOT_BATCH], dot[SLOT_BATCH];
#pragma unroll
      for (int q = 0; q < SLOT_BATCH; ++q) {
        row[q] = j0 + q < k ? slot_row[t * k + j0 + q] : -1;
        if ((unsigned)row[q] >= (unsigned)rows) row[q] = -1;
        wt[q] = row[q] >= 0 ? w[t * k + j0 + q] : 0.0f;
        dot[q] = 0.0f;
      }
      for (int c = threadIdx.x * N; c < H; c += blockDim.x * N) {
        Raw<DT, N> d, v[SLOT_BATCH];
        d.template load_row<false, AL>(at<DT>(dy, t * H), c, H);
#pragma unroll
        for (int q = 0; q < SLOT_BATCH; ++q)
          if (row[q] >= 0) v[q].template load_row<true, AL>(at<DT>(ys, (int64_t)row[q] * H), c, H);
        d.template settle<AL>(c, H);
#pragma unroll
        for (int q = 0; q < SLOT_BATCH; ++q) {
          if (row[q] < 0) continue;
          v[q].template settle<AL>(c, H);
          float o[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float g = d.get(i);
            dot[q] = fmaf(g, v[q].get(i), dot[q]);
            o[i] = wt[q] * g;
          }
          Raw<DT, N> r;
          r.set(o);
          r.template store_row<true, AL>(at<DT>(dys, (int64_t)row[q] * H), c, H);
        }
      }
      group_sum<SLOT_BATCH>(dot, red, waves, threadIdx.x & 63, threadIdx.x >> 6);
      if (threadIdx.x == 0) {
#pragma unroll
        for (int q = 0; q < SLOT_BATCH; ++q)
          if (j0 + q < k) dw[t * k + j0 + q] = row[q] >= 0 ? dot[q] : 0.0f;
      }
      __syncthreads();   // red is free again
    }
  }
}

bool rows_aligned(int64_t row_bytes, const void* a, const void* b, const void* c = nullptr) {
  return row_bytes % 16 == 0 && (((uintptr_t)a | (uintptr_t)b | (uintptr_t)c) & 15) == 0;
}

// Longer launches stride over their units (a grid holds below 2^32 threads).
constexpr int64_t MAX_GRID = (int64_t)1 << 20;
unsigned wave_grid(int64_t units) { return (unsigned)std::min((units + MR_WAVES - 1) / MR_WAVES, MAX_GRID); }


// f(type, elements of a 16-byte piece, aligned)
template <class F>
void dispatch_piece(DType dt, int H, bool aligned, F&& f) {
  dispatch_dt(dt, [&](auto d) {
    std::integral_constant<int, 16 / dt_size<decltype(d)::value>> n;
    if (H < n) f(d, std::integral_constant<int, 1>(), std::true_type());   // no whole piece
    else if (aligned) f(d, n, std::true_type());
    else f(d, n, std::false_type());
  });
}

int segments(int H, int N) { return (H + 64 * N - 1) / (64 * N); }

}  // namespace

hipError_t launch_permute(const void* x, DType dt, int64_t T, int k, int H, const int32_t* slot_row, int64_t rows,
                          void* xs, hipStream_t s) {
  if (dt == DT_F16) dt = DT_BF16;          // elements are moved as they are
  dispatch_piece(dt, H, rows_aligned((int64_t)H * dt_bytes(dt), x, xs), [&](auto d, auto n, auto al) {
    constexpr int D = decltype(d)::value, N = decltype(n)::value;
    const int segs = segments(H, N);
    if constexpr (D != DT_F16)
      k_permute<D, N, decltype(al)::value><<<wave_grid(T * segs), 64 * MR_WAVES, 0, s>>>(x, T, k, H, segs, slot_row,
                                                                                        rows, xs);
  });
  return hipGetLastError();
}

hipError_t launch_unpermute(const void* ys, DType dt, int64_t rows, const int32_t* slot_row, const float* w,
                            int64_t T, int k, int H, void* y, hipStream_t s) {
  dispatch_piece(dt, H, rows_aligned((int64_t)H * dt_bytes(dt), ys, y), [&](auto d, auto n, auto al) {
    constexpr int D = decltype(d)::value, N = decltype(n)::value;
    const int segs = segments(H, N);
    k_unpermute<D, N, decltype(al)::value><<<wave_grid(T * segs), 64 * MR_WAVES, 0, s>>>(ys, rows, slot_row, w, T, k,
                                                                                        H, segs, y);
  });
  return hipGetLastError();
}

hipError_t launch_unpermute_grad(const void* dy, const void* ys, DType dt, int64_t rows, const int32_t* slot_row,
                                 const float* w, int64_t T, int k, int H, void* dys, float* dw, hipStream_t s) {
  dispatch_piece(dt, H, rows_aligned((int64_t)H * dt_bytes(dt), ys, dy, dys), [&](auto d, auto n, auto al) {
    constexpr int D = decltype(d)::value, N = decltype(n)::value;
    // a wave for every 64 pieces of the row: fewer waves with more pieces each were slower (14, 7, 4
    // and 2 waves, 7168 bf16: 182, 186, 187 and 192 us)
    const int waves = std::min(16, segments(H, N));
    k_unpermute_grad<D, N, decltype(al)::value><<<(unsigned)std::min<int64_t>(T, MAX_GRID), 64 * waves, 0, s>>>(
        dy, ys, rows, slot_row, w, T, k, H, dys, dw);
  });
  return hipGetLastError();
}

}  // namespace mx
