// A paged cache of rows held in MXFP8 or MXFP4: rows quantised as they are
// written, and the rows of sequences read back through their page tables.
//
//   write  the row of slot slots[t] (page slots[t] / page_size, its row slots[t] %
//          page_size) = MXFP8(x[t]) or MXFP4(x[t]): per 32 columns the scale byte
//          max(floor(log2 amax) - emax + 127, 0), emax 8 (E4M3) or 2 (E2M1), and
//          x * 2^(127 - byte) rounded to nearest even, saturating, the sign kept; a
//          block with an infinity or a NaN gets the byte 0xFF and zero codes
//   read   out[r] = code * 2^(byte - 127), r the row of position r - seq_off[b] of
//          sequence b, at page page_table[b, position / page_size]
//
// Both stream rows with next to no arithmetic, so HBM bandwidth bounds them. A lane
// has 8 columns (16 bytes of a 16-bit type, 8 or 4 of codes), four lanes a block of 32:
// a wave's loads and stores are whole contiguous runs, and a block's largest magnitude
// is two DPP exchanges within its four lanes. Measured, in a graph: 128000 rows of 576
// columns read from MXFP8 to bf16 in 47 us (224 MB, 4.7 TB/s; a copy of 512 MB reaches
// 5.2), 8400 rows of 2048 fp16 columns written as MXFP4 in 10.3 and read in 10.2 (44 MB each).
#include <algorithm>

#include "rows.h"

namespace mx {

namespace {

constexpr int CACHE_THREADS = 256;

// The larger magnitude (as bits) of a lane and the lanes that a quad permutation names.
template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0u, v, CTRL, 0xF, 0xF, false));
}

// 8 values of a block, scaled, as codes: 8 bytes (FP8) or 4 (FP4).
template <bool FP8>
__device__ __forceinline__ void encode(const float (&v)[8], float up, uint32_t (&q)[FP8 ? 2 : 1]) {
  if constexpr (FP8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // v_cvt_pk_fp8_f32 rounds to nearest even, subnormals too; what rounds beyond 448 saturates before
      float s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = fminf(fmaxf(v[4 * h + j] * up, -448.0f), 448.0f);
      int d = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
      q[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], d, true);
    }
  } else {
    uint32_t d = 0;
    d = quant_pair_f32_unit<0>(d, v[0] * up, v[1] * up);
    d = quant_pair_f32_unit<1>(d, v[2] * up, v[3] * up);
    d = quant_pair_f32_unit<2>(d, v[4] * up, v[5] * up);
    d = quant_pair_f32_unit<3>(d, v[6] * up, v[7] * up);
    q[0] = d;
  }
}

constexpr int WRITE_AHEAD = 2;     // pieces of a lane that are in flight together

template <int DT, bool FP8>
__global__ __launch_bounds__(CACHE_THREADS) void k_cache_write(const void* __restrict__ x, int64_t ldx,
                                                               const int32_t* __restrict__ slots, uint32_t units,
                                                               uint32_t per_row, uint32_t n_slots,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
  constexpr int EMAX = FP8 ? 8 : 2, BYTES = FP8 ? 8 : 4;
  // whole blocks of 32 columns: per_row and units are multiples of four, so a block's four lanes go together
  for (int64_t u0 = (int64_t)blockIdx.x * (CACHE_THREADS * WRITE_AHEAD) + threadIdx.x; u0 < units;
       u0 += (int64_t)gridDim.x * (CACHE_THREADS * WRITE_AHEAD)) {
    Raw<DT, 8> r[WRITE_AHEAD];
    uint32_t slot[WRITE_AHEAD], col[WRITE_AHEAD];
#pragma unroll
    for (int j = 0; j < WRITE_AHEAD; ++j) {
      const int64_t want = u0 + j * CACHE_THREADS;
      const uint32_t u = (uint32_t)(want < units ? want : u0), t = u / per_row;
      col[j] = u - t * per_row;
      slot[j] = want < units ? (uint32_t)slots[t] : n_slots;
      r[j].load(at<DT>(x, (int64_t)t * ldx), col[j] * 8);
    }
#pragma unroll
    for (int j = 0; j < WRITE_AHEAD; ++j) {
      if (slot[j] >= n_slots) continue;
      const uint32_t c = col[j];
      float v[8];
      uint32_t am = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = r[j].get(i);
        am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      }
      am = quad_max<0xB1>(am);   // quad_perm 1 0 3 2
      am = quad_max<0x4E>(am);   // quad_perm 2 3 0 1
      const int ef = (int)(am >> 23);
      uint32_t sb = (uint32_t)max(ef - EMAX, 0);
      float up = __uint_as_float((254u - sb) << 23);
      if (ef == 0xFF) {
        sb = 0xFFu;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        up = 0.0f;
      }
      uint32_t q[FP8 ? 2 : 1];
      encode<FP8>(v, up, q);
      uint8_t* dst = codes + ((int64_t)slot[j] * per_row + c) * BYTES;
      if constexpr (FP8) *(uint2*)dst = make_uint2(q[0], q[1]);
      else *(uint32_t*)dst = q[0];
      if ((c & 3) == 0) scales[(int64_t)slot[j] * (per_row >> 2) + (c >> 2)] = (uint8_t)sb;
    }
  }
}

// 8 codes times their scale, in the type's own bits.
template <int DT, bool FP8>
__device__ __forceinline__ void decode(const uint32_t (&q)[FP8 ? 2 : 1], uint32_t sb, Raw<DT, 8>& o) {
  const float s = sb == 0xFFu ? __uint_as_float(0x7FC00000u) : e8m0_to_f32(sb);
  float v[8];
  if constexpr (FP8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(q[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(q[h], true);
      v[4 * h] = a[0]; v[4 * h + 1] = a[1]; v[4 * h + 2] = b[0]; v[4 * h + 3] = b[1];
    }
  } else {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.0f, 0),
                b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.0f, 1),
                c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.0f, 2),
                d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.0f, 3);
    v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
    v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= s;
  o.set(v);
}

constexpr int READ_ROWS = 32;      // rows of a workgroup at most
constexpr int READ_AHEAD = 4;      // pieces of a lane whose codes are in flight together

// The sequences that a workgroup's rows are of: offsets 64 at a time narrow down to the last one that starts at or before its
// first row, and those from there on are looked up in LDS, not by a search of dependent loads for each row.
struct Window {
  int64_t first;
  int32_t off[64];
};
__device__ __forceinline__ void find_window(const int32_t* seq_off, int64_t B, int64_t r0, int l, Window& w) {
  int64_t lo = 0, n = B;
  while (n > 64) {
    const int64_t step = (n + 63) / 64;
    const bool before = step * l < n && seq_off[lo + step * l] <= r0;
    const int64_t skip = step * (int64_t)max((int)__popcll(__ballot(before)) - 1, 0);
    lo += skip;
    n = min(step, n - skip);
  }
  const int64_t skip = max((int)__popcll(__ballot(l < n && seq_off[lo + min((int64_t)l, n - 1)] <= r0)) - 1, 0);
  lo += skip;
  w.off[l] = seq_off[min(lo + l, B)];
  if (l == 0) w.first = lo;
}

// `rows_each` rows to a workgroup, as many as READ_AHEAD pieces a lane are (32 whatever the width left 8400 rows of 2048
// columns 262 workgroups: 19 us instead of 10.2; 2 or 8 pieces: 128000 rows of 576 in 53 or 52 us instead of 50). A piece is
// 8 columns: consecutive lanes have consecutive pieces, those of the rows behind one another.
template <int DT, bool FP8>
__global__ __launch_bounds__(CACHE_THREADS) void k_cache_read(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, uint32_t pages,
                                                              uint32_t page_size, uint32_t per_row, int rows_each,
                                                              uint32_t step_row, uint32_t step_col,
                                                              const int32_t* __restrict__ page_table, int64_t table_width,
                                                              const int32_t* __restrict__ seq_off, int64_t B, int64_t rows,
                                                              void* __restrict__ out) {
  constexpr int BYTES = FP8 ? 8 : 4;
  __shared__ int64_t where[READ_ROWS];      // the cache's row of each row; -1: nothing to read, -2: not a sequence's
  __shared__ Window win;
  const uint32_t row0 = threadIdx.x / per_row, col0 = threadIdx.x - row0 * per_row;
  for (int64_t r0 = (int64_t)blockIdx.x * rows_each; r0 < rows; r0 += (int64_t)gridDim.x * rows_each) {
    if (threadIdx.x < 64) {
      const int64_t first = seq_off[0], last = seq_off[B], r = r0 + threadIdx.x;
      find_window(seq_off, B, r0, threadIdx.x, win);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      int64_t at = -2;
      if ((int)threadIdx.x < rows_each && r < rows && r >= first && r < last) {
        int64_t lo = 0, n = min(B - win.first, (int64_t)64);      // the last sequence that starts at or before r
        while (n > 1) {
          const int64_t half = n >> 1;
          if (win.off[lo + half] <= r) { lo += half; n -= half; }
          else n = half;
        }
        int32_t begin = win.off[lo];
        lo += win.first;
        if (lo == win.first + 63) {                               // or one behind the window
          n = B - lo;
          while (n > 1) {
            const int64_t half = n >> 1;
            if (seq_off[lo + half] <= r) { lo += half; n -= half; }
            else n = half;
          }
          begin = seq_off[lo];
        }
        const uint32_t pos = (uint32_t)(r - begin), col = pos / page_size;
        at = -1;
        if ((int64_t)col < table_width) {
          const uint32_t page = (uint32_t)page_table[lo * table_width + col];
          if (page < pages) at = (int64_t)page * page_size + (pos - col * page_size);
        }
      }
      if ((int)threadIdx.x < rows_each) where[threadIdx.x] = at;
    }
    __syncthreads();
    uint32_t row = row0, c = col0;
    while (row < (uint32_t)rows_each) {
      uint32_t q[READ_AHEAD][FP8 ? 2 : 1], sb[READ_AHEAD], cs[READ_AHEAD], rs[READ_AHEAD];
      int64_t w[READ_AHEAD];
#pragma unroll
      for (int j = 0; j < READ_AHEAD; ++j) {
        rs[j] = row;
        cs[j] = c;
        w[j] = row < (uint32_t)rows_each ? where[row] : -2;
        row += step_row;
        c += step_col;
        if (c >= per_row) { c -= per_row; ++row; }
        q[j][0] = 0;
        if constexpr (FP8) q[j][1] = 0;
        sb[j] = 0;
        if (w[j] >= 0) {
          const uint8_t* p = codes + (w[j] * per_row + cs[j]) * BYTES;
          if constexpr (FP8) {
            const uint2 v = *(const uint2*)p;
            q[j][0] = v.x;
            q[j][1] = v.y;
          } else {
            q[j][0] = *(const uint32_t*)p;
          }
          sb[j] = scales[w[j] * (per_row >> 2) + (cs[j] >> 2)];
        }
      }
#pragma unroll
      for (int j = 0; j < READ_AHEAD; ++j) {
        if (w[j] == -2) continue;
        Raw<DT, 8> o;
        decode<DT, FP8>(q[j], sb[j], o);
        o.template store<true>(at<DT>(out, (r0 + rs[j]) * (int64_t)per_row * 8), cs[j] * 8);
      }
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_cache_write(const void* x, DType dt, int64_t ldx, int64_t T, int64_t width, bool fp8,
                              const int32_t* slots, int64_t n_slots, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const uint32_t units = (uint32_t)(T * (width / 8));
  const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)units + CACHE_THREADS * WRITE_AHEAD - 1) /
                                                        (CACHE_THREADS * WRITE_AHEAD), 1 << 20);
  dispatch_dt(dt, [&](auto d) {
    constexpr int D = decltype(d)::value;
    auto* k = fp8 ? k_cache_write<D, true> : k_cache_write<D, false>;
    k<<<grid, CACHE_THREADS, 0, s>>>(x, ldx, slots, units, (uint32_t)(width / 8), (uint32_t)n_slots, codes, scales);
  });
  return hipGetLastError();
}

hipError_t launch_cache_read(const uint8_t* codes, const uint8_t* scales, int64_t pages, int64_t page_size,
                             int64_t width, bool fp8, const int32_t* page_table, int64_t table_width,
                             const int32_t* seq_off, int64_t B, int64_t rows, void* out, DType dt, hipStream_t s) {
  const int64_t per_row = width / 8;
  const int each = (int)std::clamp<int64_t>(CACHE_THREADS * READ_AHEAD / per_row, 1, READ_ROWS);
  const unsigned grid = (unsigned)std::min<int64_t>((rows + each - 1) / each, 1 << 20);
  dispatch_dt(dt, [&](auto d) {
    constexpr int D = decltype(d)::value;
    auto* k = fp8 ? k_cache_read<D, true> : k_cache_read<D, false>;
    k<<<grid, CACHE_THREADS, 0, s>>>(codes, scales, (uint32_t)pages, (uint32_t)page_size, (uint32_t)per_row, each,
                                     (uint32_t)(CACHE_THREADS / per_row), (uint32_t)(CACHE_THREADS % per_row),
                                     page_table, table_width, seq_off, B, rows, out);
  });
  return hipGetLastError();
}

}  // namespace mx
