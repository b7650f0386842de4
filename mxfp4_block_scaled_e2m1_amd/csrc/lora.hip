// Low-rank adapters of many requests on top of a shared projection:
//   y[t] += scale_a * B_a (A_a x[t])      a = the adapter of token t, or none
// with A_a [R, K], B_a [N, R]. Tokens arrive sorted by adapter (route.hip), so
// that a tile of sorted rows shares its A and B.
//
// Two launches. Shrink forms v = A x in fp32, the K axis split over the waves
// of a workgroup (joined in LDS) and over workgroups (partial sums in the
// workspace, joined by the second launch in split order: no atomics). Expand
// adds B v to y. The arithmetic, 2 R (K + N) flops per token, is small next to
// moving x, y and the adapters in use, so both are bound by memory: by HBM for
// prompts, by latency for a few tokens.
//
// v stays fp32-accurate: for the matrix unit each value is split into two
// 16-bit halves, hi + lo, after a power-of-two scaling of the token's row
// (rounding v to one bf16 would be off by up to 2^-9 of every product, and fp16 could
// overflow); the second product costs no memory traffic. y is rounded once.
#include <algorithm>
#include <type_traits>

#include "rows.h"

namespace mx {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int LORA_WAVES = 4;

template <int DT>
__device__ __forceinline__ f32x4 mma(u32v4 a, u32v4 b, f32x4 c) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

struct Tile {
  int adapter, row0, rows;   // sorted rows [row0, row0 + rows) of one adapter; adapter < 0: no such tile
};

// The tile-th tile of up to TM sorted rows, adapters in order: 64 adapters at a
// time, a prefix sum of their tile counts over the lanes.
template <int TM>
__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ off, int n, int M, int tile) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int a0 = 0; a0 < n; a0 += 64) {
    const int a = a0 + lane;
    int lo = 0, hi = 0;
    if (a < n) {
      lo = min(max(off[a], 0), M);
      hi = min(max(off[a + 1], lo), M);
    }
    const int cnt = (hi - lo + TM - 1) / TM;
    int inc = cnt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(inc, d);
      if (lane >= d) inc += u;
    }
    const uint64_t hit = __ballot(before + inc > tile);
    if (hit) {
      const int l = __ffsll((long long)hit) - 1;
      const int first = before + __builtin_amdgcn_readlane(inc, l) - __builtin_amdgcn_readlane(cnt, l);
      const int row0 = __builtin_amdgcn_readlane(lo, l) + (tile - first) * TM;
      return {a0 + l, row0, min(TM, __builtin_amdgcn_readlane(hi, l) - row0)};
    }
    before += __builtin_amdgcn_readlane(inc, 63);
  }
  return {-1, 0, 0};
}

// v [split][sorted row][R] of one tile: MT x RT blocks of 16 tokens x 16 ranks.
// Grid: tile, K split, group of 16 RT ranks.
template <int DT, int MT, int RT>
__global__ __launch_bounds__(64 * LORA_WAVES) void k_lora_shrink(LoraArgs p) {
  constexpr int TM = 16 * MT;
  __shared__ f32x4 sh[LORA_WAVES][MT * RT][64];
  const Tile tile = find_tile<TM>(p.adapter_off, p.n, p.M, blockIdx.x);
  if (tile.adapter < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.y, r0 = blockIdx.z * 16 * RT;
  const int c = lane & 15, q8 = (lane >> 4) * 8;
  // rows past the tile or the rank repeat the last one; their results are not kept
  const uint16_t* xr[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = tile.row0 + min(m * 16 + c, tile.rows - 1);
    const int tok = min(max(p.row_token[row], 0), p.M - 1);
    xr[m] = (const uint16_t*)p.x + (int64_t)tok * p.ldx + q8;
  }
  const uint16_t* ar[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
    ar[r] = (const uint16_t*)p.a + ((int64_t)tile.adapter * p.R + min(r0 + r * 16 + c, p.R - 1)) * p.K + q8;
  f32x4 acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[m][r] = f32x4{0.f, 0.f, 0.f, 0.f};
  // the 32-wide K steps, split evenly over (split, wave)
  const int steps = (p.K + 31) / 32, parts = p.splits * LORA_WAVES, part = split * LORA_WAVES + wave;
  const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
  for (int s = s0; s < s1; ++s) {
    const int k = s * 32;
    const bool in = k + q8 < p.K;      // K % 8 == 0: a lane's eight elements are in or out
    u32v4 xv[MT], av[RT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xv[m] = in ? *(const u32v4*)(xr[m] + k) : u32v4{0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < RT; ++r) av[r] = in ? *(const u32v4*)(ar[r] + k) : u32v4{0, 0, 0, 0};
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[m][r] = mma<DT>(av[r], xv[m], acc[m][r]);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r) sh[wave][m * RT + r][lane] = acc[m][r];
  __syncthreads();
  // block b of the tile: lane l holds ranks 4 (l / 16) .. + 3 of token l % 16
  float* out = p.part + (int64_t)split * p.M * p.R;
  for (int i = threadIdx.x; i < MT * RT * 64; i += 64 * LORA_WAVES) {
    const int b = i >> 6, l = i & 63;
    f32x4 v = sh[0][b][l];
#pragma unroll
    for (int w = 1; w < LORA_WAVES; ++w) v += sh[w][b][l];
    const int row = (b / RT) * 16 + (l & 15), r = r0 + (b % RT) * 16 + (l >> 4) * 4;
    if (row < tile.rows && r < p.R) *(f32x4*)(out + (int64_t)(tile.row0 + row) * p.R + r) = v;
  }
}

// y += scale B v of one tile. A wave takes 64 columns at a time as four
// matrix products of 16 columns each, column 16 (i / 4) + 4 f + i % 4 as row i
// of product f, so that a lane ends up with 16 consecutive columns of a token.
// Grid: tile, run of column groups.
template <int DT, int MT>
__global__ __launch_bounds__(64 * LORA_WAVES) void k_lora_expand(LoraArgs p) {
  constexpr int TM = 16 * MT;
  extern __shared__ uint32_t lds[];
  const Tile tile = find_tile<TM>(p.adapter_off, p.n, p.M, blockIdx.x);
  if (tile.adapter < 0) return;
  const int Rp = (p.R + 31) / 32 * 32, pitch = Rp + 8;     // 16-bit elements; the pad spreads the banks
  uint16_t* vh = (uint16_t*)lds;                            // [TM][pitch] hi
  uint16_t* vl = vh + TM * pitch;                           // [TM][pitch] lo
  float* fac = (float*)(vl + TM * pitch);                   // [TM] scale * 2^e
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float scale = p.scale != nullptr ? p.scale[tile.adapter] : 1.0f;
  for (int row = wave; row < TM; row += LORA_WAVES) {
    float v[LORA_MAX_RANK / 64];
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < LORA_MAX_RANK / 64; ++j) {
      const int r = j * 64 + lane;
      v[j] = 0.0f;
      if (r < p.R && row < tile.rows)
        for (int s = 0; s < p.splits; ++s) v[j] += p.part[((int64_t)s * p.M + tile.row0 + row) * p.R + r];
      amax = fmaxf(amax, fabsf(v[j]));
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
    // 2^-e with 2^e the exponent of the row's largest value, where that is an ordinary number
    const uint32_t ex = __float_as_uint(amax) >> 23;
    const bool plain = ex >= 2 && ex <= 252;
    const float down = plain ? __uint_as_float((254u - ex) << 23) : 1.0f;
    const float up = plain ? __uint_as_float(ex << 23) : 1.0f;
#pragma unroll
    for (int j = 0; j < LORA_MAX_RANK / 64; ++j) {
      const int r = j * 64 + lane;
      if (r < Rp) {
        const float u = v[j] * down;
        const uint32_t h = pack2<DT>(u, 0.0f);
        const float hf = lo_f32<DT>(h);
        const float rest = fabsf(hf) < INFINITY ? u - hf : 0.0f;   // an inf or NaN travels in hi alone
        vh[row * pitch + r] = (uint16_t)h;
        vl[row * pitch + r] = (uint16_t)pack2<DT>(rest, 0.0f);
      }
    }
    if (lane == 0) fac[row] = scale * up;
  }
  __syncthreads();
  const int c = lane & 15, q = lane >> 4;
  const uint16_t* bm = (const uint16_t*)p.b + (int64_t)tile.adapter * p.N * p.R;
  const int groups = (p.N + 63) / 64;                       // of 64 columns
  const int g0 = (int)((int64_t)groups * blockIdx.y / gridDim.y), g1 = (int)((int64_t)groups * (blockIdx.y + 1) / gridDim.y);
  int64_t yrow[MT];
  float f[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = m * 16 + c;
    const int tok = row < tile.rows ? p.row_token[tile.row0 + row] : -1;
    yrow[m] = (unsigned)tok < (unsigned)p.M ? (int64_t)tok * p.ldy : -1;
    f[m] = fac[row];
  }
  for (int g = g0 + wave; g < g1; g += LORA_WAVES) {
    const int n0 = g * 64;
    f32x4 acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < Rp; k += 32) {
      u32v4 bv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = min(n0 + 16 * (c >> 2) + 4 * j + (c & 3), p.N - 1);
        bv[j] = k + q * 8 < p.R ? *(const u32v4*)(bm + (int64_t)n * p.R + k + q * 8) : u32v4{0, 0, 0, 0};
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int at = (m * 16 + c) * pitch + k + q * 8;
        const u32v4 h = *(const u32v4*)(vh + at), l = *(const u32v4*)(vl + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[m][j] = mma<DT>(bv[j], l, acc[m][j]);
          acc[m][j] = mma<DT>(bv[j], h, acc[m][j]);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (yrow[m] < 0) continue;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int n = n0 + 16 * q + 8 * half;
        if (n >= p.N) continue;        // N % 8 == 0
        Raw<DT, 8> y;
        y.load(at<DT>(p.y, yrow[m]), n);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = fmaf(f[m], acc[m][2 * half + (i >> 2)][i & 3], y.get(i));
        y.set(o);
        y.store(at<DT>(p.y, yrow[m]), n);
      }
    }
  }
}

// Sorted rows per tile: 64 where adapters have many rows each, else 16 (a tile
// holds one adapter's rows, so more would mostly be padding).
int lora_mt(int64_t M, int n) { return M >= 32 * (int64_t)std::min<int64_t>(n, M) && M >= 64 ? 4 : 1; }
int lora_tiles(int64_t M, int n, int mt) {
  return (int)(M / (16 * mt) + std::min<int64_t>(n, M));
}

}  // namespace

// K splits of the shrink: about two workgroups per compute unit of an MI355X,
// each wave at least two 32-wide steps.
int lora_splits(int64_t M, int64_t K, int R, int n) {
  const int mt = lora_mt(M, n);
  const int64_t tiles = (M + 16 * mt - 1) / (16 * mt);
  const int64_t groups = (R + 63) / 64;
  int64_t s = 512 / std::max<int64_t>(1, tiles * groups);
  s = std::min<int64_t>(s, (K + 31) / 32 / (2 * LORA_WAVES));
  return (int)std::max<int64_t>(1, std::min<int64_t>(s, 16));
}

hipError_t launch_lora_shrink(const LoraArgs& p, hipStream_t s) {
  const int mt = lora_mt(p.M, p.n);
  const int rt = p.R <= 16 ? 1 : p.R <= 32 ? 2 : 4;
  const dim3 grid((unsigned)lora_tiles(p.M, p.n, mt), (unsigned)p.splits, (unsigned)((p.R + 16 * rt - 1) / (16 * rt)));
  auto go = [&](auto d, auto m, auto r) {
    k_lora_shrink<decltype(d)::value, decltype(m)::value, decltype(r)::value><<<grid, 64 * LORA_WAVES, 0, s>>>(p);
  };
  auto by_rt = [&](auto d, auto m) {
    if (rt == 1) go(d, m, std::integral_constant<int, 1>());
    else if (rt == 2) go(d, m, std::integral_constant<int, 2>());
    else go(d, m, std::integral_constant<int, 4>());
  };
  auto by_mt = [&](auto d) {
    if (mt == 1) by_rt(d, std::integral_constant<int, 1>());
    else by_rt(d, std::integral_constant<int, 4>());
  };
  if (p.dt == DT_BF16) by_mt(DtC<DT_BF16>());
  else by_mt(DtC<DT_F16>());
  return hipGetLastError();
}

hipError_t launch_lora_expand(const LoraArgs& p, hipStream_t s) {
  const int mt = lora_mt(p.M, p.n), tm = 16 * mt;
  const int tiles = lora_tiles(p.M, p.n, mt);
  const int groups = (p.N + 63) / 64;
  const int runs = std::max(1, std::min((groups + LORA_WAVES - 1) / LORA_WAVES, 1024 / std::max(1, (int)(p.M + tm - 1) / tm)));
  const int Rp = (p.R + 31) / 32 * 32;
  const size_t lds = (size_t)tm * (Rp + 8) * 4 + tm * 4;
  const dim3 grid((unsigned)tiles, (unsigned)runs);
  auto go = [&](auto d) {
    if (mt == 1) k_lora_expand<decltype(d)::value, 1><<<grid, 64 * LORA_WAVES, lds, s>>>(p);
    else k_lora_expand<decltype(d)::value, 4><<<grid, 64 * LORA_WAVES, lds, s>>>(p);
  };
  if (p.dt == DT_BF16) go(DtC<DT_BF16>());
  else go(DtC<DT_F16>());
  return hipGetLastError();
}

}  // namespace mx
