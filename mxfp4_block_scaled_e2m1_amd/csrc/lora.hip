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

constexpr int SHRINK_WAVES = 4;   // waves of a shrink workgroup, which split its K range
constexpr int EXPAND_WAVES = 4;   // waves of an expand workgroup, which split its columns

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
  int adapter, row0, rows;   // sorted rows [row0, row0 + rows) of one adapter; adapter < 0: none
  int piece;                 // which of the tile's `pieces` workgroups this is
};

// The tile of workgroup `id`, of `pieces` workgroups per tile. A tile is up to TM
// sorted rows of one adapter, adapters in order; how many there are is only known
// here, so workgroups past the last one get none. Neighbouring tiles mostly share
// an adapter, and workgroups go to the 8 XCDs in turn, so each XCD is given a
// contiguous run of the work: its L2 then holds a few adapters instead of all
// (8 adapters of 64 x 7168 beside 4096 tokens: 7.3 MB, more than its 4 MB).
template <int TM>
__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ off, int n, int M, int id, int pieces) {
  const int lane = threadIdx.x & 63;
  // 64 adapters at a time: a prefix sum of their tile counts over the lanes
  auto chunk = [&](int a0, int& lo, int& hi, int& cnt) {
    const int a = a0 + lane;
    lo = hi = 0;
    if (a < n) {
      lo = min(max(off[a], 0), M);
      hi = min(max(off[a + 1], lo), M);
    }
    cnt = (hi - lo + TM - 1) / TM;
    int inc = cnt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(inc, d);
      if (lane >= d) inc += u;
    }
    return inc;
  };
  int lo, hi, cnt, inc = chunk(0, lo, hi, cnt);
  int total = __builtin_amdgcn_readlane(inc, 63);
  for (int a0 = 64; a0 < n; a0 += 64) total += __builtin_amdgcn_readlane(chunk(a0, lo, hi, cnt), 63);
  const int work = total * pieces;
  if (id >= work) return {-1, 0, 0, 0};
  const int xcd = id & 7, mine = (work >> 3) * xcd + min(xcd, work & 7) + (id >> 3);
  const int tile = mine / pieces;
  int before = 0;
  for (int a0 = 0; a0 < n; a0 += 64) {
    if (n > 64) inc = chunk(a0, lo, hi, cnt);
    const uint64_t hit = __ballot(before + inc > tile);
    if (hit) {
      const int l = __ffsll((long long)hit) - 1;
      const int first = before + __builtin_amdgcn_readlane(inc, l) - __builtin_amdgcn_readlane(cnt, l);
      const int row0 = __builtin_amdgcn_readlane(lo, l) + (tile - first) * TM;
      return {a0 + l, row0, min(TM, __builtin_amdgcn_readlane(hi, l) - row0), mine - tile * pieces};
    }
    before += __builtin_amdgcn_readlane(inc, 63);
  }
  return {-1, 0, 0, 0};
}

// Between the lanes of one wave: LDS writes before, reads after.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// v [split][sorted row][R] of one tile: MT x RT blocks of 16 tokens x 16 ranks.
// A matrix operand wants 16 rows side by side in the lanes, but a load whose
// neighbouring lanes are in different rows takes the address path one row at a time
// (4096 x 7168, rank 64: 39 us that way even with x in L2). So a wave loads whole
// 128-byte lines, eight lanes each, the rows of a 64-wide step of K, turns them
// in an LDS area of its own (pitch 144: conflict-free) and has the next
// two steps' loads in flight meanwhile. The waves take the steps of a split in turn,
// 1 KB of a row together, and join their sums in LDS.
// Workgroups of a tile: K splits by groups of 16 RT ranks.
constexpr int SHRINK_PITCH = 128 + 16;
template <int DT, int MT, int RT>
__global__ __launch_bounds__(64 * SHRINK_WAVES) void k_lora_shrink(LoraArgs p) {
  constexpr int TM = 16 * MT, XI = 2 * MT, AI = 2 * RT;      // loads of eight rows: of x, of A
  constexpr int AREA = 16 * (MT + RT) * SHRINK_PITCH;
  constexpr int JOIN = MT * RT * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t lds[SHRINK_WAVES * (AREA > JOIN ? AREA : JOIN)];
  const int rgroups = (p.R + 16 * RT - 1) / (16 * RT);
  const Tile tile = find_tile<TM>(p.adapter_off, p.n, p.M, blockIdx.x, p.splits * rgroups);
  if (tile.adapter < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = tile.piece / rgroups, r0 = (tile.piece - split * rgroups) * 16 * RT;
  const int lrow = lane >> 3, lcol = (lane & 7) * 8;          // of a load
  // rows past the tile or the rank repeat the last one; their results are not kept
  int tok[XI];
#pragma unroll
  for (int i = 0; i < XI; ++i) tok[i] = p.row_token[tile.row0 + min(8 * i + lrow, tile.rows - 1)];
  const uint16_t* am = (const uint16_t*)p.a + (int64_t)tile.adapter * p.R * p.K;
  uint32_t ao[AI];
#pragma unroll
  for (int i = 0; i < AI; ++i) ao[i] = (uint32_t)min(r0 + 8 * i + lrow, p.R - 1) * (uint32_t)p.K + lcol;
  f32x4 acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[m][r] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Step {
    u32v4 a[AI], x[XI];
  };
  const uint16_t* xr[XI];
  auto fetch_a = [&](Step& f, int k) {
#pragma unroll
    for (int i = 0; i < AI; ++i) f.a[i] = *(const u32v4*)(am + k + ao[i]);
  };
  auto fetch_x = [&](Step& f, int k) {
#pragma unroll
    for (int i = 0; i < XI; ++i) f.x[i] = __builtin_nontemporal_load((const u32v4*)(xr[i] + k));
  };
  uint8_t* area = lds + wave * AREA;
  uint8_t* put = area + lrow * SHRINK_PITCH + lcol * 2;
  const uint8_t* get = area + (lane & 15) * SHRINK_PITCH + (lane >> 4) * 16;
  auto stage = [&](const Step& f) {
    wave_sync();
#pragma unroll
    for (int i = 0; i < XI; ++i) *(u32v4*)(put + 8 * i * SHRINK_PITCH) = f.x[i];
#pragma unroll
    for (int i = 0; i < AI; ++i) *(u32v4*)(put + 8 * (XI + i) * SHRINK_PITCH) = f.a[i];
    wave_sync();
  };
  auto multiply = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32v4 af[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) af[r] = *(const u32v4*)(get + 16 * (MT + r) * SHRINK_PITCH + 64 * h);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const u32v4 xf = *(const u32v4*)(get + 16 * m * SHRINK_PITCH + 64 * h);
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[m][r] = mma<DT>(af[r], xf, acc[m][r]);
      }
    }
  };
  // this wave's steps: of the split's, every SHRINK_WAVES-th
  const int steps = p.K / 64, s0 = (int)((int64_t)steps * split / p.splits) + wave;
  const int n = ((int)((int64_t)steps * (split + 1) / p.splits) - s0 + SHRINK_WAVES - 1) / SHRINK_WAVES;
  auto k_of = [&](int i) { return (s0 + i * SHRINK_WAVES) * 64; };
  Step fa, fb;
  if (n > 0) fetch_a(fa, k_of(0));       // does not wait for the tokens
#pragma unroll
  for (int i = 0; i < XI; ++i) xr[i] = (const uint16_t*)p.x + (int64_t)min(max(tok[i], 0), p.M - 1) * p.ldx + lcol;
  if (n > 0) {
    // two steps in flight; no condition on a load inside the loop, or its wait
    // would be for everything
    fetch_x(fa, k_of(0));
    fetch_a(fb, k_of(min(1, n - 1)));
    fetch_x(fb, k_of(min(1, n - 1)));
    int i = 0;
    for (; i + 3 < n; i += 2) {
      stage(fa);
      fetch_a(fa, k_of(i + 2));
      fetch_x(fa, k_of(i + 2));
      multiply();
      stage(fb);
      fetch_a(fb, k_of(i + 3));
      fetch_x(fb, k_of(i + 3));
      multiply();
    }
    stage(fa);
    if (i + 2 < n) {
      fetch_a(fa, k_of(i + 2));
      fetch_x(fa, k_of(i + 2));
    }
    multiply();
    if (i + 1 < n) {
      stage(fb);
      multiply();
    }
    if (i + 2 < n) {
      stage(fa);
      multiply();
    }
  }
  if (split == p.splits - 1 && wave == SHRINK_WAVES - 1 && steps * 64 < p.K) {
    // the rest of K, a multiple of 8: a lane's eight elements are in or out
    const int k = steps * 64;
#pragma unroll
    for (int i = 0; i < AI; ++i) fa.a[i] = u32v4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < XI; ++i) fa.x[i] = u32v4{0, 0, 0, 0};
    if (k + lcol < p.K) {
      fetch_a(fa, k);
      fetch_x(fa, k);
    }
    stage(fa);
    multiply();
  }
  __syncthreads();                 // the areas become the sums to join
  f32x4* sh = (f32x4*)lds;         // [wave][block][lane]
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r) sh[(wave * MT * RT + m * RT + r) * 64 + lane] = acc[m][r];
  __syncthreads();
  // block b of the tile: lane l holds ranks 4 (l / 16) .. + 3 of token l % 16
  float* out = p.part + (int64_t)split * p.M * p.R;
  for (int i = threadIdx.x; i < MT * RT * 64; i += 64 * SHRINK_WAVES) {
    const int b = i >> 6, l = i & 63;
    f32x4 u = sh[i];
#pragma unroll
    for (int w = 1; w < SHRINK_WAVES; ++w) u += sh[w * MT * RT * 64 + i];
    const int row = (b / RT) * 16 + (l & 15), r = r0 + (b % RT) * 16 + (l >> 4) * 4;
    if (row < tile.rows && r < p.R) *(f32x4*)(out + (int64_t)(tile.row0 + row) * p.R + r) = u;
  }
}

// y += scale B v of one tile, RP the rank rounded up to 32, 64 or 128. A wave
// takes 64 columns at a time, their ranks up to 64 at a time: these rows of B come
// in whole lines, one piece ahead, and are turned into matrix operands in the
// wave's own LDS area, and so are the products on their way to y, which is read
// and written 128 bytes a token (with the operands' own lanes, 16 tokens side
// by side, the address path took most of 53 us for 4096 x 7168, rank 64).
// Workgroups of a tile: runs of `run` column groups.
template <int DT, int MT, int RP>
__global__ __launch_bounds__(64 * EXPAND_WAVES) void k_lora_expand(LoraArgs p, int run) {
  constexpr int TM = 16 * MT, VP = RP + 8;                   // pitch of v in 16-bit elements
  constexpr int RH = RP < 64 ? RP : 64, HALVES = RP / RH;    // ranks at a time
  constexpr int BP = RH * 2 + 16, CP = 64 * 4 + 16;          // pitches in bytes: of B, of the products
  constexpr int AREA = 64 * BP > 16 * CP ? 64 * BP : 16 * CP;
  __shared__ __attribute__((aligned(16))) uint16_t vh[TM * VP], vl[TM * VP];
  __shared__ __attribute__((aligned(16))) uint8_t lds[EXPAND_WAVES * AREA];
  __shared__ float fac[TM];                                  // scale * 2^e
  const int groups = (p.N + 63) / 64;                        // of 64 columns
  const Tile tile = find_tile<TM>(p.adapter_off, p.n, p.M, blockIdx.x, (groups + run - 1) / run);
  if (tile.adapter < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float scale = p.scale != nullptr ? p.scale[tile.adapter] : 1.0f;
  const int c = lane & 15, q = lane >> 4, lrow = lane >> 3, lcol = (lane & 7) * 8;
  int ytok[2 * MT];
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) ytok[i] = p.row_token[tile.row0 + min(8 * i + lrow, tile.rows - 1)];
  // B pieces of 16 bytes. Ranks up to 32: the group's rows are one run of
  // 64 R / 8 pieces, 64 at a time. Above: eight lanes per row, those past the rank
  // repeat its last piece (what they bring is masked below).
  constexpr int BI = RH / 8;
  const int per_row = p.R / 8;
  uint32_t bsrc[BI], bput[BI];
#pragma unroll
  for (int i = 0; i < BI; ++i) {
    const int flat = i * 64 + lane;
    const int row = RP == 32 ? flat / per_row : flat >> 3, piece = RP == 32 ? flat - row * per_row : flat & 7;
    bsrc[i] = RP == 32 ? flat * 8 : row * p.R;
    bput[i] = row * BP + piece * 16;
  }
  const uint16_t* bm = (const uint16_t*)p.b + (int64_t)tile.adapter * p.N * p.R;
  u32v4 bv[BI];
  auto fetch = [&](int g, int h) {
    const int n0 = g * 64, rows = min(64, p.N - n0);
    const uint16_t* bg = bm + (int64_t)n0 * p.R;
#pragma unroll
    for (int i = 0; i < BI; ++i) {
      uint32_t at;
      if constexpr (RP == 32) at = min(bsrc[i], (uint32_t)(rows * p.R - 8));
      else at = min(bsrc[i], (uint32_t)((rows - 1) * p.R)) + min(h * 64 + (lane & 7) * 8, p.R - 8);
      if (RP != 32 || i < per_row) bv[i] = *(const u32v4*)(bg + at);
    }
  };
  const int g0 = tile.piece * run, g1 = min(groups, g0 + run);
  if (g0 + wave < g1) fetch(g0 + wave, 0);                   // on its way while v is formed
  // v of the tile: RP / 4 lanes per row, four ranks each; the splits' partial
  // sums, eight loads at a time, in split order
  constexpr int PER = RP / 4, ROWS = 64 / PER;
  const int r = (lane & (PER - 1)) * 4;
  for (int row = wave * ROWS + lane / PER; row < TM; row += EXPAND_WAVES * ROWS) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (r < p.R && row < tile.rows) {
      const float* src = p.part + (int64_t)(tile.row0 + row) * p.R + r;
      const int64_t next = (int64_t)p.M * p.R;
      for (int s = 0; s < p.splits; s += 8) {
        f32x4 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = *(const f32x4*)(src + (int64_t)min(s + i, p.splits - 1) * next);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (s + i < p.splits) v += u[i];
      }
    }
    float down = 1.0f, up = 1.0f;
    if constexpr (DT == DT_F16) {
      // 2^-e with 2^e the exponent of the row's largest value, where that is an
      // ordinary number; bf16 has fp32's range and needs none
      float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
      for (int d = PER / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
      const uint32_t ex = __float_as_uint(amax) >> 23;
      if (ex >= 2 && ex <= 252) {
        down = __uint_as_float((254u - ex) << 23);
        up = __uint_as_float(ex << 23);
      }
    }
    uint32_t h[2], l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float u0 = v[2 * i] * down, u1 = v[2 * i + 1] * down;
      h[i] = pack2<DT>(u0, u1);
      const float h0 = lo_f32<DT>(h[i]), h1 = hi_f32<DT>(h[i]);
      // an inf or NaN travels in hi alone
      l[i] = pack2<DT>(fabsf(h0) < INFINITY ? u0 - h0 : 0.0f, fabsf(h1) < INFINITY ? u1 - h1 : 0.0f);
    }
    *(u32v2*)(vh + row * VP + r) = u32v2{h[0], h[1]};
    *(u32v2*)(vl + row * VP + r) = u32v2{l[0], l[1]};
    if (r == 0) fac[row] = scale * up;
  }
  // y pieces: token 8 i + lane / 8 of the tile, columns 8 (lane % 8) of the group;
  // rows past the tile repeat the last one and are not written
  const char* yr[2 * MT];
  bool mine[2 * MT];
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    mine[i] = 8 * i + lrow < tile.rows && (unsigned)ytok[i] < (unsigned)p.M;
    yr[i] = at<DT>((const void*)p.y, (int64_t)min(max(ytok[i], 0), p.M - 1) * p.ldy);
  }
  uint8_t* area = lds + wave * AREA;
  __syncthreads();
  for (int g = g0 + wave; g < g1; g += EXPAND_WAVES) {
    const int n0 = g * 64, n = min(n0 + lcol, p.N - 8);     // N % 8 == 0
    Raw<DT, 8> y[2 * MT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) y[i].load(yr[i], n);
    f32x4 acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      wave_sync();
#pragma unroll
      for (int i = 0; i < BI; ++i)
        if (RP != 32 || i < per_row) *(u32v4*)(area + bput[i]) = bv[i];
      wave_sync();
      // the next piece, or at the end this one again: no condition on the loads
      if (h + 1 < HALVES) fetch(g, h + 1);
      else fetch(min(g + EXPAND_WAVES, groups - 1), 0);
#pragma unroll
      for (int k = 0; k < RH; k += 32) {
        const int r0 = h * RH + k + q * 8;
        u32v4 bf[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bf[j] = *(const u32v4*)(area + (16 * j + c) * BP + k * 2 + q * 16);
          if (r0 >= p.R) bf[j] = u32v4{0, 0, 0, 0};          // past the rank: whatever LDS held
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int w = (m * 16 + c) * VP + r0;
          const u32v4 hi = *(const u32v4*)(vh + w), lo = *(const u32v4*)(vl + w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[m][j] = mma<DT>(bf[j], lo, acc[m][j]);
            acc[m][j] = mma<DT>(bf[j], hi, acc[m][j]);
          }
        }
      }
    }
    // product j: columns 16 j + 4 q .. + 3 of token c
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      wave_sync();
#pragma unroll
      for (int j = 0; j < 4; ++j) *(f32x4*)(area + c * CP + (16 * j + 4 * q) * 4) = acc[m][j];
      wave_sync();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = 2 * m + half;
        const f32x4* d = (const f32x4*)(area + (8 * half + lrow) * CP + lcol * 4);
        const f32x4 d0 = d[0], d1 = d[1];
        const float f = fac[8 * i + lrow];
        float o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[e] = fmaf(f, d0[e], y[i].get(e));
          o[4 + e] = fmaf(f, d1[e], y[i].get(4 + e));
        }
        y[i].set(o);
        if (mine[i] && n0 + lcol < p.N) y[i].store((char*)yr[i], n);
      }
    }
  }
}

// 16-row blocks per tile. A tile holds one adapter's rows, so it is no larger than
// an adapter's share; and a larger one reads A and B less often but leaves fewer
// workgroups, so it takes many rows to pay.
int row_blocks(int64_t M, int n, int most, int64_t from) {
  const int64_t share = M / std::min<int64_t>(n, std::max<int64_t>(M, 1));
  return M >= from && share >= 16 * most ? most : 1;
}
constexpr int SHRINK_MT = 2, EXPAND_MT = 4;
int shrink_mt(int64_t M, int n) { return row_blocks(M, n, SHRINK_MT, 1024); }
int expand_mt(int64_t M, int n) { return row_blocks(M, n, EXPAND_MT, 2048); }
// Upper bound of the tiles of mt 16-row blocks: every adapter adds one partly filled at most.
int64_t lora_tiles(int64_t M, int n, int mt) { return M / (16 * mt) + std::min<int64_t>(n, M); }

}  // namespace

// K splits of the shrink: the number that a workgroup's steps and the rounds of
// workgroups, two on each CU of an MI355X, make fastest; a workgroup costs about
// three steps beside its own. 1 to 16, each wave at least one step.
int lora_splits(int64_t M, int64_t K, int R, int n) {
  const int mt = shrink_mt(M, n);
  const int64_t tiles = (M + 16 * mt - 1) / (16 * mt) + std::min<int64_t>(n, M) / 2, groups = (R + 63) / 64;
  const int64_t steps = K / 64, most = std::min<int64_t>(16, std::max<int64_t>(1, steps / SHRINK_WAVES));
  int best = 1;
  double least = 0;
  for (int s = 1; s <= most; ++s) {
    const int64_t rounds = (tiles * groups * s + 511) / 512;
    const double cost = (double)rounds * ((double)steps / (s * SHRINK_WAVES) + 3.0);
    if (s == 1 || cost < least) {
      best = s;
      least = cost;
    }
  }
  return best;
}

hipError_t launch_lora_shrink(const LoraArgs& p, hipStream_t s) {
  const int mt = shrink_mt(p.M, p.n);
  const int rt = p.R <= 16 ? 1 : p.R <= 32 ? 2 : 4;
  const unsigned grid = (unsigned)(lora_tiles(p.M, p.n, mt) * p.splits * ((p.R + 16 * rt - 1) / (16 * rt)));
  auto go = [&](auto d, auto m, auto r) {
    k_lora_shrink<decltype(d)::value, decltype(m)::value, decltype(r)::value><<<grid, 64 * SHRINK_WAVES, 0, s>>>(p);
  };
  auto by_rt = [&](auto d, auto m) {
    if (rt == 1) go(d, m, std::integral_constant<int, 1>());
    else if (rt == 2) go(d, m, std::integral_constant<int, 2>());
    else go(d, m, std::integral_constant<int, 4>());
  };
  auto by_mt = [&](auto d) {
    if (mt == 1) by_rt(d, std::integral_constant<int, 1>());
    else by_rt(d, std::integral_constant<int, SHRINK_MT>());
  };
  if (p.dt == DT_BF16) by_mt(DtC<DT_BF16>());
  else by_mt(DtC<DT_F16>());
  return hipGetLastError();
}

hipError_t launch_lora_expand(const LoraArgs& p, hipStream_t s) {
  const int mt = expand_mt(p.M, p.n);
  const int groups = (p.N + 63) / 64;
  // runs of column groups: as many workgroups as fit the CUs of an MI355X at once,
  // since each joins the tile's splits anew. 4096 x 7168, rank 64: 31.2 us at two
  // per CU, 41.3 at three (two rounds, the second half empty), 36.8 at four
  const int64_t runs = std::max<int64_t>(1, (mt == 1 ? 4 : 2) * 256 / lora_tiles(p.M, p.n, mt));
  const int each = (int)((groups + runs * EXPAND_WAVES - 1) / (runs * EXPAND_WAVES));
  const int run = each * EXPAND_WAVES;
  const unsigned grid = (unsigned)(lora_tiles(p.M, p.n, mt) * ((groups + run - 1) / run));
  auto go = [&](auto d, auto m, auto r) {
    k_lora_expand<decltype(d)::value, decltype(m)::value, decltype(r)::value><<<grid, 64 * EXPAND_WAVES, 0, s>>>(p, run);
  };
  auto by_r = [&](auto d, auto m) {
    if (p.R <= 32) go(d, m, std::integral_constant<int, 32>());
    else if (p.R <= 64) go(d, m, std::integral_constant<int, 64>());
    else go(d, m, std::integral_constant<int, 128>());
  };
  auto by_mt = [&](auto d) {
    if (mt == 1) by_r(d, std::integral_constant<int, 1>());
    else by_r(d, std::integral_constant<int, EXPAND_MT>());
  };
  if (p.dt == DT_BF16) by_mt(DtC<DT_BF16>());
  else by_mt(DtC<DT_F16>());
  return hipGetLastError();
}

}  // namespace mx
