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
// v is formed in fp32. For the matrix unit each value is cut into three 16-bit
// pieces that add up to it: in bf16 exactly (8 bits each), in fp16, after a
// power-of-two scaling of the token's row, exactly down to 2^-15 of the row's
// largest value and to within 2^-38 of that one below. So the second product is off
// by fp32's own rounding only, also where it cancels y. (Two pieces, 16 bits of v in
// bf16, left 2^-17 of each product; the third costs matrix and LDS cycles but no memory
// traffic: 7168 + 7168 columns, 4096 tokens, rank 64 40.6 -> 42.1 us, 8192 tokens, rank
// 128 92.4 -> 98.5.) y is rounded once.
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

// Three pieces of each of u0, u1, packed in pairs: piece[0] + piece[1] + piece[2] = u, each cut off towards
// zero, so that the next takes what is left exactly. An inf or NaN travels in the first alone (a NaN that
// arithmetic gave has its highest mantissa bit set, which the first piece keeps).
template <int DT>
__device__ __forceinline__ void cut3(float u0, float u1, uint32_t (&piece)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    float h0, h1;
    if constexpr (DT == DT_BF16) {
      const uint32_t w0 = __float_as_uint(u0), w1 = __float_as_uint(u1);
      piece[i] = __builtin_amdgcn_perm(w1, w0, 0x07060302u);   // the upper halves
      h0 = __uint_as_float(w0 & 0xFFFF0000u);
      h1 = __uint_as_float(w1 & 0xFFFF0000u);
    } else {
      piece[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(u0, u1));
      h0 = lo_f32<DT>(piece[i]);
      h1 = hi_f32<DT>(piece[i]);
    }
    const bool f0 = i > 0 || fabsf(u0) < INFINITY, f1 = i > 0 || fabsf(u1) < INFINITY;
    u0 = f0 ? u0 - h0 : 0.0f;
    u1 = f1 ? u1 - h1 : 0.0f;
  }
}

// acc + 0 * (two elements): NaN if one is infinite or NaN.
template <int DT>
__device__ __forceinline__ float dot0(uint32_t w, float acc) {
  if constexpr (DT == DT_BF16) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, 0u), acc, false);
  } else {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, w), __builtin_bit_cast(f16x2, 0u), acc, false);
  }
}

// A tile is up to TM sorted rows of one adapter, adapters in order. How many there
// are, and where each lies, is only known on the device: every wave looks at
// the adapters' offsets itself, 64 at a time.
struct Tile {
  int adapter, row0, rows;   // sorted rows [row0, row0 + rows)
};
template <int TM>
struct Tiles {
  const int32_t* off;
  int n, M, total;
  int lo, hi, cnt, inc;      // of the lane's adapter among the first 64: rows, tiles, tiles up to it

  __device__ __forceinline__ void look(int a0) {
    const int lane = threadIdx.x & 63, a = a0 + lane;
    lo = hi = 0;
    if (a < n) {
      lo = min(max(off[a], 0), M);
      hi = min(max(off[a + 1], lo), M);
    }
    cnt = (hi - lo + TM - 1) / TM;
    inc = cnt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(inc, d);
      if (lane >= d) inc += u;
    }
  }
  __device__ __forceinline__ Tiles(const int32_t* off_, int n_, int M_) : off(off_), n(n_), M(M_) {
    total = 0;
    for (int a0 = (n - 1) / 64 * 64; a0 >= 0; a0 -= 64) {    // ends on the first 64
      look(a0);
      total += __builtin_amdgcn_readlane(inc, 63);
    }
  }
  __device__ __forceinline__ Tile find(int tile) {
    int before = 0;
    for (int a0 = 0; a0 < n; a0 += 64) {
      if (n > 64) look(a0);
      const uint64_t hit = __ballot(before + inc > tile);
      if (hit) {
        const int l = __ffsll((long long)hit) - 1;
        const int first = before + __builtin_amdgcn_readlane(inc, l) - __builtin_amdgcn_readlane(cnt, l);
        const int row0 = __builtin_amdgcn_readlane(lo, l) + (tile - first) * TM;
        return {a0 + l, row0, min(TM, __builtin_amdgcn_readlane(hi, l) - row0)};
      }
      before += __builtin_amdgcn_readlane(inc, 63);
    }
    return {0, 0, 0};
  }
};

// Workgroups go to the 8 XCDs in turn, and neighbouring tiles mostly share an
// adapter: each XCD gets a contiguous run of the `work` pieces, so that its L2
// holds a few adapters (8 adapters of 64 x 7168: 7.3 MB, more than its 4 MB).
__device__ __forceinline__ int xcd_run(int id, int work) {
  const int xcd = id & 7;
  return (work >> 3) * xcd + min(xcd, work & 7) + (id >> 3);
}

// How the shrink's work is shared out. A unit is a tile and a group of ranks, its
// work the 64-wide steps of K (a shorter rest of K goes with the last); units
// one after another make one row of steps, cut into equal runs of q, one per
// workgroup, so that all finish together however many tiles there are. A unit's
// v is then the sum of what the workgroups from first() to last() left of it.
// (Divisions cost a few calls of this their latency: what the host knows of q comes
// with the arguments.)
struct Share {
  uint32_t steps, q, total;
  __device__ __forceinline__ Share(const LoraArgs& p, int units) {
    steps = max(p.K / 64, 1);
    total = (uint32_t)units * steps;
    q = max((total + (1u << p.slots_log2) - 1) >> p.slots_log2, (uint32_t)p.least);
  }
  __device__ __forceinline__ int groups() const { return (total + q - 1) / q; }
  __device__ __forceinline__ int first(int unit) const { return (uint32_t)unit * steps / q; }
  __device__ __forceinline__ int last(int unit) const { return ((uint32_t)(unit + 1) * steps - 1) / q; }
};

// Between the lanes of one wave: LDS writes before, reads after.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Parts of v, [part][sorted row][R]: per unit MT x RT blocks of 16 tokens x 16 ranks.
// A matrix operand wants 16 rows side by side in the lanes, but a load whose
// neighbouring lanes are in different rows takes the address path one row at a time
// (4096 x 7168, rank 64: 39 us that way, 35 with x in L2). So a wave loads whole
// 128-byte lines, eight lanes each, the rows of a 64-wide step of K, turns them
// in an LDS area of its own (pitch 144: conflict-free) and has the next
// two steps' loads in flight meanwhile. The waves take a workgroup's steps in turn,
// 512 bytes of a row together, and join their sums in LDS.
constexpr int SHRINK_PITCH = 128 + 16;
template <int DT, int MT, int RT>
__global__ __launch_bounds__(64 * SHRINK_WAVES) void k_lora_shrink(LoraArgs p) {
  constexpr int TM = 16 * MT, XI = 2 * MT, AI = 2 * RT;      // loads of eight rows: of x, of A
  constexpr int AREA = 16 * (MT + RT) * SHRINK_PITCH;
  constexpr int JOIN = MT * RT * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t lds[SHRINK_WAVES * (AREA > JOIN ? AREA : JOIN)];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rlog = p.R > 16 * RT;       // groups of 16 RT ranks: 1 or, above 64 ranks, 2
  Tiles<TM> tiles(p.adapter_off, p.n, p.M);
  const Share share(p, tiles.total << rlog);
  const int all = share.groups();
  if ((int)blockIdx.x >= all) return;
  const int group = xcd_run(blockIdx.x, all);
  uint32_t at = group * share.q;
  const uint32_t end = min(at + share.q, share.total);
  while (at < end) {
    const int unit = at / share.steps, k0 = at - unit * share.steps, k1 = min(share.steps, k0 + end - at);
    at += k1 - k0;
    const Tile tile = tiles.find(unit >> rlog);
    const int r0 = (unit & rlog) * 16 * RT;
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
    // this wave's whole steps: of the workgroup's, every SHRINK_WAVES-th
    const int s0 = k0 + wave, n = (min(k1, p.K / 64) - s0 + SHRINK_WAVES - 1) / SHRINK_WAVES;
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
    if (k1 == (int)share.steps && wave == SHRINK_WAVES - 1 && p.K % 64 != 0) {
      // the rest of K, a multiple of 8: a lane's eight elements are in or out
      const int k = p.K / 64 * 64;
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
    float* out = p.part + (int64_t)(group - share.first(unit)) * p.M * p.R;
    for (int i = threadIdx.x; i < MT * RT * 64; i += 64 * SHRINK_WAVES) {
      const int b = i >> 6, l = i & 63;
      f32x4 u = sh[i];
#pragma unroll
      for (int w = 1; w < SHRINK_WAVES; ++w) u += sh[w * MT * RT * 64 + i];
      const int row = (b / RT) * 16 + (l & 15), r = r0 + (b % RT) * 16 + (l >> 4) * 4;
      if (row < tile.rows && r < p.R) *(f32x4*)(out + (int64_t)(tile.row0 + row) * p.R + r) = u;
    }
    __syncthreads();                 // and areas again
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
__global__ __launch_bounds__(64 * EXPAND_WAVES) void k_lora_expand(LoraArgs p, int run, int runs) {
  constexpr int TM = 16 * MT, VP = RP + 8;                   // pitch of v in 16-bit elements
  constexpr int RH = RP < 64 ? RP : 64, HALVES = RP / RH;    // ranks at a time
  // and in the area: of large tiles of many ranks half of them, which leaves LDS for two workgroups
  constexpr int SH = MT > 1 && RP > 64 ? 32 : RH;
  constexpr int BP = SH * 2 + 16, CP = 64 * 4 + 16;          // pitches in bytes: of B, of the products
  constexpr int AREA = 64 * BP > 16 * CP ? 64 * BP : 16 * CP;
  __shared__ __attribute__((aligned(16))) uint16_t vp[3][TM * VP];   // v's pieces
  __shared__ __attribute__((aligned(16))) uint8_t lds[EXPAND_WAVES * AREA];
  __shared__ float fac[TM];                                  // scale * 2^e
  const int groups = (p.N + 63) / 64;                        // of 64 columns
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Tiles<TM> tiles(p.adapter_off, p.n, p.M);
  const int work = tiles.total * runs;
  if ((int)blockIdx.x >= work) return;
  const int mine_at = xcd_run(blockIdx.x, work), index = mine_at / runs;
  const Tile tile = tiles.find(index);
  const int rlog = RP > 64;                                  // as in the shrink
  const Share share(p, tiles.total << rlog);
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
    bput[i] = row * BP + piece % (SH / 8) * 16;
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
  const int g0 = (mine_at - index * runs) * run, g1 = min(groups, g0 + run);
  if (g0 + wave < g1) fetch(g0 + wave, 0);                   // on its way while v is formed
  // v of the tile: RP / 4 lanes per row, four ranks each, ITER rows per thread; the
  // sum of the parts in their order, eight loads in flight (row by row they cost a
  // tile of 64 rows and 128 ranks eight latencies: 1024 + 1024 columns of 8192 tokens
  // took 28.1 us and take 25.1)
  constexpr int PER = RP / 4, ROWS = 64 / PER;
  constexpr int ITER = TM > EXPAND_WAVES * ROWS ? TM / (EXPAND_WAVES * ROWS) : 1, AHEAD = 8 / ITER;
  const int r = (lane & (PER - 1)) * 4, vrow = wave * ROWS + lane / PER;
  f32x4 vs[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) vs[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (r < p.R) {
    const int unit = (index << rlog) + (r >> 6), parts = share.last(unit) - share.first(unit) + 1;
    const float* src[ITER];
#pragma unroll
    for (int i = 0; i < ITER; ++i)     // rows past the tile repeat the last one: never used
      src[i] = p.part + (int64_t)(tile.row0 + min(vrow + i * EXPAND_WAVES * ROWS, tile.rows - 1)) * p.R + r;
    const int64_t next = (int64_t)p.M * p.R;
    for (int s = 0; s < parts; s += AHEAD) {
      f32x4 u[AHEAD][ITER];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
#pragma unroll
        for (int i = 0; i < ITER; ++i) u[j][i] = *(const f32x4*)(src[i] + (int64_t)min(s + j, parts - 1) * next);
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
#pragma unroll
        for (int i = 0; i < ITER; ++i)
          if (s + j < parts) vs[i] += u[j][i];
    }
  }
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int row = vrow + i * EXPAND_WAVES * ROWS;
    if (row >= TM) continue;
    const f32x4 v = vs[i];
    float down = 1.0f, up = 1.0f;
    if constexpr (DT == DT_F16) {
      // 2^(14 - e) with 2^e the exponent of the row's largest value, so that the pieces
      // use what fp16 has on both sides; bf16 has fp32's range and needs none
      float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
      for (int d = PER / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
      const uint32_t ex = max(__float_as_uint(amax) >> 23, 15u);      // 2^126 at most
      if (ex < 255) {
        down = __uint_as_float((268u - ex) << 23);
        up = __uint_as_float((ex - 14u) << 23);
      }
    }
    uint32_t c0[3], c1[3];
    cut3<DT>(v[0] * down, v[1] * down, c0);
    cut3<DT>(v[2] * down, v[3] * down, c1);
#pragma unroll
    for (int j = 0; j < 3; ++j) *(u32v2*)(vp[j] + row * VP + r) = u32v2{c0[j], c1[j]};
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
  // An infinite B: its products with a value's pieces (zeros, mostly) do not add up to the
  // one with the value, and NaN comes out. Those sums once more, by the formula. (Looking
  // for them takes 0.3 us of 42 at 4096 tokens of 7168 + 7168 columns, rank 64.)
  auto by_formula = [&](f32x4 (&acc)[MT][4], int n0) {
    const uint16_t* br = bm + (int64_t)min(n0 + lane, p.N - 1) * p.R;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      wave_sync();
#pragma unroll
      for (int j = 0; j < 4; ++j) *(f32x4*)(area + c * CP + (16 * j + 4 * q) * 4) = acc[m][j];
      wave_sync();
#pragma unroll 1
      for (int row = 0; row < 16; ++row) {
        float* out = (float*)(area + row * CP) + lane;
        if (*out == *out) continue;
        const uint16_t* vr = &vp[0][(16 * m + row) * VP];
        float sum = 0.0f;
#pragma unroll 1
        for (int k = 0; k < p.R && sum == sum; ++k)
          sum = fmaf(lo_f32<DT>(vr[k]) + (lo_f32<DT>(vr[TM * VP + k]) + lo_f32<DT>(vr[2 * TM * VP + k])),
                     lo_f32<DT>(br[k]), sum);
        *out = sum;
      }
      wave_sync();
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][j] = *(const f32x4*)(area + c * CP + (16 * j + 4 * q) * 4);
    }
  };
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
    float odd = 0.0f;                // large tiles: NaN from the first infinite (or NaN) B on
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
#pragma unroll
      for (int part = 0; part < RH; part += SH) {
        wave_sync();
        if (SH == RH || (lane & 7) / (SH / 8) == part / SH) {
#pragma unroll
          for (int i = 0; i < BI; ++i)
            if (RP != 32 || i < per_row) *(u32v4*)(area + bput[i]) = bv[i];
        }
        wave_sync();
        // the next piece, or at the end this one again: no condition on the loads
        if (part + SH == RH) {
          if (h + 1 < HALVES) fetch(g, h + 1);
          else fetch(min(g + EXPAND_WAVES, groups - 1), 0);
        }
#pragma unroll
        for (int k = 0; k < SH; k += 32) {
          if (h * RH + part + k >= p.R) break;               // nothing but padding
          const int r0 = h * RH + part + k + q * 8;
          u32v4 bf[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            bf[j] = *(const u32v4*)(area + (16 * j + c) * BP + k * 2 + q * 16);
            if (r0 >= p.R) bf[j] = u32v4{0, 0, 0, 0};        // past the rank: whatever LDS held
#pragma unroll
            for (int i = 0; i < (MT > 1 ? 4 : 0); ++i) odd = dot0<DT>(bf[j][i], odd);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const int w = (m * 16 + c) * VP + r0;
#pragma unroll
            for (int i = 2; i >= 0; --i) {                   // the small pieces first
              const u32v4 v = *(const u32v4*)(vp[i] + w);
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[m][j] = mma<DT>(bf[j], v, acc[m][j]);
            }
          }
        }
      }
    }
    // whether to look for such sums: of a large tile by its operands, of a small one by its fewer sums
    bool look = odd != odd;
    if constexpr (MT == 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        look |= __builtin_isunordered(acc[0][j][0], acc[0][j][1]) || __builtin_isunordered(acc[0][j][2], acc[0][j][3]);
    }
    if (__ballot(look)) by_formula(acc, n0);
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
// workgroups, so it takes many rows and much to read of each to pay. One block
// against four, rank 64, 4 adapters, us: 1024 tokens of 7168 + 7168 columns 21.8 and
// 22.9, 4096 of them 51.6 and 44.0; 4096 tokens of 2048 + 512 15.0 and 15.8, of
// 2048 + 2048 21.2 and 21.0; 8192 tokens of 512 + 512 15.0 and 15.9, of 1024 + 1024
// 21.4 and 20.5, of 2048 + 2048 34.8 and 30.4.
constexpr int BIG_MT = 4;
bool big_rows(int64_t M, int n) { return M >= 2048 && M / n >= 16 * BIG_MT; }
int row_blocks(const LoraArgs& p) {
  return big_rows(p.M, p.n) && (int64_t)p.M * (p.K + p.N) >= (int64_t)1 << 24 ? BIG_MT : 1;
}
// Upper bound of the tiles of mt 16-row blocks: every adapter adds one partly filled at most.
int64_t lora_tiles(int64_t M, int n, int mt) { return M / (16 * mt) + std::min<int64_t>(n, M); }

// 16-rank blocks of a shrink workgroup
int rank_blocks(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : 4; }
// Shrink workgroups that fit the CUs of an MI355X at once (registers: one of
// four waves with large tiles, else two).
int slots_log2(int mt) { return mt == 1 ? 9 : 8; }
// Workgroups that may share one unit's K: what fills the slots, 16 at most.
int shrink_parts(int64_t M, int mt) {
  const int64_t tiles = std::max<int64_t>(1, M / (16 * mt));
  return (int)std::min<int64_t>(16, 2 + ((1 << slots_log2(mt)) + tiles - 1) / tiles);
}

hipError_t launch_expand(const LoraArgs& p, int mt, hipStream_t s) {
  const int groups = (p.N + 63) / 64;
  // Runs of column groups, `each` per wave. Workgroups that do not fit the CUs of an
  // MI355X at once (two of large tiles, else four) wait for another round, and each
  // forms the tile's v anew, half a group of a wave's time: of what fills one to
  // eight rounds, the one of the least rounds x (each + 1/2). 7168 + 7168 columns, rank
  // 64, 8 adapters, the most that one round holds against this, us: 4096 tokens 43.0
  // and 42.9, 8192 85 and 77, 20000 216 and 188, 34000 366 and 317.
  const int64_t tiles = lora_tiles(p.M, p.n, mt), slots = (mt == 1 ? 4 : 2) * 256;
  int run = 0, all_runs = 0;
  for (int64_t k = 1, least = INT64_MAX; k <= 8; ++k) {
    const int64_t runs = std::max<int64_t>(1, k * slots / tiles);
    const int each = (int)((groups + runs * EXPAND_WAVES - 1) / (runs * EXPAND_WAVES));
    const int some = (groups + each * EXPAND_WAVES - 1) / (each * EXPAND_WAVES);
    const int64_t cost = (tiles * some + slots - 1) / slots * (2 * each + 1);
    if (cost < least) {
      least = cost;
      run = each * EXPAND_WAVES;
      all_runs = some;
    }
    if (each == 1) break;              // no shorter runs
  }
  const unsigned grid = (unsigned)(tiles * all_runs);
  auto go = [&](auto d, auto m, auto r) {
    k_lora_expand<decltype(d)::value, decltype(m)::value, decltype(r)::value>
        <<<grid, 64 * EXPAND_WAVES, 0, s>>>(p, run, all_runs);
  };
  auto by_r = [&](auto d, auto m) {
    if (p.R <= 32) go(d, m, std::integral_constant<int, 32>());
    else if (p.R <= 64) go(d, m, std::integral_constant<int, 64>());
    else go(d, m, std::integral_constant<int, 128>());
  };
  auto by_mt = [&](auto d) {
    if (mt == 1) by_r(d, std::integral_constant<int, 1>());
    else by_r(d, std::integral_constant<int, BIG_MT>());
  };
  if (p.dt == DT_BF16) by_mt(DtC<DT_BF16>());
  else by_mt(DtC<DT_F16>());
  return hipGetLastError();
}

}  // namespace

// The workspace is asked for without N, so it holds the parts of either tile.
int lora_parts(int64_t M, int n) {
  return std::max(shrink_parts(M, 1), big_rows(M, n) ? shrink_parts(M, BIG_MT) : 0);
}

hipError_t launch_lora(const LoraArgs& args, hipStream_t s) {
  LoraArgs p = args;
  const int mt = row_blocks(p), rt = rank_blocks(p.R);
  const int steps = std::max(p.K / 64, 1), parts = shrink_parts(p.M, mt);
  p.slots_log2 = slots_log2(mt);
  // a run of q = ceil(steps / (parts - 1)) steps or more touches a unit at most `parts` times
  p.least = std::max(SHRINK_WAVES, (steps + parts - 2) / (parts - 1));
  const int64_t units = lora_tiles(p.M, p.n, mt) << (p.R > 64);
  const unsigned grid = (unsigned)std::min<int64_t>(1 << p.slots_log2, (units * steps + p.least - 1) / p.least);
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
    else by_rt(d, std::integral_constant<int, BIG_MT>());
  };
  if (p.dt == DT_BF16) by_mt(DtC<DT_BF16>());
  else by_mt(DtC<DT_F16>());
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_expand(p, mt, s);
}

}  // namespace mx
