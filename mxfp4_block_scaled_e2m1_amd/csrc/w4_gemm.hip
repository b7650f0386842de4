// Many tokens of the linear layer with 4-bit weights and group scales (w4.hip has the
// formula and the form for few tokens): a matrix product bound by the matrix cores.
//
// 256 tokens x 256 weight rows per workgroup of 8 waves, each 128 tokens x 64 rows as
// 4 x 2 blocks of V_MFMA_F32_32X32X16. A stage of 64 columns is 32 KB of activations,
// 8 KB of codes and the scales of its two blocks of 32 columns; three stages are in LDS,
// copied there directly (GLOBAL_LOAD_LDS) two stages ahead, one barrier a stage. The
// codes stay 4 bits until a wave expands its rows' in registers (twice per code and
// workgroup; the activations are what LDS bandwidth goes to).
//
// MXFP4 with bf16 activations: code * 2^(byte - 127) is a bf16 number as long as no byte
// is above 252, so the scale goes into the expansion and the products add up in place.
// Everything else (fp16, which has no such range; INT4, whose scale has bits of its own;
// MXFP4 with larger bytes) multiplies the fp32 sum of a group by its scale.
//
// The scales come as a table [K / 32][N] of fp32 that a small kernel before makes (the
// rows of scales are neither aligned nor next to each other for a stage).
#include <algorithm>
#include <cstdlib>

#include "w4_expand.h"

namespace mx {

namespace {

constexpr int TK = 64;                    // columns of a stage
constexpr int SLOTS = 3;

// A workgroup's tile: WM x WN waves of 32 I tokens x 32 J weight rows each.
template <int WM, int WN, int I, int J>
struct Tile {
  static constexpr int IB = I, JB = J, WAVES_M = WM, WAVES_N = WN, THREADS = 64 * WM * WN;
  static constexpr int TM = 32 * I * WM, TN = 32 * J * WN;
  static constexpr int X_BYTES = TM * TK * 2, W_BYTES = TN * TK / 2, S_BYTES = 2 * TN * 4;
  static constexpr int SLOT = X_BYTES + W_BYTES + 2 * S_BYTES;   // the second table: zero points
  // The output tile takes the stages' place, its rows at a pitch that spreads them over the banks.
  static constexpr int Y_PITCH = TN * 2 + 8;
  static constexpr int SMEM = SLOTS * SLOT > TM * Y_PITCH ? SLOTS * SLOT : TM * Y_PITCH;
  static constexpr int X_COPIES = X_BYTES / (16 * THREADS);
  static_assert(W_BYTES == 16 * THREADS && 2 * TN == THREADS, "one copy of codes and one table entry a thread");
};

// Copies of 16 or 4 bytes a lane to LDS, lane i's to base + 16 i or 4 i. Inline, so that the compiler does not
// wait for them before every LDS read: the loop waits for a stage's copies itself.
__device__ __forceinline__ void copy16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void copy4(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(lds) : "memory", "m0");
}

// 16-byte chunk c (of 8) of activation row r: 16 rows at one chunk fall in 16 bank groups.
__device__ __forceinline__ int x_off(int r, int c) { return r * (TK * 2) + ((c ^ ((r >> 1) & 7)) << 4); }
// 16-byte chunk c (of 2, a block of 32 columns each) of code row r.
__device__ __forceinline__ int w_off(int r, int c) { return r * (TK / 2) + ((c ^ ((r >> 3) & 1)) << 4); }

template <int DT>
__device__ __forceinline__ f32x16 mfma32(u32v4 a, u32v4 b, const f32x16& c) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Until no more than N of the wave's copies are under way and its LDS reads are done, then the barrier.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  static_assert(N == 0 || (N >= 4 && N <= 7), "a wait for each count");
  if constexpr (N == 0) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else if constexpr (N == 4) asm volatile("s_waitcnt vmcnt(4) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else if constexpr (N == 5) asm volatile("s_waitcnt vmcnt(5) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else if constexpr (N == 6) asm volatile("s_waitcnt vmcnt(6) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else asm volatile("s_waitcnt vmcnt(7) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The tile's products. GROUPS: scaled sums per block of 32 columns (1) or per stage (2, groups of
// 64 or more); 0: scales in the expansion.
template <class T, int DT, bool INT, int GROUPS>
__device__ __forceinline__ void w4_tile(const W4Args& a, uint8_t* smem, int64_t t0, int64_t n0) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int TM = T::TM, TN = T::TN, IB = T::IB, JB = T::JB, XC = T::X_COPIES;
  constexpr int X_BYTES = T::X_BYTES, W_BYTES = T::W_BYTES, S_BYTES = T::S_BYTES, SLOT = T::SLOT, Y_PITCH = T::Y_PITCH;
  const int r32 = lane & 31, h = lane >> 5, wn = wave % T::WAVES_N, wm = wave / T::WAVES_N;
  const int blocks = (int)(a.K / 32), stages = (blocks + 1) / 2;

  // this thread's chunks of the activations and the codes, and its entry of each table
  const char* xs[XC];
  int xc[XC];
#pragma unroll
  for (int c = 0; c < XC; ++c) {
    const int p = (wave * XC + c) * 64 + lane, r = p >> 3;
    xc[c] = (p & 7) ^ ((r >> 1) & 7);
    xs[c] = at<DT>(a.x, min(t0 + r, a.M - 1) * a.ldx) + xc[c] * 16;
  }
  const int wr = tid >> 1, wc = (tid & 1) ^ ((wr >> 3) & 1);
  const uint8_t* ws = a.w + min(n0 + wr, a.N - 1) * (a.K / 2) + wc * 16;
  const int sb = tid / TN;                            // the block of the stage whose table entry this thread copies
  const float* ss = a.scale_table + min(n0 + tid % TN, a.N - 1);
  const uint32_t* zs = a.zero_table + min(n0 + tid % TN, a.N - 1);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)smem;
  auto issue = [&](int st) {                           // XC + 2 copies, INT one more
    const uint32_t base = lds0 + (uint32_t)(st % SLOTS) * SLOT;
    // the last stage may have one block: its second half is the first again, and not used
    const bool whole = 2 * st + 1 < blocks;
#pragma unroll
    for (int c = 0; c < XC; ++c)
      copy16(xs[c] + (int64_t)st * (TK * 2) - (whole || xc[c] < 4 ? 0 : 64), base + (wave * XC + c) * 1024);
    copy16(ws + (int64_t)st * (TK / 2) - (whole || wc == 0 ? 0 : 16), base + X_BYTES + wave * 1024);
    const int64_t blk = 2 * st + (whole ? sb : 0);
    copy4(ss + blk * a.N, base + X_BYTES + W_BYTES + wave * 256);
    if constexpr (INT) copy4(zs + blk * a.N, base + X_BYTES + W_BYTES + S_BYTES + wave * 256);
  };

  f32x16 acc[IB][JB];
#pragma unroll
  for (int i = 0; i < IB; ++i)
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  issue(0);
  if (stages > 1) issue(1);
  for (int st = 0; st < stages; ++st) {
    // stage st is there (a later one may be on its way), and all waves are done with the stage before
    if (st + 1 < stages) {
      wait_barrier<XC + 2 + INT>();
    } else {
      wait_barrier<0>();
    }
    if (st + 2 < stages) issue(st + 2);
    const uint8_t* sx = smem + (st % SLOTS) * SLOT;
    const uint8_t* sw = sx + X_BYTES;
    const float* sc = (const float*)(sw + W_BYTES);
    const bool whole = 2 * st + 1 < blocks;
    // lane (row, h) has columns 16 h .. 16 h + 15 of a block: step 2 b + m takes 8 m .. 8 m + 7 of them
    u32v4 w[JB][4];
    float scale[JB][2];
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int r = (wn * JB + j) * 32 + r32;
        const u32v2 d = *(const u32v2*)(sw + w_off(r, b) + 8 * h);
        scale[j][b] = sc[b * TN + r];
        uint32_t zero = 0;
        if constexpr (INT) zero = __float_as_uint(sc[S_BYTES / 4 + b * TN + r]);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if constexpr (INT) w[j][2 * b + m] = expand_int<DT>(d[m], zero);
          else w[j][2 * b + m] = expand_fp4<DT>(d[m], GROUPS == 0 ? scale[j][b] : 1.0f);
        }
      }
#pragma unroll
    for (int i = 0; i < IB; ++i) {
      u32v4 x[4];
#pragma unroll
      for (int s = 0; s < 4; ++s)
        x[s] = *(const u32v4*)(sx + x_off((wm * IB + i) * 32 + r32, 4 * (s >> 1) + 2 * h + (s & 1)));
      if constexpr (GROUPS == 0) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          if (s == 2 && !whole) break;
#pragma unroll
          for (int j = 0; j < JB; ++j) acc[i][j] = mfma32<DT>(x[s], w[j][s], acc[i][j]);
        }
      } else {
#pragma unroll
        for (int b = 0; b < 2; b += GROUPS) {
          if (b == 1 && !whole) break;
#pragma unroll
          for (int j = 0; j < JB; ++j) {
            f32x16 p;
#pragma unroll
            for (int v = 0; v < 16; ++v) p[v] = 0.0f;
#pragma unroll
            for (int s = 2 * b; s < 2 * b + 2 * GROUPS; ++s) p = mfma32<DT>(x[s], w[j][s], p);
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = fmaf(scale[j][b], p[v], acc[i][j][v]);
          }
        }
      }
    }
  }

  // lane (r32, h) has weight row r32 of a block and tokens 8 (v / 4) + 4 h + v % 4: through LDS, and out in whole rows
  __syncthreads();
#pragma unroll
  for (int i = 0; i < IB; ++i)
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int v = 0; v < 16; v += 2) {
        const uint32_t d = pack2<DT>(acc[i][j][v], acc[i][j][v + 1]);
        const int t = (wm * IB + i) * 32 + 8 * (v / 4) + 4 * h + v % 4;
        uint8_t* p = smem + t * Y_PITCH + ((wn * JB + j) * 32 + r32) * 2;
        *(uint16_t*)p = (uint16_t)d;
        *(uint16_t*)(p + Y_PITCH) = (uint16_t)(d >> 16);
      }
  __syncthreads();
  const bool al = a.ldy % 8 == 0 && ((uintptr_t)a.y & 15) == 0;
  for (int p = tid; p < TM * (TN / 8); p += T::THREADS) {
    const int r = p / (TN / 8), c = p % (TN / 8) * 8;
    const int64_t t = t0 + r, n = n0 + c;
    if (t >= a.M || n >= a.N) continue;
    uint16_t* out = (uint16_t*)a.y + t * a.ldy + n;
    const uint16_t* in = (const uint16_t*)(smem + r * Y_PITCH + c * 2);
    if (n + 8 <= a.N) {
      const u32v2 lo = *(const u32v2*)in, hi = *(const u32v2*)(in + 4);
      const u32v4 v = {lo[0], lo[1], hi[0], hi[1]};
      if (al) *(u32v4*)out = v;
      else *(u32v4_any*)out = v;
    } else {
      for (int i = 0; i < (int)(a.N - n); ++i) out[i] = in[i];
    }
  }
}

// Scales (and zero points) as fp32, block by block of 32 columns; large[]: whether the workgroup saw an E8M0 byte above 252.
template <int DT, bool INT>
__global__ __launch_bounds__(256) void k_w4_tables(W4Args a) {
  __shared__ float tile[32][33];
  __shared__ uint32_t ztile[32][33];
  const int64_t groups = a.K >> a.group_log2, blocks = a.K / 32, rep = (int64_t)1 << (a.group_log2 - 5);
  const int64_t tn = (a.N + 31) / 32, tg = (groups + 31) / 32;
  const int lx = threadIdx.x & 31, ly = threadIdx.x >> 5;
  int big = 0;
  for (int64_t t = blockIdx.x; t < tn * tg; t += gridDim.x) {
    const int64_t n0 = t % tn * 32, g0 = t / tn * 32;
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      const int64_t n = min(n0 + ly + i, a.N - 1), g = min(g0 + lx, groups - 1);
      if constexpr (INT) {
        tile[ly + i][lx] = Raw<DT, 1>{{((const uint16_t*)a.scales)[n * groups + g]}}.get(0);
        ztile[ly + i][lx] = zero_bits<DT>(a.zeros != nullptr ? a.zeros[n * groups + g] : 8u);
      } else {
        const uint32_t b = ((const uint8_t*)a.scales)[n * groups + g];
        big |= b > 252u;
        tile[ly + i][lx] = e8m0(b);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      const int64_t n = n0 + lx, g = g0 + ly + i;
      if (n < a.N && g < groups)
        for (int64_t b = g * rep; b < min((g + 1) * rep, blocks); ++b) {
          a.scale_table[b * a.N + n] = tile[lx][ly + i];
          if constexpr (INT) a.zero_table[b * a.N + n] = ztile[lx][ly + i];
        }
    }
    __syncthreads();
  }
  if constexpr (!INT) {
    big = __syncthreads_or(big);
    if (threadIdx.x == 0) a.large[blockIdx.x] = big;
  }
}

template <class T, int DT, bool INT>
__global__ __launch_bounds__(T::THREADS, 2) void k_w4_gemm(W4Args a, int tiles_m, int tiles_n, int per_xcd) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::SMEM];
  // consecutive workgroups are on different XCDs: each XCD takes a run of tiles, four token tiles by all of the rows'
  const int L = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if (L >= tiles_m * tiles_n) return;
  const int band = L / (4 * tiles_n), m0 = band * 4, high = min(4, tiles_m - m0), i = L - band * 4 * tiles_n;
  const int64_t t0 = (int64_t)(m0 + i % high) * T::TM, n0 = (int64_t)(i / high) * T::TN;
  if constexpr (INT) {
    if (a.group_log2 == 5) w4_tile<T, DT, true, 1>(a, smem, t0, n0);
    else w4_tile<T, DT, true, 2>(a, smem, t0, n0);
  } else if constexpr (DT == DT_BF16) {
    int seen = 0;
    for (int i = threadIdx.x; i < W4_TABLE_GRID; i += T::THREADS) seen |= a.large[i];
    const bool large = __syncthreads_or(seen);
    if (large) w4_tile<T, DT, false, 1>(a, smem, t0, n0);
    else w4_tile<T, DT, false, 0>(a, smem, t0, n0);
  } else {
    w4_tile<T, DT, false, 1>(a, smem, t0, n0);
  }
}

}  // namespace

hipError_t launch_w4_gemm(const W4Args& a, hipStream_t s) {
  const auto go = [&](auto tile, auto d, auto in) {
    typedef decltype(tile) T;
    constexpr int D = decltype(d)::value;
    constexpr bool I = decltype(in)::value;
    const int tm = (int)((a.M + T::TM - 1) / T::TM), tn = (int)((a.N + T::TN - 1) / T::TN), per_xcd = (tm * tn + 7) / 8;
    k_w4_tables<D, I><<<W4_TABLE_GRID, 256, 0, s>>>(a);
    k_w4_gemm<T, D, I><<<8 * per_xcd, T::THREADS, 0, s>>>(a, tm, tn, per_xcd);
  };
  const auto types = [&](auto tile) {
    if (a.dt == DT_BF16) {
      if (a.int4) go(tile, DtC<DT_BF16>(), std::true_type());
      else go(tile, DtC<DT_BF16>(), std::false_type());
    } else {
      if (a.int4) go(tile, DtC<DT_F16>(), std::true_type());
      else go(tile, DtC<DT_F16>(), std::false_type());
    }
  };
  static const bool small = getenv("W4SMALL") != nullptr;
  if (small) types(Tile<2, 2, 2, 2>());
  else types(Tile<2, 4, 4, 2>());
  return hipGetLastError();
}

}  // namespace mx
