// Linear layer of unquantised activations with 4-bit weights and group scales:
//   y[t, n] = sum_g scale[n, g] * sum_{c in group g} x[t, c] * (code[n, c] - zero[n, g])
// MXFP4: E2M1 codes, one E8M0 byte per 32 columns, no zero. INT4: codes 0 .. 15, a scale
// of the activations' type and a zero point (8 without) per 32, 64 or 128 columns.
//
// Here for few tokens (w4_gemm.hip has many): a pass over the weights, which HBM bounds.
// The codes less their zero points become 16-bit values exactly and enter
// V_MFMA_F32_16X16X32 as they are; the scale multiplies the fp32 sum of its group. So no
// weight is rounded, and every scale that fp32 holds does its work (an MXFP4 scale is far
// outside fp16, and scale * code of INT4 needs 15 bits where bf16 has 8).
//
// A workgroup has 16 NT weight rows and 16 MT tokens; its waves share K in steps of 128
// columns and add up through LDS at the end. Rows come in by copies straight to LDS
// (GLOBAL_LOAD_LDS), each of 16 rows x 64 bytes, four neighbouring lanes a row's 64: a
// step's codes of 16 rows, or the activations of 16 tokens in a block of 32 columns. (A
// load in the matrix operand's own layout has neighbouring lanes in different rows, and
// the address path takes it apart lane by lane: 64 tokens of 7168 -> 7168 took 42 to 89
// us.) Every wave has copies of its own under way, DW steps of codes and RX blocks of
// activations ahead, and waits for nobody else's.
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

// 4 x 4 transposition between the four rows of 16 lanes and four registers: afterwards
// register i of lane row q is what register q of lane row i was.
__device__ __forceinline__ void transpose4(uint32_t (&d)[4]) {
  auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
  auto e = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto f = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  d[0] = e[0]; d[1] = e[1]; d[2] = f[0]; d[3] = f[1];
}

// Words at any address.
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));

// The scales (and zero points) of a row's step of 128 columns. GL: log2 of a group's columns.
template <int DT, bool INT, int GL>
struct Scales {
  static constexpr int N = 128 >> GL;
  static constexpr int SW = INT && N == 4 ? 2 : 1, WORDS = INT ? SW + 1 : 1;   // as they lie in memory, then the zero points
  uint32_t w[WORDS];
  // row: the row's scales; zeros: its zero points, or null; step: which 128 columns
  __device__ __forceinline__ void load(const uint8_t* row, const uint8_t* zeros, int64_t step) {
    if constexpr (!INT) {
      w[0] = *(const u32_any*)(row + 4 * step);
    } else {
      const uint8_t* p = row + 2 * N * step;
      if constexpr (N == 1) w[0] = *(const uint16_t*)p;
      else w[0] = *(const u32_any*)p;
      if constexpr (N == 4) w[1] = *(const u32_any*)(p + 4);
      w[SW] = 0x08080808u;
      if (zeros != nullptr) {
        if constexpr (N == 1) w[SW] = zeros[step];
        else if constexpr (N == 2) w[SW] = *(const u16_any*)(zeros + 2 * step);
        else w[SW] = *(const u32_any*)(zeros + 4 * step);
      }
    }
  }
  __device__ __forceinline__ float scale(int g) const {
    if constexpr (!INT) return e8m0((w[0] >> (8 * g)) & 0xFFu);
    else return g % 2 ? hi_f32<DT>(w[g / 2]) : lo_f32<DT>(w[g / 2]);
  }
  __device__ __forceinline__ uint32_t zero(int g) const {
    if constexpr (INT) return zero_bits<DT>((w[SW] >> (8 * g)) & 0xFFu);
    else return 0;
  }
};

// A copy of 16 bytes a lane to LDS, lane i's to lds + 16 i. Inline, so that the compiler does not wait
// for it before every LDS read; wait_copies<N>() does until no more than N of the wave's are under way.
__device__ __forceinline__ void copy16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// The wave's LDS reads are done: a copy may take their place.
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <int DT, bool INT>
__device__ __forceinline__ u32v4 expand(uint32_t d, uint32_t zero) {
  if constexpr (INT) return expand_int<DT>(d, zero);
  else return expand_fp4<DT>(d, 1.0f);
}

constexpr int CHUNK = 64;     // steps whose scales are in LDS together

// LDS of a workgroup: each wave's copies, then the scales; the sums at the end take their place.
template <int WORDS, int NT, int MT, int W, int DW, int RX>
constexpr int W4_RING = W * (DW * NT + RX * MT) * 1024;
template <int WORDS, int NT, int MT, int W, int DW, int RX>
constexpr int W4_SMEM = W4_RING<WORDS, NT, MT, W, DW, RX> + WORDS * CHUNK * (16 * NT + 1) * 4;

template <int DT, bool INT, int GL, int NT, int MT, int W, int DW, int RX>
__global__ __launch_bounds__(64 * W) void k_w4(W4Args a) {
  typedef Scales<DT, INT, GL> Sc;
  constexpr int RING = W4_RING<Sc::WORDS, NT, MT, W, DW, RX>, SMEM = W4_SMEM<Sc::WORDS, NT, MT, W, DW, RX>;
  constexpr int G = 128 >> GL, B = 4 / G;        // groups of a step, blocks of 32 columns of a group
  constexpr int PITCH = 16 * NT + 1;             // of a step's scales
  static_assert(SMEM >= W * NT * MT * 1024 && SMEM <= 160 * 1024, "LDS");
  static_assert(RX >= 2 && RX + 4 <= 4 * DW && RX * MT + NT < 64, "the waits for the copies");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[SMEM];
  uint32_t* sw = (uint32_t*)(smem + RING);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * NT, t0 = (int64_t)blockIdx.y * 16 * MT;
  const int steps = (int)(a.K / 128);
  const int64_t groups = a.K >> GL;
  // what this lane copies: of row lane / 4 the 16 bytes that stand at lane % 4 in LDS. Chunk c of row i stands at c ^
  // (i / 4 % 4), so that 16 rows' reads of one chunk fall in 16 bank groups.
  const int cr = lane >> 2, cc = (lane & 3) ^ ((lane >> 4) & 3);
  const uint8_t* wsrc[NT];
  const char* xsrc[MT];
#pragma unroll
  for (int i = 0; i < NT; ++i) wsrc[i] = a.w + min(n0 + 16 * i + cr, a.N - 1) * (a.K / 2) + 16 * cc;
#pragma unroll
  for (int j = 0; j < MT; ++j) xsrc[j] = at<DT>(a.x, min(t0 + 16 * j + cr, a.M - 1) * a.ldx) + 16 * cc;
  uint8_t* ring = smem + wave * (DW * NT + RX * MT) * 1024;
  const uint32_t lds = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)ring;
  const uint32_t at16 = r * 64 + ((q ^ (r >> 2)) << 4);       // where this lane reads row r's chunk q
  f32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  for (int c0 = 0; c0 < steps; c0 += CHUNK) {
    const int cn = min(CHUNK, steps - c0);
    const int mine = wave < cn ? (cn - wave + W - 1) / W : 0;      // steps c0 + wave, c0 + wave + W, ..
    const int blocks = 4 * mine;
    auto copy_w = [&](int i) {
#pragma unroll
      for (int k = 0; k < NT; ++k)
        copy16(wsrc[k] + (int64_t)(c0 + wave + W * i) * 64, lds + ((i % DW) * NT + k) * 1024);
    };
    auto copy_x = [&](int n) {
#pragma unroll
      for (int j = 0; j < MT; ++j)
        copy16(xsrc[j] + ((int64_t)(c0 + wave + W * (n >> 2)) * 256 + (n & 3) * 64),
               lds + (DW * NT + (n % RX) * MT + j) * 1024);
    };
    // all codes that the ring takes, then the activations
    for (int i = 0; i < min(DW, mine); ++i) copy_w(i);
    for (int n = 0; n < min(RX, blocks); ++n) copy_x(n);
    for (int i = threadIdx.x; i < cn * 16 * NT; i += 64 * W) {
      const int row = i / cn, s = i - row * cn;
      const int64_t n = min(n0 + row, a.N - 1);
      Sc t;
      t.load((const uint8_t*)a.scales + n * groups * (INT ? 2 : 1), a.zeros == nullptr ? nullptr : a.zeros + n * groups,
             c0 + s);
#pragma unroll
      for (int k = 0; k < Sc::WORDS; ++k) sw[(k * CHUNK + s) * PITCH + row] = t.w[k];
    }
    __syncthreads();
    for (int i = 0; i < mine; ++i) {
      uint32_t d[NT][4];
      Sc sc[NT];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        u32v4 x[B][MT];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int n = 4 * i + g * B + b;
          // Copied after block n's activations were those of RX - 1 more blocks (near the end fewer: then all is
          // waited for), and, if the step before ended at most RX blocks ago and had any to copy, its codes. Step i's
          // own codes were copied before block 4 i's activations, since RX + 4 <= 4 DW.
          constexpr int X = (RX - 1) * MT;
          if (n + RX > blocks) wait_copies<0>();
          else if (g * B + b < RX && i > 0 && i - 1 + DW < mine) wait_copies<X + NT>();
          else wait_copies<X>();
          if (g * B + b == 0) {
#pragma unroll
            for (int k = 0; k < NT; ++k) {
              const u32v4 v = *(const u32v4*)(ring + ((i % DW) * NT + k) * 1024 + at16);
#pragma unroll
              for (int e = 0; e < 4; ++e) d[k][e] = v[e];
#pragma unroll
              for (int e = 0; e < Sc::WORDS; ++e) sc[k].w[e] = sw[(e * CHUNK + wave + W * i) * PITCH + 16 * k + r];
              transpose4(d[k]);      // block b's codes: columns 8 q .. 8 q + 7 of it in d[k][b]
            }
          }
#pragma unroll
          for (int j = 0; j < MT; ++j) x[b][j] = *(const u32v4*)(ring + (DW * NT + (n % RX) * MT + j) * 1024 + at16);
          wait_reads();
          if (n + RX < blocks) copy_x(n + RX);
        }
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          const float scale = sc[k].scale(g);
          const uint32_t zero = sc[k].zero(g);
          u32v4 wv[B];
#pragma unroll
          for (int b = 0; b < B; ++b) wv[b] = expand<DT, INT>(d[k][g * B + b], zero);
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int b = 0; b < B; ++b) p = mfma<DT>(x[b][j], wv[b], p);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[k][j][e] = fmaf(scale, p[e], acc[k][j][e]);
          }
        }
      }
      if (i + DW < mine) copy_w(i + DW);
    }
    __syncthreads();               // the scales' place is free
  }
  // up to three blocks behind the last whole step, by the wave that has the fewest steps
  if (GL < 7 && wave == W - 1) {
    for (int blk = 4 * steps; blk < (int)(a.K / 32); ++blk) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int64_t n = min(n0 + 16 * i + r, a.N - 1);
        const int g = blk >> (GL - 5);
        float scale;
        uint32_t zero = 0;
        if constexpr (INT) {
          scale = Raw<DT, 1>{{((const uint16_t*)a.scales)[n * groups + g]}}.get(0);
          zero = zero_bits<DT>(a.zeros != nullptr ? a.zeros[n * groups + g] : 8u);
        } else {
          scale = e8m0(((const uint8_t*)a.scales)[n * groups + g]);
        }
        const u32v4 wv = expand<DT, INT>(*(const uint32_t*)(a.w + n * (a.K / 2) + (int64_t)blk * 16 + 4 * q), zero);
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const f32x4 p = mfma<DT>(*(const u32v4*)(at<DT>(a.x, min(t0 + 16 * j + r, a.M - 1) * a.ldx + 8 * q) + (int64_t)blk * 64), wv, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(scale, p[e], acc[i][j][e]);
        }
      }
    }
  }

  // lane (r, q) has tokens 4 q + e of weight row r
  float(*part)[NT * MT][4][64] = (float(*)[NT * MT][4][64])smem;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[wave][i * MT + j][e][lane] = acc[i][j][e];
  __syncthreads();
  const int rows = (int)min(a.M - t0, (int64_t)16 * MT);
  for (int o = threadIdx.x; o < rows * 16 * NT; o += 64 * W) {
    const int t = o / (16 * NT), n = o % (16 * NT);
    if (n0 + n >= a.N) continue;
    const float* p = &part[0][n / 16 * MT + t / 16][t % 4][t % 16 / 4 * 16 + n % 16];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) sum += p[i * (NT * MT * 4 * 64)];
    Raw<DT, 1> out;
    out.set(&sum);
    out.store(at<DT>(a.y, (t0 + t) * a.ldy + n0), (uint32_t)n);
  }
}

}  // namespace

hipError_t launch_w4(const W4Args& a, hipStream_t s) {
  if (a.M > W4_FEW) return launch_w4_gemm(a, s);
  const auto go = [&](auto d, auto in, auto gl) {
    constexpr int DT = decltype(d)::value, GL = decltype(gl)::value;
    constexpr bool I = decltype(in)::value;
    const unsigned one = (unsigned)((a.N + 15) / 16), two = (unsigned)((a.N + 31) / 32);
    if (a.M <= 16) {
      if (two >= 192) k_w4<DT, I, GL, 2, 1, 8, 3, 6><<<two, 512, 0, s>>>(a);
      else k_w4<DT, I, GL, 1, 1, 8, 4, 8><<<one, 512, 0, s>>>(a);
    } else if (a.M <= 32) {
      k_w4<DT, I, GL, 2, 2, 8, 2, 4><<<two, 512, 0, s>>>(a);
    } else {
      k_w4<DT, I, GL, 2, 4, 8, 2, 3><<<two, 512, 0, s>>>(a);
    }
  };
  const auto types = [&](auto in, auto gl) {
    if (a.dt == DT_BF16) go(DtC<DT_BF16>(), in, gl);
    else go(DtC<DT_F16>(), in, gl);
  };
  using std::integral_constant;
  if (!a.int4) types(std::false_type(), integral_constant<int, 5>());
  else if (a.group_log2 == 5) types(std::true_type(), integral_constant<int, 5>());
  else if (a.group_log2 == 6) types(std::true_type(), integral_constant<int, 6>());
  else types(std::true_type(), integral_constant<int, 7>());
  return hipGetLastError();
}

}  // namespace mx
