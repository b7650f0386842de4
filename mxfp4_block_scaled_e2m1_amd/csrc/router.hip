// The router in front of the experts: scores, top-k and weights, the balance
// loss with the experts' counts, and the gradient of both.
//
// With s the scores of a token's logits z (softmax over the experts, or the
// sigmoid of each) and p the same as shares of one (softmax: p = s, sigmoid:
// p = s / sum s):
//   gate      the k experts of the largest s (+ bias), the lower index first;
//             w_j = scale * s_j  (renorm: over the chosen ones' sum)
//   balance   loss[q] = coef E / (k n^2) * sum_e c[q,e] * sum_t p[t,e] over the n
//             tokens t of sequence q, c[q,e] its slots that name e
//   gradient  with B[q,e] = coef E / (k n^2) d_loss[q] c[q,e], and x_j what slot j
//             gives the score of its expert times that score,
//               x_j = scale s_j d_w_j   (renorm: w_j (d_w_j - sum_i w_i d_w_i / scale))
//             softmax  dz_e = sum_{j names e} x_j - [no renorm] p_e sum_j x_j + p_e (B_e - sum p B)
//             sigmoid  dz_e = (1 - s_e) (sum_{j names e} x_j + p_e (B_e - sum p B))
//             since ds_e/dz = s_e (1 - s_e) for the sigmoid, and for the softmax's
//             renormalised weights what leaves through the sum is zero.
//
// An expert whose logit is -inf is off: it is never chosen and its share is 0.
//
// A token's logits are a few hundred values: a group of 16 or 32 lanes holds them
// in registers, 4 to 16 a lane (expert i * G + lane), so that a wave has two to four
// tokens in flight and what is done lane by lane (exponentials, the search for a
// lane's largest) is shared by all of them; sums and maxima over the group are four
// DPP rotations of a row of 16 lanes and one row swap. All of it is bound by
// latency and launches: a training batch of 4096 x 384 fp32 logits is 6.3 MB.
#include <algorithm>

#include "rows.h"

namespace mx {

namespace {

constexpr int GATE_THREADS = 256;

// op over a group of G lanes (16: a DPP row, 32: two rows), the result in all of them.
template <int G, class Op>
__device__ __forceinline__ uint32_t group_all(uint32_t v, Op op) {
  v = op(v, __builtin_amdgcn_update_dpp(0u, v, 0x128, 0xF, 0xF, false));   // row_ror 8, 4, 2, 1
  v = op(v, __builtin_amdgcn_update_dpp(0u, v, 0x124, 0xF, 0xF, false));
  v = op(v, __builtin_amdgcn_update_dpp(0u, v, 0x122, 0xF, 0xF, false));
  v = op(v, __builtin_amdgcn_update_dpp(0u, v, 0x121, 0xF, 0xF, false));
  if constexpr (G == 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_all<G>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int G>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_all<G>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}
template <int G>
__device__ __forceinline__ float group_fmax(float v) {
  return __uint_as_float(group_all<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int G>
__device__ __forceinline__ float group_add(float v) {
  return __uint_as_float(group_all<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int G>
__device__ __forceinline__ double group_add(double v) {
  auto step = [&](auto move) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t o = ((uint64_t)move((uint32_t)(b >> 32)) << 32) | move((uint32_t)b);
    v += __builtin_bit_cast(double, o);
  };
  step([](uint32_t x) -> uint32_t { return __builtin_amdgcn_update_dpp(0u, x, 0x128, 0xF, 0xF, false); });
  step([](uint32_t x) -> uint32_t { return __builtin_amdgcn_update_dpp(0u, x, 0x124, 0xF, 0xF, false); });
  step([](uint32_t x) -> uint32_t { return __builtin_amdgcn_update_dpp(0u, x, 0x122, 0xF, 0xF, false); });
  step([](uint32_t x) -> uint32_t { return __builtin_amdgcn_update_dpp(0u, x, 0x121, 0xF, 0xF, false); });
  if constexpr (G == 32) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
    v = __builtin_bit_cast(double, ((uint64_t)hi[0] << 32) | lo[0]) +
        __builtin_bit_cast(double, ((uint64_t)hi[1] << 32) | lo[1]);
  }
  return v;
}

template <int DT>
__device__ __forceinline__ float logit(const char* row, int e) {
  Raw<DT, 1> r;
  r.load(row, (uint32_t)e);
  return r.get(0);
}

// The lane's logits of a token; -inf behind the last expert.
template <int DT, int G, int V>
__device__ __forceinline__ void load_logits(const char* row, int E, int l, float (&z)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) z[i] = i * G + l < E ? logit<DT>(row, i * G + l) : -INFINITY;
}

// The shares p of the lane's logits, 0 for all where no expert is on (or, of
// sigmoids, none is above 0). Also the softmax's largest logit and sum.
template <int G, int V>
__device__ __forceinline__ void shares(const float (&z)[V], bool sigmoid, float (&p)[V], float& top, float& total) {
  top = 0.0f;
  if (!sigmoid) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, z[i]);
    top = group_fmax<G>(m);
    if (top == -INFINITY) top = 0.0f;
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    p[i] = sigmoid ? 1.0f / (1.0f + expf(-z[i])) : expf(z[i] - top);
    sum += p[i];
  }
  total = group_add<G>(sum);
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] *= inv;
}

// A float's place among the floats as an unsigned number, -0 with +0. 0 is kept for an
// expert that is off, 1 for a NaN, which so comes behind every number.
__device__ __forceinline__ uint32_t place(float z) {
  const uint32_t u = __float_as_uint(z + 0.0f);
  if (z == -INFINITY) return 0u;
  if (z != z) return 1u;
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint64_t place(double z) {
  const uint64_t u = __builtin_bit_cast(uint64_t, z + 0.0);
  if (z != z) return 1u;
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// Scores as they are chosen by. Without a bias the logits themselves: their order is
// the scores'. With one the sum is formed in 64 bits: of 4096 tokens' neighbours in
// order some lie closer than 32 bits of a score tell apart.
template <int G, int V, bool BIAS>
struct Keys;
template <int G, int V>
struct Keys<G, V, false> {
  uint32_t key[V];
  __device__ __forceinline__ void make(const float (&z)[V], bool, const float*, int, int) {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = place(z[i]);
  }
  // The group's best expert, taken out of the keys; -1 where all that is left is off.
  __device__ __forceinline__ int take(int l) {
    uint32_t b = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > b) { b = key[i]; at = i * G + l; }
    const uint32_t top = group_max<G>(b);
    const int e = (int)group_min<G>(b == top ? (uint32_t)at : 0xFFFFu);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * G + l == e) key[i] = 0;
    return top == 0 ? -1 : e;
  }
};
template <int G, int V>
struct Keys<G, V, true> {
  uint64_t key[V];
  __device__ __forceinline__ void make(const float (&z)[V], bool sigmoid, const float* bias, int E, int l) {
    double s[V], sum = 0.0;
    float m = -INFINITY;
    if (!sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, z[i]);
      m = group_fmax<G>(m);
      if (m == -INFINITY) m = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = sigmoid ? 1.0 / (1.0 + exp(-(double)z[i])) : exp((double)z[i] - (double)m);
      sum += s[i];
    }
    double inv = 1.0;
    if (!sigmoid) inv = 1.0 / group_add<G>(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * G + l;
      key[i] = z[i] == -INFINITY ? 0u : place(s[i] * inv + (e < E ? (double)bias[e] : 0.0));
    }
  }
  __device__ __forceinline__ int take(int l) {
    uint64_t b = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > b) { b = key[i]; at = i * G + l; }
    const uint32_t hi = group_max<G>((uint32_t)(b >> 32));
    const uint32_t lo = group_max<G>((uint32_t)(b >> 32) == hi ? (uint32_t)b : 0u);
    const int e = (int)group_min<G>(b == (((uint64_t)hi << 32) | lo) ? (uint32_t)at : 0xFFFFu);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * G + l == e) key[i] = 0;
    return (hi | lo) == 0 ? -1 : e;
  }
};

// What the lanes of a wave wrote to LDS is there for all of them.
__device__ __forceinline__ void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The scores of the chosen experts, in the lane's slots l, l + G, .. (0 for a slot
// without an expert): over their sum when `renorm`. The softmax's renormalised ones
// are a softmax over the chosen logits, which no underflow of the others' spoils.
template <int DT, int G>
__device__ __forceinline__ void slot_scores(const char* row, const int32_t* sel, int k, int E, int l, bool sigmoid,
                                            bool renorm, float top, float total, float (&s)[MAX_TOPK / G]) {
  float z[MAX_TOPK / G], m = -INFINITY;
#pragma unroll
  for (int q = 0; q < MAX_TOPK / G; ++q) {
    const int j = q * G + l;
    const int e = j < k ? sel[j] : -1;
    z[q] = (unsigned)e < (unsigned)E ? logit<DT>(row, e) : -INFINITY;
    m = fmaxf(m, z[q]);
  }
  if (!sigmoid && renorm) {
    top = group_fmax<G>(m);
    if (top == -INFINITY) top = 0.0f;
  }
  float sum = 0.0f;
#pragma unroll
  for (int q = 0; q < MAX_TOPK / G; ++q) {
    s[q] = sigmoid ? 1.0f / (1.0f + expf(-z[q])) : expf(z[q] - top);
    sum += s[q];
  }
  if (renorm) total = group_add<G>(sum);
  else if (sigmoid) total = 1.0f;
#pragma unroll
  for (int q = 0; q < MAX_TOPK / G; ++q) s[q] = total == 0.0f ? 0.0f : s[q] / total;
}

template <int DT, int G, int V, bool BIAS>
__global__ __launch_bounds__(GATE_THREADS) void k_gate(const void* __restrict__ logits, int64_t T, int E, bool sigmoid,
                                                       const float* __restrict__ bias, int k, bool renorm, float scale,
                                                       int32_t* __restrict__ ids, float* __restrict__ w) {
  constexpr int PER = GATE_THREADS / G;
  __shared__ int32_t sel[PER][MAX_TOPK];
  const int l = threadIdx.x % G, g = threadIdx.x / G;
  for (int64_t t0 = (int64_t)blockIdx.x * PER; t0 < T; t0 += (int64_t)gridDim.x * PER) {
    const bool live = t0 + g < T;
    const int64_t t = live ? t0 + g : T - 1;        // all lanes go along: DPP reads only active ones
    const char* row = at<DT>(logits, t * E);
    float z[V], top = 0.0f, total = 1.0f;
    load_logits<DT, G, V>(row, E, l, z);
    if (!sigmoid && !renorm) {
      float p[V];
      shares<G, V>(z, false, p, top, total);
    }
    Keys<G, V, BIAS> keys;
    keys.make(z, sigmoid, bias, E, l);
    for (int j = 0; j < k; ++j) {
      const int e = keys.take(l);
      if (l == 0) sel[g][j] = e;
    }
    wave_lds();
    float s[MAX_TOPK / G];
    slot_scores<DT, G>(row, sel[g], k, E, l, sigmoid, renorm, top, total, s);
#pragma unroll
    for (int q = 0; q < MAX_TOPK / G; ++q) {
      const int j = q * G + l;
      if (live && j < k) {
        ids[t * k + j] = sel[g][j];
        w[t * k + j] = scale * s[q];
      }
    }
    wave_lds();
  }
}

// Tokens a .. b of sequence q; none where the offsets are out of order or range.
__device__ __forceinline__ void tokens_of(const int32_t* seq_off, int64_t q, int64_t T, int64_t& a, int64_t& b) {
  a = seq_off != nullptr ? min(max((int64_t)seq_off[q], (int64_t)0), T) : 0;
  b = seq_off != nullptr ? min(max((int64_t)seq_off[q + 1], a), T) : T;
}

constexpr int BAL_THREADS = 512;
constexpr int BAL_WAVES = BAL_THREADS / 64;

// One expert's count and sum of shares in a sequence are summed by one thread, which
// has them as `c` and `p`; the workgroup sums the loss.
__device__ __forceinline__ void balance_out(int64_t q, int64_t n, int E, int k, float coef, int c, float p, float* red,
                                            float* loss, int32_t* counts) {
  const int e = threadIdx.x;
  if (e < E) counts[q * E + e] = c;
  const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
  float v[1] = {e < E ? ((float)c * inv) * (p * inv) : 0.0f};
  group_sum<1>(v, red, BAL_WAVES, threadIdx.x & 63, threadIdx.x >> 6);
  if (e == 0) loss[q] = coef * ((float)E / (float)k) * v[0];
}

// Workgroup (split, sequence): the sums of p and the counts over its part of the
// sequence's tokens.
template <int DT, int G, int V>
__global__ __launch_bounds__(BAL_THREADS) void k_balance(const void* __restrict__ logits, int64_t T, int E, bool sigmoid,
                                                         const int32_t* __restrict__ ids, int k,
                                                         const int32_t* __restrict__ seq_off, float coef,
                                                         float* __restrict__ part_p, int32_t* __restrict__ part_c,
                                                         float* __restrict__ loss, int32_t* __restrict__ counts) {
  constexpr int PER = BAL_THREADS / G;
  __shared__ float sums[BAL_WAVES][G * V];
  __shared__ int32_t hist[BAL_THREADS];
  __shared__ float red[16];
  const int64_t q = blockIdx.y;
  int64_t a, b;
  tokens_of(seq_off, q, T, a, b);
  const int64_t per = (b - a + gridDim.x - 1) / gridDim.x;
  const int64_t lo = min(b, a + per * blockIdx.x), hi = min(b, lo + per);
  hist[threadIdx.x] = 0;
  __syncthreads();
  for (int64_t i = lo * k + threadIdx.x; i < hi * k; i += BAL_THREADS) {
    const uint32_t e = (uint32_t)ids[i];
    if (e < (uint32_t)E) atomicAdd(&hist[e], 1);
  }
  const int l = threadIdx.x % G, g = threadIdx.x / G;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  for (int64_t t0 = lo; t0 < hi; t0 += PER) {
    const bool live = t0 + g < hi;
    float z[V], p[V], top, total;
    load_logits<DT, G, V>(at<DT>(logits, (live ? t0 + g : hi - 1) * E), E, l, z);
    shares<G, V>(z, sigmoid, p, top, total);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += live ? p[i] : 0.0f;
  }
  // over the wave's groups, then the waves
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (G == 16) {
      const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[i]), __float_as_uint(acc[i]), false, false);
      acc[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[i]), __float_as_uint(acc[i]), false, false);
    acc[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    if ((threadIdx.x & 63) < G) sums[threadIdx.x >> 6][i * G + l] = acc[i];
  }
  __syncthreads();
  float p = 0.0f;
  if (threadIdx.x < G * V) {
#pragma unroll
    for (int i = 0; i < BAL_WAVES; ++i) p += sums[i][threadIdx.x];
  }
  const int c = hist[threadIdx.x];
  if (part_p == nullptr) {
    balance_out(q, b - a, E, k, coef, c, p, red, loss, counts);
  } else if ((int)threadIdx.x < E) {
    const int64_t at = (q * gridDim.x + blockIdx.x) * E + threadIdx.x;
    part_p[at] = p;
    part_c[at] = c;
  }
}

// The parts of a sequence, in their order.
__global__ __launch_bounds__(BAL_THREADS) void k_balance_sum(const float* __restrict__ part_p,
                                                             const int32_t* __restrict__ part_c, int splits, int64_t T,
                                                             int E, int k, const int32_t* __restrict__ seq_off, float coef,
                                                             float* __restrict__ loss, int32_t* __restrict__ counts) {
  __shared__ float red[16];
  const int64_t q = blockIdx.x;
  int64_t a, b;
  tokens_of(seq_off, q, T, a, b);
  float p = 0.0f;
  int c = 0;
  if ((int)threadIdx.x < E) {
    const int64_t at = q * splits * E + threadIdx.x;
#pragma unroll 8
    for (int i = 0; i < splits; ++i) {
      p += part_p[at + (int64_t)i * E];
      c += part_c[at + (int64_t)i * E];
    }
  }
  balance_out(q, b - a, E, k, coef, c, p, red, loss, counts);
}

struct GateGrad {
  const void* logits;
  int64_t T;
  int E;
  bool sigmoid;
  const int32_t* ids;
  int k;
  bool renorm;
  float scale;
  const float* d_w;          // may be null
  const int32_t* counts;     // may be null
  const int32_t* seq_off;
  int64_t S;
  float coef;
  const float* d_loss;
  void* d_logits;
};

template <int DT, int G, int V>
__global__ __launch_bounds__(GATE_THREADS) void k_gate_grad(GateGrad a) {
  constexpr int PER = GATE_THREADS / G, Q = MAX_TOPK / G;
  __shared__ int32_t sel[PER][MAX_TOPK];
  __shared__ float val[PER][MAX_TOPK];
  const int l = threadIdx.x % G, g = threadIdx.x / G, E = a.E, k = a.k;
  for (int64_t t0 = (int64_t)blockIdx.x * PER; t0 < a.T; t0 += (int64_t)gridDim.x * PER) {
    const bool live = t0 + g < a.T;
    const int64_t t = live ? t0 + g : a.T - 1;
    const char* row = at<DT>(a.logits, t * E);
    float z[V], p[V], d[V], top, total;
    load_logits<DT, G, V>(row, E, l, z);
    shares<G, V>(z, a.sigmoid, p, top, total);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.0f;
    if (a.counts != nullptr) {
      // the last sequence that starts at or before t, if it reaches t
      int64_t lo = 0, n = a.S;
      if (a.seq_off != nullptr) {
        while (n > 1) {
          const int64_t half = n >> 1;
          if (a.seq_off[lo + half] <= t) { lo += half; n -= half; }
          else n = half;
        }
      }
      int64_t first, last;
      tokens_of(a.seq_off, lo, a.T, first, last);
      const float inv = 1.0f / (float)max(last - first, (int64_t)1);
      const float f = t >= first && t < last ? a.coef * ((float)E / (float)k) * a.d_loss[lo] * inv * inv : 0.0f;
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * G + l;
        d[i] = e < E ? f * (float)a.counts[lo * E + e] : 0.0f;
        dot = fmaf(p[i], d[i], dot);
      }
      dot = group_add<G>(dot);
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = p[i] * (d[i] - dot);
    }
    if (a.d_w != nullptr) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int j = q * G + l;
        if (j < k) sel[g][j] = a.ids[t * k + j];
      }
      wave_lds();
      float s[Q], dw[Q], mean = 0.0f;
      slot_scores<DT, G>(row, sel[g], k, E, l, a.sigmoid, a.renorm, top, total, s);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int j = q * G + l;
        const bool has = j < k && (unsigned)sel[g][j] < (unsigned)E;
        dw[q] = has ? a.d_w[t * k + j] : 0.0f;
        mean = fmaf(s[q], dw[q], mean);
      }
      mean = a.renorm ? group_add<G>(mean) : 0.0f;
      float sum = 0.0f;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int j = q * G + l;
        const float x = a.scale * s[q] * (dw[q] - mean);
        sum += x;
        if (j < k) val[g][j] = x;
      }
      wave_lds();
      if (!a.sigmoid && !a.renorm) {
        sum = group_add<G>(sum);
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = fmaf(-p[i], sum, d[i]);
      }
      for (int j = 0; j < k; ++j) {
        const int e = sel[g][j];
        const float x = val[g][j];
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] += i * G + l == e ? x : 0.0f;
      }
      wave_lds();
    }
    char* out = at<DT>(a.d_logits, t * E);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * G + l;
      if (a.sigmoid) d[i] *= 1.0f / (1.0f + expf(z[i]));
      Raw<DT, 1> o;
      o.set(&d[i]);
      if (live && e < E) o.store(out, (uint32_t)e);
    }
  }
}

// f(lanes of a token, values of a lane). 16 lanes while a lane's values are few.
template <class F>
void dispatch_experts(int E, F&& f) {
  using std::integral_constant;
  if (E <= 64) f(integral_constant<int, 16>(), integral_constant<int, 4>());
  else if (E <= 128) f(integral_constant<int, 16>(), integral_constant<int, 8>());
  else if (E <= 256) f(integral_constant<int, 32>(), integral_constant<int, 8>());
  else if (E <= 384) f(integral_constant<int, 32>(), integral_constant<int, 12>());
  else f(integral_constant<int, 32>(), integral_constant<int, 16>());
}

unsigned token_grid(int64_t T, int per) { return (unsigned)std::min<int64_t>((T + per - 1) / per, (int64_t)1 << 20); }

}  // namespace

hipError_t launch_gate(const void* logits, DType dt, int64_t T, int E, bool sigmoid, const float* bias, int k,
                       bool renorm, float scale, int32_t* ids, float* w, hipStream_t s) {
  dispatch_dt(dt, [&](auto d) {
    dispatch_experts(E, [&](auto lanes, auto values) {
      constexpr int D = decltype(d)::value, G = decltype(lanes)::value, V = decltype(values)::value;
      const unsigned grid = token_grid(T, GATE_THREADS / G);
      if (bias != nullptr)
        k_gate<D, G, V, true><<<grid, GATE_THREADS, 0, s>>>(logits, T, E, sigmoid, bias, k, renorm, scale, ids, w);
      else
        k_gate<D, G, V, false><<<grid, GATE_THREADS, 0, s>>>(logits, T, E, sigmoid, bias, k, renorm, scale, ids, w);
    });
  });
  return hipGetLastError();
}

int balance_splits(int64_t T, int64_t S) {
  // at most 64 parts of a sequence, of 32 tokens or more on average, about 512 workgroups
  return (int)std::max<int64_t>(1, std::min({(int64_t)64, T / S / 32, (512 + S - 1) / S}));
}

hipError_t launch_balance(const void* logits, DType dt, int64_t T, int E, bool sigmoid, const int32_t* ids, int k,
                          const int32_t* seq_off, int64_t S, float coef, float* part, float* loss, int32_t* counts,
                          hipStream_t s) {
  const int splits = balance_splits(T, S);
  float* pp = splits > 1 ? part : nullptr;
  int32_t* pc = splits > 1 ? (int32_t*)(part + S * splits * E) : nullptr;
  // (a grid's y is at most 65535)
  for (int64_t q0 = 0; q0 < S; q0 += 32768) {
    const unsigned n = (unsigned)std::min<int64_t>(S - q0, 32768);
    dispatch_dt(dt, [&](auto d) {
      dispatch_experts(E, [&](auto lanes, auto values) {
        constexpr int D = decltype(d)::value, G = decltype(lanes)::value, V = decltype(values)::value;
        k_balance<D, G, V><<<dim3((unsigned)splits, n), BAL_THREADS, 0, s>>>(
            logits, T, E, sigmoid, ids, k, seq_off == nullptr ? nullptr : seq_off + q0, coef,
            pp == nullptr ? nullptr : pp + q0 * splits * E, pc == nullptr ? nullptr : pc + q0 * splits * E, loss + q0,
            counts + q0 * E);
      });
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (splits > 1)
    k_balance_sum<<<(unsigned)S, BAL_THREADS, 0, s>>>(pp, pc, splits, T, E, k, seq_off, coef, loss, counts);
  return hipGetLastError();
}

hipError_t launch_gate_grad(const void* logits, DType dt, int64_t T, int E, bool sigmoid, const int32_t* ids, int k,
                            bool renorm, float scale, const float* d_w, const int32_t* counts, const int32_t* seq_off,
                            int64_t S, float coef, const float* d_loss, void* d_logits, hipStream_t s) {
  const GateGrad a{logits, T, E, sigmoid, ids, k, renorm, scale, d_w, counts, seq_off, S, coef, d_loss, d_logits};
  dispatch_dt(dt, [&](auto d) {
    dispatch_experts(E, [&](auto lanes, auto values) {
      constexpr int D = decltype(d)::value, G = decltype(lanes)::value, V = decltype(values)::value;
      k_gate_grad<D, G, V><<<token_grid(T, GATE_THREADS / G), GATE_THREADS, 0, s>>>(a);
    });
  });
  return hipGetLastError();
}

}  // namespace mx
