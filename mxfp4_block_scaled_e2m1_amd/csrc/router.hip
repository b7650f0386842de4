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

// The lane's logits of a token; -inf behind the last expert. Every load is made (of the last expert where there is none), so
// that they go out one behind the other.
template <int DT, int G, int V>
__device__ __forceinline__ void load_logits(const char* row, int E, int l, float (&z)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) z[i] = logit<DT>(row, min(i * G + l, E - 1));
#pragma unroll
  for (int i = 0; i < V; ++i) z[i] = i * G + l < E ? z[i] : -INFINITY;
}

// e^d for d <= 0, to about a step and a half of fp32; 0 below 2^-126. The rounding of d / ln 2 goes back into the result:
// without that a probability of e^-20 is off by 40 half steps.
__device__ __forceinline__ float exp_down(float d) {
  d = d < -104.0f ? -104.0f : d;               // (a NaN stays)
  const float t = d * 0x1.715476p+0f;
  const float r = fmaf(d, 0x1.4ae0cp-26f, fmaf(d, 0x1.715476p+0f, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, r * 0x1.62e43p-1f, e);
}
// 1 / (1 + e^-z), to about three steps.
__device__ __forceinline__ float sigmoid_f32(float z) {
  const float e = exp_down(-fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + e);
  return z < 0.0f ? e * r : r;
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
    p[i] = sigmoid ? sigmoid_f32(z[i]) : exp_down(z[i] - top);
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
    s[q] = sigmoid ? sigmoid_f32(z[q]) : exp_down(z[q] - top);
    sum += s[q];
  }
  if (renorm) total = group_add<G>(sum);
  else if (sigmoid) total = 1.0f;
#pragma unroll
  for (int q = 0; q < MAX_TOPK / G; ++q) s[q] = total == 0.0f ? 0.0f : s[q] / total;
}

// What 32 bits of s + b are off by at most: the exponential's argument is rounded to 2^-24 of itself, which moves a
// sigmoid by 2^-24 |z| s (1 - s) < 2^-26 and a softmax's share by less than 2^-25; four more roundings, the softmax's sum of
// up to 512 terms 16 a lane, and the sum with b. With room of as much again.
__device__ __forceinline__ float key_error(bool sigmoid, float key) {
  return (sigmoid ? 0x1p-20f : 0x1p-17f) + 0x1p-22f * fabsf(key);
}

// The choice with a bias: 32 bits of s + b leave few experts that can be among the k, and those alone are weighed in 64
// bits, one a lane (64 bits of all: 14.7 us instead of 8.8 for 4096 tokens of 384 experts). False where there are more of
// them than lanes. sel: the group's k places; list, key: its LDS.
template <int G, int V>
__device__ __forceinline__ bool choose_by_bias(const float (&z)[V], bool sigmoid, const float* bias, int E, int k, int l,
                                               int32_t* sel, int32_t* count, uint16_t* list, uint64_t* keys,
                                               float* cand_z) {
  float m = 0.0f, sum = 0.0f, a[V];
  if (!sigmoid) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, z[i]);
    m = group_fmax<G>(m);
    if (m == -INFINITY) m = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    a[i] = sigmoid ? sigmoid_f32(z[i]) : exp_down(z[i] - m);
    sum += a[i];
  }
  float inv = 1.0f;
  if (!sigmoid) inv = __builtin_amdgcn_rcpf(group_add<G>(sum));
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * G + l;
    a[i] = fmaf(a[i], inv, e < E ? bias[e] : 0.0f);
    key[i] = z[i] == -INFINITY ? 0u : max(place(a[i]), 1u);
  }
  // the k-th largest, equal ones together
  uint32_t left[V], kth = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) left[i] = key[i];
  int got = 0;                      // of all the wave's groups the slowest sets the pace
  while (true) {
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) b = max(b, left[i]);
    b = group_max<G>(b);
    if (got < k) kth = b;
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      n += left[i] == b;
      left[i] = left[i] == b ? 0u : left[i];
    }
    got += (int)group_all<G>(n, [](uint32_t p, uint32_t q) { return p + q; });
    if (__all(got >= k || b == 0)) break;
  }
  // kth 0: fewer than k are on, and all of them are chosen; 1: NaN among them, and all are weighed
  const float t = kth <= 1u ? -INFINITY : __uint_as_float((kth >> 31) ? kth & 0x7FFFFFFFu : ~kth);
  const float least = t - 2.0f * key_error(sigmoid, t);
  if (l == 0) *count = 0;
  wave_lds();
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (key[i] != 0 && !(a[i] < least)) {
      const int at = atomicAdd(count, 1);
      if (at < G) {
        list[at] = (uint16_t)(i * G + l);
        cand_z[at] = z[i];
      }
    }
  wave_lds();
  const int n = *count;
  if (!__all(n <= G)) return false;
  double total = 1.0;
  if (!sigmoid) {
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) part += exp((double)z[i] - (double)m);
    total = group_add<G>(part);
  }
  const int e = l < n ? list[l] : 0;
  uint64_t mine = 0;
  if (l < n) {
    const double zz = (double)cand_z[l];
    mine = place((sigmoid ? 1.0 / (1.0 + exp(-zz)) : exp(zz - (double)m) / total) + (double)bias[e]);
    keys[l] = mine;
  }
  for (int j = l; j < k; j += G) sel[j] = -1;
  wave_lds();
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const uint64_t o = keys[j];
    rank += o > mine || (o == mine && list[j] < e);
  }
  if (l < n && rank < k) sel[rank] = e;
  wave_lds();
  return true;
}

template <int DT, int G, int V, bool BIAS>
__global__ __launch_bounds__(GATE_THREADS) void k_gate(const void* __restrict__ logits, int64_t T, int E, bool sigmoid,
                                                       const float* __restrict__ bias, int k, bool renorm, float scale,
                                                       int32_t* __restrict__ ids, float* __restrict__ w) {
  constexpr int PER = GATE_THREADS / G;
  __shared__ int32_t sel[PER][MAX_TOPK];
  __shared__ uint64_t keys[BIAS ? PER : 1][G];
  __shared__ float cand_z[BIAS ? PER : 1][G];
  __shared__ int32_t count[BIAS ? PER : 1];
  __shared__ uint16_t list[BIAS ? PER : 1][G];
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
    bool chosen = false;
    if constexpr (BIAS)
      chosen = choose_by_bias<G, V>(z, sigmoid, bias, E, k, l, sel[g], &count[g], list[g], keys[g], cand_z[g]);
    if (!chosen) {
      Keys<G, V, BIAS> keys_of;
      keys_of.make(z, sigmoid, bias, E, l);
      for (int j = 0; j < k; ++j) {
        const int e = keys_of.take(l);
        if (l == 0) sel[g][j] = e;
      }
      wave_lds();
    }
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

constexpr int BAL_THREADS = 1024;
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

// Workgroup (split, sequence): the sums of p and the counts over its part of the sequence's
// tokens.
template <int DT, int G, int V>
__global__ __launch_bounds__(BAL_THREADS) void k_balance(const void* __restrict__ logits, int64_t T, int E, bool sigmoid,
                                                         const int32_t* __restrict__ ids, int k,
                                                         const int32_t* __restrict__ seq_off, float coef,
                                                         float* __restrict__ part_p, int32_t* __restrict__ part_c,
                                                         float* __restrict__ loss, int32_t* __restrict__ counts) {
  constexpr int PER = BAL_THREADS / G;
  __shared__ float sums[BAL_WAVES][G * V];
  __shared__ int32_t hist[512];
  __shared__ float red[16];
  const int64_t q = blockIdx.y;
  int64_t a, b;
  tokens_of(seq_off, q, T, a, b);
  const int64_t per = (b - a + gridDim.x - 1) / gridDim.x;
  const int64_t lo = min(b, a + per * blockIdx.x), hi = min(b, lo + per);
  const int l = threadIdx.x % G, g = threadIdx.x / G;
  const int64_t slots = (hi - lo) * k;
  uint32_t first = E;
  if ((int64_t)threadIdx.x < slots) first = (uint32_t)ids[lo * k + threadIdx.x];
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  if (threadIdx.x < 512) hist[threadIdx.x] = 0;
  __syncthreads();
  for (int64_t t0 = lo; t0 < hi; t0 += PER) {
    float z[V], p[V], top, total;
    load_logits<DT, G, V>(at<DT>(logits, min(t0 + g, hi - 1) * E), E, l, z);
    if (t0 == lo) {
      if (first < (uint32_t)E) atomicAdd(&hist[first], 1);
      for (int64_t i = threadIdx.x + BAL_THREADS; i < slots; i += BAL_THREADS) {
        const uint32_t e = (uint32_t)ids[lo * k + i];
        if (e < (uint32_t)E) atomicAdd(&hist[e], 1);
      }
    }
    shares<G, V>(z, sigmoid, p, top, total);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += t0 + g < hi ? p[i] : 0.0f;
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
  const int c = threadIdx.x < 512 ? hist[threadIdx.x] : 0;
  if (part_p == nullptr) {
    balance_out(q, b - a, E, k, coef, c, p, red, loss, counts);
  } else if ((int)threadIdx.x < E) {
    const int64_t at = (q * gridDim.x + blockIdx.x) * E + threadIdx.x;
    part_p[at] = p;
    part_c[at] = c;
  }
}

// The parts of a sequence, in their order: runs of them side by side, then the runs.
__global__ __launch_bounds__(BAL_THREADS) void k_balance_sum(const float* __restrict__ part_p,
                                                             const int32_t* __restrict__ part_c, int splits, int64_t T,
                                                             int E, int k, const int32_t* __restrict__ seq_off, float coef,
                                                             float* __restrict__ loss, int32_t* __restrict__ counts) {
  __shared__ float red[16], sum_p[BAL_THREADS];
  __shared__ int32_t sum_c[BAL_THREADS];
  const int64_t q = blockIdx.x;
  int64_t a, b;
  tokens_of(seq_off, q, T, a, b);
  const int runs = min(BAL_THREADS / E, 8), run = threadIdx.x / E, e = threadIdx.x - run * E;
  float p = 0.0f;
  int c = 0;
  if (run < runs) {
    const int64_t at = q * splits * E + e;
#pragma unroll 16
    for (int i = splits * run / runs; i < splits * (run + 1) / runs; ++i) {
      p += part_p[at + (int64_t)i * E];
      c += part_c[at + (int64_t)i * E];
    }
  }
  sum_p[threadIdx.x] = p;
  sum_c[threadIdx.x] = c;
  __syncthreads();
  if (run == 0) {
    for (int i = 1; i < runs; ++i) {
      p += sum_p[i * E + e];
      c += sum_c[i * E + e];
    }
  }
  balance_out(q, b - a, E, k, coef, c, p, red, loss, counts);
}

// The last of the S + 1 offsets that is at or before t, G of them at a time; -1 where t is before all of them.
template <int G>
__device__ __forceinline__ int64_t sequence_of(const int32_t* seq_off, int64_t S, int64_t t, int l) {
  int64_t lo = 0, n = S + 1;        // the last offset at or before t is one of lo .. lo + n - 1, or none
  while (n > G) {
    const int64_t step = (n + G - 1) / G, at = lo + step * l;
    const uint32_t before = group_all<G>(step * l < n && seq_off[min(at, S)] <= t ? 1u : 0u,
                                         [](uint32_t p, uint32_t q) { return p + q; });
    if (before > 0) {
      const int64_t skip = step * (int64_t)(before - 1);
      lo += skip;
      n = min(step, n - skip);
    } else {
      n = 1;
    }
  }
  const uint32_t here = group_all<G>(l < n && seq_off[min(lo + l, S)] <= t ? 1u : 0u,
                                     [](uint32_t p, uint32_t q) { return p + q; });
  return here == 0 ? -1 : lo + here - 1;
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
    // everything that hangs on nothing else is asked for first
    load_logits<DT, G, V>(row, E, l, z);
    int32_t id[Q];
    float dw[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int64_t j = t * k + min(q * G + l, k - 1);
      id[q] = a.d_w != nullptr ? a.ids[j] : -1;
      dw[q] = a.d_w != nullptr ? a.d_w[j] : 0.0f;
    }
    int64_t lo = 0;
    if (a.counts != nullptr && a.seq_off != nullptr) lo = sequence_of<G>(a.seq_off, a.S, t, l);
    lo = min(lo, a.S - 1);          // (behind the last sequence: it does not reach t)
    shares<G, V>(z, a.sigmoid, p, top, total);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.0f;
    if (a.counts != nullptr) {
      float f = 0.0f;
      if (lo >= 0) {
        int64_t first, last;
        tokens_of(a.seq_off, lo, a.T, first, last);
        const float inv = 1.0f / (float)max(last - first, (int64_t)1);
        if (t >= first && t < last) f = a.coef * ((float)E / (float)k) * a.d_loss[lo] * inv * inv;
      }
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * G + l;
        d[i] = e < E && lo >= 0 ? f * (float)a.counts[lo * E + e] : 0.0f;
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
        if (j < k) sel[g][j] = id[q];
      }
      wave_lds();
      float s[Q], mean = 0.0f;
      slot_scores<DT, G>(row, sel[g], k, E, l, a.sigmoid, a.renorm, top, total, s);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int j = q * G + l;
        if (!(j < k && (unsigned)id[q] < (unsigned)E)) dw[q] = 0.0f;
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
      if (a.sigmoid) d[i] *= sigmoid_f32(-z[i]);
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
  const integral_constant<int, 16> g16;
  const integral_constant<int, 32> g32;
  if (E <= 64) f(g16, integral_constant<int, 4>());
  else if (E <= 128) f(g16, integral_constant<int, 8>());
  else if (E <= 192) f(g32, integral_constant<int, 6>());
  else if (E <= 256) f(g32, integral_constant<int, 8>());
  else if (E <= 320) f(g32, integral_constant<int, 10>());
  else if (E <= 384) f(g32, integral_constant<int, 12>());
  else f(g32, integral_constant<int, 16>());
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
  // parts of a sequence: of 32 tokens or more on average, at most 80, about 512 workgroups in all
  return (int)std::max<int64_t>(1, std::min({(int64_t)80, T / S / 32, (512 + S - 1) / S}));
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
