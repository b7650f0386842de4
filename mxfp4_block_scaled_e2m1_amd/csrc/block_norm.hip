// The norms before and after a block, fused with the block's gate and the
// residual scale. With rms(v) = sqrt(mean(v^2) + eps) over a row of H elements:
//   u  = y / rms(y) * w_post            (u = y without w_post)
//   r' = residual + s * gate * u        (gate 1, per channel, per token or full)
//   n  = r' / rms(r') * w_pre           (the next block's input)
// and without y only n of the residual itself (the first norm of a stack).
// n is formed from the fp32 r', not from its rounding to the stored type.
//
// Backward, at the stored r' (rh = r' / rms(r'), yh = y / rms(y)):
//   dr  = dr'_out + (dn w_pre - rh mean(dn w_pre rh)) / rms(r')   = d residual
//   du  = s gate dr;  dgate = s dr u, summed over what a gate value covers
//   dy  = (du w_post - yh mean(du w_post yh)) / rms(y)            (du without w_post)
//   dw_pre = sum_t dn rh;  dw_post = sum_t du yh
// The row statistics are formed again from the rows, which are read anyway.
//
// Both passes do a few operations per element: HBM bandwidth bounds them (each
// input row read once, each output row written once), and the row of a
// workgroup stays in registers between its sums. All sums are fp32.
#include <algorithm>
#include <type_traits>

#include "rows.h"

namespace mx {

namespace {

// Element c of the row held by thread tid, piece v: (v * threads + tid) * N.
template <int DT, int RDT, int N, int V>
__global__ __launch_bounds__(1024) void k_block_norm(BlockNormArgs a) {
  __shared__ float red[2 * 16];
  const int threads = blockDim.x, waves = threads >> 6, tid = threadIdx.x;
  const int H = a.H;
  const float inv_h = 1.0f / (float)H;
  Raw<DT, N> wpost[V], wpre[V], gch[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * threads + tid) * N;
    wpost[v].zero(); wpre[v].zero(); gch[v].zero();
    if (c < H) {
      if (a.w_post) wpost[v].load(a.w_post, c);
      if (a.w_pre) wpre[v].load(a.w_pre, c);
      if (a.gate_kind == GATE_CHANNEL) gch[v].load(a.gate, c);
    }
  }
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t base = t * H;
    Raw<DT, N> yr[V], gr[V];
    Raw<RDT, N> rr[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * threads + tid) * N;
      yr[v].zero(); rr[v].zero(); gr[v].zero();
      if (c < H) {
        if (a.y) yr[v].load(a.y, base + c);
        rr[v].load(a.residual, base + c);
        if (a.gate_kind == GATE_FULL) gr[v].load(a.gate, base + c);
      }
    }
    float r[V][N];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < N; ++i) r[v][i] = rr[v].get(i);
    if (a.y) {
      float f = a.res_scale;
      if (a.gate_kind == GATE_TOKEN) {
        Raw<DT, 1> g;
        g.load(a.gate, t);
        f *= g.get(0);
      }
      if (a.w_post) {
        float ss[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < N; ++i) ss[0] = fmaf(yr[v].get(i), yr[v].get(i), ss[0]);
        group_sum<1>(ss, red, waves);
        f *= rsqrtf(ss[0] * inv_h + a.eps);
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float u = yr[v].get(i) * f;
          if (a.w_post) u *= wpost[v].get(i);
          if (a.gate_kind == GATE_CHANNEL) u *= gch[v].get(i);
          if (a.gate_kind == GATE_FULL) u *= gr[v].get(i);
          r[v][i] += u;
        }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * threads + tid) * N;
        if (c < H) {
          Raw<RDT, N> o;
          o.set(r[v]);
          o.store(a.residual_out, base + c);
        }
      }
    }
    if (a.w_pre) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) ss[0] = fmaf(r[v][i], r[v][i], ss[0]);
      group_sum<1>(ss, red + 16, waves);
      const float f = rsqrtf(ss[0] * inv_h + a.eps);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * threads + tid) * N;
        if (c < H) {
          float n[N];
#pragma unroll
          for (int i = 0; i < N; ++i) n[i] = r[v][i] * f * wpre[v].get(i);
          Raw<DT, N> o;
          o.set(n);
          o.store(a.normed, base + c);
        }
      }
    }
    // the two sums of a row use the two halves of red, and a barrier of one
    // keeps the other's next use apart; with a single sum per row it takes one
    if (!(a.y && a.w_post && a.w_pre)) __syncthreads();
  }
}

// A workgroup strides over rows and keeps the column sums of its rows in
// registers: part [grid][2][H] fp32 (w_pre's, then the shared sum of w_post and
// a channel gate, see k_block_norm_cols).
template <int DT, int RDT, int N, int V>
__global__ __launch_bounds__(1024) void k_block_norm_grad(BlockNormGradArgs a) {
  __shared__ float red[4 * 16];
  const int threads = blockDim.x, waves = threads >> 6, tid = threadIdx.x;
  const int H = a.H;
  const float inv_h = 1.0f / (float)H;
  Raw<DT, N> wpost[V], wpre[V], gch[V];
  float cpre[V][N], cpost[V][N];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * threads + tid) * N;
    wpost[v].zero(); wpre[v].zero(); gch[v].zero();
    if (c < H) {
      if (a.w_post) wpost[v].load(a.w_post, c);
      if (a.w_pre) wpre[v].load(a.w_pre, c);
      if (a.gate_kind == GATE_CHANNEL) gch[v].load(a.gate, c);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) cpre[v][i] = cpost[v][i] = 0.0f;
  }
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t base = t * H;
    Raw<DT, N> yr[V], dn[V], gr[V];
    Raw<RDT, N> rr[V], dro[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * threads + tid) * N;
      yr[v].zero(); dn[v].zero(); gr[v].zero(); rr[v].zero(); dro[v].zero();
      if (c < H) {
        if (a.w_pre) {
          rr[v].load(a.residual_out, base + c);
          dn[v].load(a.d_normed, base + c);
        }
        if (a.y) yr[v].load(a.y, base + c);
        if (a.d_residual_out) dro[v].load(a.d_residual_out, base + c);
        if (a.gate_kind == GATE_FULL) gr[v].load(a.gate, base + c);
      }
    }
    // sums of r'^2, dn w_pre r' and y^2
    float s1[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x = rr[v].get(i), y = yr[v].get(i);
        s1[0] = fmaf(x, x, s1[0]);
        s1[1] = fmaf(dn[v].get(i) * wpre[v].get(i), x, s1[1]);
        s1[2] = fmaf(y, y, s1[2]);
      }
    group_sum<3>(s1, red, waves);
    const float fr = rsqrtf(s1[0] * inv_h + a.eps);
    const float mr = s1[1] * fr * inv_h * fr;      // mean(dn w_pre rh) / rms(r')
    const float fy = a.w_post ? rsqrtf(s1[2] * inv_h + a.eps) : 1.0f;
    float dr[V][N];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * threads + tid) * N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        dr[v][i] = dro[v].get(i);
        if (a.w_pre) {
          const float rh = rr[v].get(i) * fr, d = dn[v].get(i);
          cpre[v][i] = fmaf(d, rh, cpre[v][i]);
          dr[v][i] += d * wpre[v].get(i) * fr - rh * mr;
        }
      }
      if (c < H) {
        Raw<RDT, N> o;
        o.set(dr[v]);
        o.store(a.d_residual, base + c);
      }
    }
    if (a.y) {
      float gt = a.res_scale;
      if (a.gate_kind == GATE_TOKEN) {
        Raw<DT, 1> g;
        g.load(a.gate, t);
        gt *= g.get(0);
      }
      // the sum of dr u (times gate values inside the row): dgate of a token
      // gate, and the mean that dy needs
      float s2[1] = {0.0f};
      if (a.w_post || a.gate_kind == GATE_TOKEN) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            float d = dr[v][i] * yr[v].get(i);
            if (a.w_post) d *= wpost[v].get(i);
            if (a.gate_kind == GATE_CHANNEL) d *= gch[v].get(i);
            if (a.gate_kind == GATE_FULL) d *= gr[v].get(i);
            s2[0] += d;
          }
        group_sum<1>(s2, red + 48, waves);
        s2[0] *= fy;
      }
      if (a.gate_kind == GATE_TOKEN && tid == 0) ((float*)a.dgate)[t] = a.res_scale * s2[0];
      const float my = gt * s2[0] * inv_h;         // mean(du w_post yh)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * threads + tid) * N;
        float dy[N], dg[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float yh = yr[v].get(i) * fy;
          const float w = a.w_post ? wpost[v].get(i) : 1.0f;
          float g = gt;
          if (a.gate_kind == GATE_CHANNEL) g *= gch[v].get(i);
          if (a.gate_kind == GATE_FULL) g *= gr[v].get(i);
          // columns: du yh; a channel gate's value is left to the last step,
          // since its own gradient is the same sum times w_post
          cpost[v][i] = fmaf(dr[v][i] * (a.gate_kind == GATE_CHANNEL ? gt : g), yh, cpost[v][i]);
          const float d = g * dr[v][i] * w;
          dy[i] = a.w_post ? fy * (d - yh * my) : d;
          dg[i] = a.res_scale * dr[v][i] * yh * w;
        }
        if (c < H) {
          Raw<DT, N> o;
          o.set(dy);
          o.store(a.dy, base + c);
          if (a.gate_kind == GATE_FULL) {
            o.set(dg);
            o.store(a.dgate, base + c);
          }
        }
      }
    }
    __syncthreads();   // red is free again
  }
  float* part = a.part + (int64_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * threads + tid) * N;
    if (c < H) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (a.w_pre) part[c + i] = cpre[v][i];
        if (a.y) part[H + c + i] = cpost[v][i];
      }
    }
  }
}

// Column sums over the workgroups' partial sums, in workgroup order: 64 columns
// by 16 runs of parts per workgroup, then the runs in order.
template <int DT>
__global__ __launch_bounds__(1024) void k_block_norm_cols(BlockNormGradArgs a, int parts) {
  __shared__ float sh[2][16][64];
  const int lane = threadIdx.x & 63, run = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const int lo = parts * run / 16, hi = parts * (run + 1) / 16;
  const bool pre = a.dw_pre != nullptr, channel = a.gate_kind == GATE_CHANNEL, post = a.dw_post != nullptr || channel;
  float s[2] = {0.0f, 0.0f};
  if (c < a.H) {
    for (int p = lo; p < hi; ++p) {
      const float* q = a.part + (int64_t)p * 2 * a.H + c;
      if (pre) s[0] += q[0];
      if (post) s[1] += q[a.H];
    }
  }
  sh[0][run][lane] = s[0];
  sh[1][run][lane] = s[1];
  __syncthreads();
  if (run != 0 || c >= a.H) return;
  for (int r = 1; r < 16; ++r) {
    s[0] += sh[0][r][lane];
    s[1] += sh[1][r][lane];
  }
  if (pre) a.dw_pre[c] = s[0];
  if (channel) {
    Raw<DT, 1> g, w;
    g.load(a.gate, c);
    if (a.w_post) w.load(a.w_post, c);
    const bool rows = parts > 0;          // an empty sum is 0 whatever the factor
    ((float*)a.dgate)[c] = a.w_post && rows ? s[1] * w.get(0) : s[1];
    if (rows) s[1] *= g.get(0);
  }
  if (a.dw_post) a.dw_post[c] = s[1];
}

// Pieces of N elements per thread (V) and waves of a row.
struct RowShape {
  int V, waves;
};
RowShape row_shape(int H, int N, int most_waves) {
  const int pieces = (H + N - 1) / N;
  const int V = (pieces + 64 * most_waves - 1) / (64 * most_waves);
  const int v = V <= 1 ? 1 : V <= 2 ? 2 : V <= 4 ? 4 : V <= 8 ? 8 : 16;
  return {v, (pieces + 64 * v - 1) / (64 * v)};
}

template <class F>
void dispatch_v(int V, F&& f) {
  if (V == 1) f(std::integral_constant<int, 1>());
  else if (V == 2) f(std::integral_constant<int, 2>());
  else if (V == 4) f(std::integral_constant<int, 4>());
  else if (V == 8) f(std::integral_constant<int, 8>());
  else f(std::integral_constant<int, 16>());
}

// (activation type, residual type): the same, or an fp32 residual
template <class F>
void dispatch_pair(DType dt, DType rdt, F&& f) {
  dispatch_dt(dt, [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (rdt == DT_F32) f(d, DtC<DT_F32>());
    else if constexpr (D != DT_F32) f(d, d);
  });
}

}  // namespace

// Eight elements per piece where every row starts on 16 bytes.
bool block_norm_vec(int H, uintptr_t all_pointers) { return H % 8 == 0 && all_pointers % 16 == 0; }

int block_norm_grad_grid(int64_t T, int H) {
  const RowShape s = row_shape(H, 8, 16);
  return (int)std::min<int64_t>(T, (int64_t)cu_count() * std::max(1, 16 / s.waves));
}

hipError_t launch_block_norm(const BlockNormArgs& a, bool vec, hipStream_t s) {
  const int N = vec ? 8 : 1;
  const RowShape sh = row_shape(a.H, N, vec ? 8 : 16);
  const int grid = (int)std::min<int64_t>(a.T, (int64_t)cu_count() * std::max(1, 32 / sh.waves));
  dispatch_pair(a.dt, a.rdt, [&](auto d, auto r) {
    constexpr int D = decltype(d)::value, R = decltype(r)::value;
    if (vec) {
      if (sh.V == 1) k_block_norm<D, R, 8, 1><<<grid, 64 * sh.waves, 0, s>>>(a);
      else if (sh.V == 2) k_block_norm<D, R, 8, 2><<<grid, 64 * sh.waves, 0, s>>>(a);
      else k_block_norm<D, R, 8, 4><<<grid, 64 * sh.waves, 0, s>>>(a);
    } else {
      dispatch_v(sh.V, [&](auto v) {
        k_block_norm<D, R, 1, decltype(v)::value><<<grid, 64 * sh.waves, 0, s>>>(a);
      });
    }
  });
  return hipGetLastError();
}

hipError_t launch_block_norm_grad(const BlockNormGradArgs& a, bool vec, hipStream_t s) {
  const int N = vec ? 8 : 1;
  const RowShape sh = row_shape(a.H, N, 16);
  const int grid = block_norm_grad_grid(a.T, a.H);
  dispatch_pair(a.dt, a.rdt, [&](auto d, auto r) {
    constexpr int D = decltype(d)::value, R = decltype(r)::value;
    if (grid == 0) {
      // no rows: the column sums are zeros
    } else if (vec) {
      if (sh.V == 1) k_block_norm_grad<D, R, 8, 1><<<grid, 64 * sh.waves, 0, s>>>(a);
      else k_block_norm_grad<D, R, 8, 2><<<grid, 64 * sh.waves, 0, s>>>(a);
    } else {
      dispatch_v(sh.V, [&](auto v) {
        k_block_norm_grad<D, R, 1, decltype(v)::value><<<grid, 64 * sh.waves, 0, s>>>(a);
      });
    }
    if (a.dw_pre || a.dw_post || a.gate_kind == GATE_CHANNEL)
      k_block_norm_cols<D><<<(a.H + 63) / 64, 1024, 0, s>>>(a, grid);
  });
  return hipGetLastError();
}

}  // namespace mx
