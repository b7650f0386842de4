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

// The rows of a group: the workgroup's groups take rows side by side and stride
// over them by the grid. Every group makes the same number of turns, so that all
// meet at the barriers; one past the last row works on zeros and stores nothing.
// PF: two row buffers, the next row fetched before the turn on this one.
template <bool PF, class Row, class Fetch, class Turn>
__device__ __forceinline__ void walk_rows(int64_t T, int groups, int group, Fetch&& fetch, Turn&& turn) {
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t t0 = (int64_t)blockIdx.x * groups;
  Row f0;
  fetch(f0, t0 + group);
  if constexpr (PF) {
    Row f1;
    while (true) {
      fetch(f1, t0 + step + group);
      turn(f0, t0 + group);
      t0 += step;
      if (t0 >= T) break;
      fetch(f0, t0 + step + group);
      turn(f1, t0 + group);
      t0 += step;
      if (t0 >= T) break;
    }
  } else {
    while (true) {
      turn(f0, t0 + group);
      t0 += step;
      if (t0 >= T) break;
      fetch(f0, t0 + group);
    }
  }
}

// A group of `gw` waves holds a row, element c in thread tid, piece v:
// (v * threads + tid) * N. A workgroup holds blockDim / (64 gw) such groups, which
// take rows side by side, and strides over the rows. GATE: the gate kind. PF: the
// next row's pieces are loaded before this row's sums are waited for: with
// one or two workgroups on a CU the sums would otherwise leave HBM idle, and many
// are slower (the streams they make spread over HBM).
template <int DT, int RDT, int N, int V, int GATE, bool PF, bool AL>
__global__ __launch_bounds__(1024) void k_block_norm(BlockNormArgs a, int gw) {
  __shared__ float red_all[16 * 2 * 16];                 // per group 2 * 16
  const int threads = gw * 64, groups = blockDim.x / threads, lane = threadIdx.x & 63;
  const int group = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) / gw), tid = threadIdx.x - group * threads;
  const int wave = tid >> 6;
  float* red = red_all + group * 32;
  const int H = a.H;
  const float inv_h = 1.0f / (float)H;
  const bool has_y = a.y != nullptr, has_post = a.w_post != nullptr, has_pre = a.w_pre != nullptr;
  Raw<DT, N> wpost[V], wpre[V], gch[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * threads + tid) * N;
    wpost[v].zero(); wpre[v].zero(); gch[v].zero();
    if (c < H) {
      if (has_post) wpost[v].template load_row<false, AL>(a.w_post, c, H);
      else wpost[v].fill(1.0f);
      if (has_pre) wpre[v].template load_row<false, AL>(a.w_pre, c, H);
      if (GATE == GATE_CHANNEL) gch[v].template load_row<false, AL>(a.gate, c, H);
      wpost[v].template settle<AL>(c, H);
      wpre[v].template settle<AL>(c, H);
      gch[v].template settle<AL>(c, H);
    }
  }
  struct Row {
    Raw<DT, N> y[V], g[V];
    Raw<RDT, N> res[V];
    Raw<DT, 1> gt;      // of a token gate
    __device__ __forceinline__ void settle(int v, int c, int H) {
      y[v].template settle<AL>(c, H);
      if (GATE == GATE_FULL) g[v].template settle<AL>(c, H);
      res[v].template settle<AL>(c, H);
    }
  };
  auto fetch = [&](Row& f, int64_t t) {
    const int64_t base = t * H;
    f.gt.zero();
    if (GATE == GATE_TOKEN && t < a.T) f.gt.load(at<DT>(a.gate, t), 0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * threads + tid) * N;
      f.y[v].zero(); f.res[v].zero(); f.g[v].zero();
      if (c < H && t < a.T) {
        if (has_y) f.y[v].template load_row<true, AL>(at<DT>(a.y, base), c, H);
        f.res[v].template load_row<true, AL>(at<RDT>(a.residual, base), c, H);
        if (GATE == GATE_FULL) f.g[v].template load_row<true, AL>(at<DT>(a.gate, base), c, H);
      }
    }
  };
  auto turn = [&](Row& f, int64_t t) {
    const bool live = t < a.T;
    const int64_t base = t * H;
    if (!AL) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * threads + tid) * N;
        if (c < H) f.settle(v, c, H);
      }
    }
    if (dt_size<DT> == 2) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        wpre[v].pin(); wpost[v].pin();
        if (GATE == GATE_CHANNEL) gch[v].pin();
      }
    }
    float s = a.res_scale;
    if (GATE == GATE_TOKEN) s *= f.gt.get(0);
    if (has_post) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) ss[0] = fmaf(f.y[v].get(i), f.y[v].get(i), ss[0]);
      group_sum<1>(ss, red, gw, lane, wave);
      s *= rsqrtf(ss[0] * inv_h + a.eps);
    }
    float r[V][N], ss[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * threads + tid) * N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        r[v][i] = f.res[v].get(i);
        if (has_y) {
          float u = f.y[v].get(i) * s * wpost[v].get(i);
          if (GATE == GATE_CHANNEL) u *= gch[v].get(i);
          if (GATE == GATE_FULL) u *= f.g[v].get(i);
          r[v][i] += u;
        }
        ss[0] = fmaf(r[v][i], r[v][i], ss[0]);
      }
      if (has_y && live && c < H) {
        Raw<RDT, N> o;
        o.set(r[v]);
        o.template store_row<false, AL>(at<RDT>(a.residual_out, base), c, H);
      }
    }
    if (has_pre) {
      group_sum<1>(ss, red + 16, gw, lane, wave);
      const float fn = rsqrtf(ss[0] * inv_h + a.eps);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * threads + tid) * N;
        if (live && c < H) {
          float n[N];
#pragma unroll
          for (int i = 0; i < N; ++i) n[i] = r[v][i] * fn * wpre[v].get(i);
          Raw<DT, N> o;
          o.set(n);
          o.template store_row<false, AL>(at<DT>(a.normed, base), c, H);
        }
      }
    }
    // the two sums of a row use the two halves of red, and a barrier of one
    // keeps the other's next use apart; with a single sum per row it takes one
    if (!(has_post && has_pre)) __syncthreads();
  };
  walk_rows<PF, Row>(a.T, groups, group, fetch, turn);
}

// The rows of a group of `gw` waves, one at a time; a workgroup holds `groups`
// such groups, which take rows side by side, and strides over the rows. Each
// thread keeps the column sums of its columns in registers; at the end the
// groups' sums are joined in LDS and the workgroup writes part [2][H] fp32
// (w_pre's, then the shared sum of w_post and a channel gate, see
// k_block_norm_cols). GATE: the gate kind. PF: the next row's pieces are loaded
// before this row's sums are waited for, since one workgroup fills a CU and its
// two row sums would otherwise leave HBM idle.
template <int DT, int RDT, int N, int V, int GATE, bool PF, bool AL>
__global__ __launch_bounds__(1024) void k_block_norm_grad(BlockNormGradArgs a, int gw) {
  __shared__ float red_all[16 * 4 * 16];                 // per group 4 * 16
  extern __shared__ float cols[];                        // [groups][H], when groups > 1
  const int threads = gw * 64, groups = blockDim.x / threads;
  const int group = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) / gw), tid = threadIdx.x - group * threads;
  float* red = red_all + group * 64;
  const int H = a.H;
  const float inv_h = 1.0f / (float)H;
  const bool has_post = a.w_post != nullptr, has_pre = a.w_pre != nullptr, has_y = a.y != nullptr,
             has_dro = a.d_residual_out != nullptr;
  Raw<DT, N> wpost[V], wpre[V], gch[V];
  float cpre[V][N], cpost[V][N];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * threads + tid) * N;
    wpost[v].zero(); wpre[v].zero(); gch[v].zero();
    if (c < H) {
      if (has_post) wpost[v].template load_row<false, AL>(a.w_post, c, H);
      else wpost[v].fill(1.0f);
      if (has_pre) wpre[v].template load_row<false, AL>(a.w_pre, c, H);
      if (GATE == GATE_CHANNEL) gch[v].template load_row<false, AL>(a.gate, c, H);
      wpost[v].template settle<AL>(c, H);
      wpre[v].template settle<AL>(c, H);
      gch[v].template settle<AL>(c, H);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) cpre[v][i] = cpost[v][i] = 0.0f;
  }
  struct Row {
    Raw<DT, N> y[V], dn[V], g[V];
    Raw<RDT, N> r[V], dro[V];
    Raw<DT, 1> gt;      // of a token gate; with the rest, for a load in between would wait for the next row's
    __device__ __forceinline__ void settle(int v, int c, int H) {
      y[v].template settle<AL>(c, H);
      dn[v].template settle<AL>(c, H);
      if (GATE == GATE_FULL) g[v].template settle<AL>(c, H);
      r[v].template settle<AL>(c, H);
      dro[v].template settle<AL>(c, H);
    }
  };
  auto fetch = [&](Row& f, int64_t t) {
    const int64_t base = t * H;
    f.gt.zero();
    if (GATE == GATE_TOKEN && t < a.T) f.gt.load(at<DT>(a.gate, t), 0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * threads + tid) * N;
      f.y[v].zero(); f.dn[v].zero(); f.g[v].zero(); f.r[v].zero(); f.dro[v].zero();
      if (c < H && t < a.T) {
        if (has_pre) {
          f.r[v].template load_row<true, AL>(at<RDT>(a.residual_out, base), c, H);
          f.dn[v].template load_row<true, AL>(at<DT>(a.d_normed, base), c, H);
        }
        if (has_y) f.y[v].template load_row<true, AL>(at<DT>(a.y, base), c, H);
        if (has_dro) f.dro[v].template load_row<true, AL>(at<RDT>(a.d_residual_out, base), c, H);
        if (GATE == GATE_FULL) f.g[v].template load_row<true, AL>(at<DT>(a.gate, base), c, H);
      }
    }
  };
  auto turn = [&](Row& f, int64_t t) {
    const bool live = t < a.T;
    const int64_t base = t * H;
    if (!AL) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * threads + tid) * N;
        if (c < H) f.settle(v, c, H);
      }
    }
    if (dt_size<DT> == 2) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        wpre[v].pin(); wpost[v].pin();
        if (GATE == GATE_CHANNEL) gch[v].pin();
      }
    }
    // sums of r'^2, dn w_pre r' and y^2
    float s1[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x = f.r[v].get(i), y = f.y[v].get(i);
        s1[0] = fmaf(x, x, s1[0]);
        s1[1] = fmaf(f.dn[v].get(i) * wpre[v].get(i), x, s1[1]);
        s1[2] = fmaf(y, y, s1[2]);
      }
    float gt = a.res_scale;
    if (GATE == GATE_TOKEN) gt *= f.gt.get(0);
    group_sum<3>(s1, red, gw, threadIdx.x & 63, tid >> 6);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (dt_size<DT> == 2) { f.y[v].pin(); f.dn[v].pin(); f.g[v].pin(); }
      if (dt_size<RDT> == 2) { f.r[v].pin(); f.dro[v].pin(); }
    }
    // what a call leaves out drops out of the formulas: without w_pre fr = 0,
    // without w_post fy = 1, my = 0 (and the weights loaded as ones); a row
    // past the last has 0 for both
    const float fr = has_pre && live ? rsqrtf(s1[0] * inv_h + a.eps) : 0.0f;
    const float mr = s1[1] * fr * inv_h * fr;      // mean(dn w_pre rh) / rms(r')
    const float fy = !live ? 0.0f : has_post ? rsqrtf(s1[2] * inv_h + a.eps) : 1.0f;
    float dr[V][N];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * threads + tid) * N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float rh = f.r[v].get(i) * fr, d = f.dn[v].get(i);
        cpre[v][i] = fmaf(d, rh, cpre[v][i]);
        dr[v][i] = fmaf(-rh, mr, fmaf(d * wpre[v].get(i), fr, f.dro[v].get(i)));
      }
      if (c < H && live) {
        Raw<RDT, N> o;
        o.set(dr[v]);
        o.template store_row<false, AL>(at<RDT>(a.d_residual, base), c, H);
      }
    }
    if (has_y) {
      // e = dr * gate values inside the row * w_post; the sum of e y is dgate of
      // a token gate and the mean that dy needs
      float s2[1] = {0.0f}, e[V][N];
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float g = dr[v][i];
          if (GATE == GATE_FULL) g *= f.g[v].get(i);
          // columns: du yh; a channel gate's value is left to the last step,
          // since its own gradient is the same sum times w_post
          cpost[v][i] = fmaf(gt * g, f.y[v].get(i) * fy, cpost[v][i]);
          if (GATE == GATE_CHANNEL) g *= gch[v].get(i);
          e[v][i] = g * wpost[v].get(i);
          s2[0] = fmaf(e[v][i], f.y[v].get(i), s2[0]);
        }
      if (has_post || GATE == GATE_TOKEN) group_sum<1>(s2, red + 48, gw, threadIdx.x & 63, tid >> 6);
      s2[0] *= fy;
      if (GATE == GATE_TOKEN && tid == 0 && live) ((float*)a.dgate)[t] = a.res_scale * s2[0];
      const float gf = gt * fy, my = has_post ? gf * s2[0] * inv_h * fy : 0.0f;   // mean(du w_post yh) / rms(y)^2
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * threads + tid) * N;
        float dy[N];
#pragma unroll
        for (int i = 0; i < N; ++i) dy[i] = fmaf(gf, e[v][i], -f.y[v].get(i) * my);
        if (c < H && live) {
          Raw<DT, N> o;
          o.set(dy);
          o.template store_row<false, AL>(at<DT>(a.dy, base), c, H);
          if (GATE == GATE_FULL) {
            float dg[N];
#pragma unroll
            for (int i = 0; i < N; ++i) dg[i] = a.res_scale * dr[v][i] * (f.y[v].get(i) * fy) * wpost[v].get(i);
            o.set(dg);
            o.template store_row<false, AL>(at<DT>(a.dgate, base), c, H);
          }
        }
      }
    }
    // red's two areas are used in turn: with both sums in a row their barriers
    // already keep this row's reads and the next row's writes apart
    if (!(has_y && (has_post || GATE == GATE_TOKEN))) __syncthreads();
  };
  walk_rows<PF, Row>(a.T, groups, group, fetch, turn);
  float* part = a.part + (int64_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (!(which == 0 ? has_pre : has_y)) continue;
    if (groups > 1) __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * threads + tid) * N;
      if (c < H) {
        Raw<DT_F32, N> o;
        o.set(which == 0 ? cpre[v] : cpost[v]);
        if (groups > 1) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (AL || c + i < H) cols[group * H + c + i] = o.get(i);
        } else {
          o.template store_row<false, AL>(part + which * H, c, H);
        }
      }
    }
    if (groups > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < H; c += blockDim.x) {
        float sum = cols[c];
        for (int g = 1; g < groups; ++g) sum += cols[g * H + c];
        part[which * H + c] = sum;
      }
    }
  }
}

// Column sums over the workgroups' partial sums, in workgroup order: 64 columns
// by 16 runs of parts per workgroup, then the runs in order. blockIdx.y: 0 the
// w_pre sums, 1 the shared sums of w_post and a channel gate.
template <int DT>
__global__ __launch_bounds__(1024) void k_block_norm_cols(BlockNormGradArgs a, int parts) {
  constexpr int B = 8;
  __shared__ float sh[16][64];
  const int lane = threadIdx.x & 63, run = threadIdx.x >> 6, which = blockIdx.y;
  const int c = blockIdx.x * 64 + lane;
  const bool channel = a.gate_kind == GATE_CHANNEL;
  if (!(which == 0 ? a.dw_pre != nullptr : a.dw_post != nullptr || channel)) return;
  const int lo = parts * run / 16, hi = parts * (run + 1) / 16;
  float s = 0.0f;
  if (c < a.H) {
    const float* q = a.part + which * a.H + c;
    int p = lo;
    for (; p + B <= hi; p += B) {      // B loads in flight
      float v[B];
#pragma unroll
      for (int i = 0; i < B; ++i) v[i] = q[(int64_t)(p + i) * 2 * a.H];
#pragma unroll
      for (int i = 0; i < B; ++i) s += v[i];
    }
    for (; p < hi; ++p) s += q[(int64_t)p * 2 * a.H];
  }
  sh[run][lane] = s;
  __syncthreads();
  if (run != 0 || c >= a.H) return;
#pragma unroll
  for (int r = 1; r < 16; ++r) s += sh[r][lane];
  if (which == 0) {
    a.dw_pre[c] = s;
    return;
  }
  if (channel) {
    Raw<DT, 1> g, w;
    g.load(a.gate, c);
    if (a.w_post) w.load(a.w_post, c);
    const bool rows = parts > 0;          // an empty sum is 0 whatever the factor
    ((float*)a.dgate)[c] = a.w_post && rows ? s * w.get(0) : s;
    if (rows) s *= g.get(0);
  }
  if (a.dw_post) a.dw_post[c] = s;
}

// Pieces of N elements per thread (V) and waves of a row of up to 16384 elements.
struct RowShape {
  int V, waves;
};
RowShape row_shape(int H, int N, int most_waves) {
  const int pieces = (H + N - 1) / N;
  const int V = (pieces + 64 * most_waves - 1) / (64 * most_waves);
  const int v = V <= 1 ? 1 : V <= 2 ? 2 : 4;
  return {v, (pieces + 64 * v - 1) / (64 * v)};
}

template <class F>
void dispatch_gate(GateKind kind, F&& f) {
  if (kind == GATE_NONE) f(std::integral_constant<int, GATE_NONE>());
  else if (kind == GATE_CHANNEL) f(std::integral_constant<int, GATE_CHANNEL>());
  else if (kind == GATE_TOKEN) f(std::integral_constant<int, GATE_TOKEN>());
  else f(std::integral_constant<int, GATE_FULL>());
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

// Elements per piece: 16 bytes of the activations.
static int piece(DType dt) { return dt == DT_F32 ? 4 : 8; }
bool block_norm_aligned(DType dt, int H, uintptr_t all_pointers) { return H % piece(dt) == 0 && all_pointers % 16 == 0; }

// One workgroup of up to 16 waves per CU of an MI355X. The way back keeps it so, at any
// count of rows: one against two, token gate, bf16, us: 300 x 7168 19.6 and 23.0, 1024
// x 4096 22.3 and 26.9, 1537 x 1024 14.4 and 13.9, 2048 x 1024 14.2 and 15.0, 3000 x
// 7168 61.2 and 68.2, 4096 x 7168 77.3 and 84.4; fp32, full gate: 300 x 1000 9.4 and
// 9.8, 1537 x 1000 17.0 and 19.6. So do rows of more than a piece per thread and
// unaligned ones (8192 x 4290 bf16: 63.8 us, two 64.7).
constexpr int ROW_GRID = 256;
// The norm itself takes two, whose rows' sums and stores fall in each other's gaps, as
// long as the rows they spread over HBM do not cost more. One against two, bf16, us:
// 1000 x 7168 14.0 and 12.5, 4096 x 7168 48.5 and 44.9 (fp32 residual 69.3 and 68.3),
// 16384 x 4096 97.7 and 97.0, 16384 x 7168 175 and 182.
int norm_grid(int64_t T, int H, int V, bool aligned) {
  return aligned && V == 1 && T * H <= (int64_t)1 << 26 ? 2 * ROW_GRID : ROW_GRID;
}
// Groups per workgroup: as many as there are rows for in every workgroup.
int row_groups(int64_t T, int waves, int grid) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(16 / waves, (T + grid - 1) / grid));
}

// An upper bound of the workgroups of the way back, each with a partial sum.
int block_norm_grad_grid(int64_t T) { return (int)std::min<int64_t>(T, ROW_GRID); }

// f(elements per piece, pieces per thread, aligned)
template <int D, class F>
void dispatch_shape(int H, int V, bool aligned, F&& f) {
  constexpr int P = D == DT_F32 ? 4 : 8;
  std::integral_constant<int, P> n;
  auto v = [&](auto vc) {
    if (aligned) f(n, vc, std::true_type());
    else f(n, vc, std::false_type());
  };
  if (H < P) f(std::integral_constant<int, 1>(), std::integral_constant<int, 1>(), std::true_type());   // no whole piece
  else if (V == 1) v(std::integral_constant<int, 1>());
  else if (V == 2) v(std::integral_constant<int, 2>());
  else if constexpr (D == DT_F32) v(std::integral_constant<int, 4>());
}

hipError_t launch_block_norm(const BlockNormArgs& a, bool aligned, hipStream_t s) {
  const RowShape sh = row_shape(a.H, piece(a.dt), 16);
  const int most = norm_grid(a.T, a.H, sh.V, aligned), groups = row_groups(a.T, sh.waves, most);
  const int grid = (int)std::min<int64_t>((a.T + groups - 1) / groups, most);
  const int threads = 64 * sh.waves * groups;
  dispatch_pair(a.dt, a.rdt, [&](auto d, auto r) {
    constexpr int D = decltype(d)::value, R = decltype(r)::value;
    dispatch_shape<D>(a.H, sh.V, aligned, [&](auto n, auto v, auto al) {
      dispatch_gate(a.gate_kind, [&](auto g) {
        constexpr int V = decltype(v)::value;
        k_block_norm<D, R, decltype(n)::value, V, decltype(g)::value, V == 1, decltype(al)::value>
            <<<grid, threads, 0, s>>>(a, sh.waves);
      });
    });
  });
  return hipGetLastError();
}

hipError_t launch_block_norm_grad(const BlockNormGradArgs& a, bool aligned, hipStream_t s) {
  const RowShape sh = row_shape(a.H, piece(a.dt), 16);
  const int groups = row_groups(a.T, sh.waves, ROW_GRID);
  const int grid = (int)std::min<int64_t>((a.T + groups - 1) / groups, ROW_GRID);
  const size_t lds = groups > 1 ? (size_t)groups * a.H * 4 : 0;
  const int threads = 64 * sh.waves * groups;
  dispatch_pair(a.dt, a.rdt, [&](auto d, auto r) {
    constexpr int D = decltype(d)::value, R = decltype(r)::value;
    // no rows: the column sums are zeros
    if (grid > 0) dispatch_shape<D>(a.H, sh.V, aligned, [&](auto n, auto v, auto al) {
      dispatch_gate(a.gate_kind, [&](auto g) {
        constexpr int V = decltype(v)::value, G = decltype(g)::value;
        // a full gate beside an fp32 residual, or unaligned rows: the next row would not
        // fit the 128 registers that a thread of a full workgroup has. Rows of more than
        // a piece per thread do not fit by themselves: 4 to 338 registers of those
        // variants (20 and more of unaligned full gates) go to scratch, and they take
        // twice the time of what they move (4096 x 16384 bf16, channel gate: 316 us, 149
        // to move).
        constexpr bool AL = decltype(al)::value;
        constexpr bool PF = V == 1 && AL && !(G == GATE_FULL && D != DT_F32 && R == DT_F32);
        k_block_norm_grad<D, R, decltype(n)::value, V, G, PF, AL>
            <<<grid, threads, lds, s>>>(a, sh.waves);
      });
    });
    if (a.dw_pre || a.dw_post || a.gate_kind == GATE_CHANNEL)
      k_block_norm_cols<D><<<dim3((a.H + 63) / 64, 2), 1024, 0, s>>>(a, grid);
  });
  return hipGetLastError();
}

}  // namespace mx
