// Layer norm over the rows of [T, d], forward (with the residual add before it) and
// backward (with the gradient that comes along the residual stream, and the sums over
// rows of the weight's and bias's gradients).
//
//   s = x + r rounded to the type;  mu = sum s / d;  rstd = (sum (s - mu)^2 / d + eps)^-1/2
//   xh = (s - mu) rstd;  y = xh w + b
//   g = dy w;  c1 = sum g / d;  c2 = sum g xh / d;  dx = rstd (g - c1 - xh c2) + dres
//   dw = sum_t dy xh;  db = sum_t dy
//
// A row is read once and stays in the registers of its team of warps, so the variance
// is the two-sweep one (no cancellation of large means) at no extra traffic. All
// statistics and sums are fp32; y, dx and s are rounded once.
#include <algorithm>

#include "tw_internal.h"
#include "tw_rows.cuh"

namespace tw {

namespace {

// Elements of a row owned by a thread: VPT chunks of 8 (VEC: consecutive elements,
// 16-byte accesses) or 8 VPT single elements (any d, alignment and row stride).
template <int DT, int VPT, bool VEC>
struct RowMap {
  using S = typename Elem<DT>::S;
  static constexpr int NE = 8 * VPT;
  static TW_DEV int col(int i, int tid, int tpr) {
    return VEC ? ((i >> 3) * tpr + tid) * 8 + (i & 7) : i * tpr + tid;
  }
  static TW_DEV void load(const S* p, int d, int tid, int tpr, float (&v)[NE]) {
    if constexpr (VEC) {
      constexpr int E = Elem<DT>::E;
#pragma unroll
      for (int k = 0; k < NE / E; ++k) {
        const int c = col(k * E, tid, tpr);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (c < d) w = *reinterpret_cast<const uint4*>(p + c);
        float u[E];
        Elem<DT>::unpack(w, u);
#pragma unroll
        for (int e = 0; e < E; ++e) v[k * E + e] = u[e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int c = col(i, tid, tpr);
        v[i] = c < d ? Elem<DT>::get(p[c]) : 0.f;
      }
    }
  }
  static TW_DEV void store(S* p, int d, int tid, int tpr, const float (&v)[NE]) {
    if constexpr (VEC) {
      constexpr int E = Elem<DT>::E;
#pragma unroll
      for (int k = 0; k < NE / E; ++k) {
        const int c = col(k * E, tid, tpr);
        float u[E];
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] = v[k * E + e];
        if (c < d) *reinterpret_cast<uint4*>(p + c) = Elem<DT>::pack(u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int c = col(i, tid, tpr);
        if (c < d) p[c] = Elem<DT>::put(v[i]);
      }
    }
  }
};

// The thread's elements of a weight vector of type DT or fp32 (fill where it is null).
template <int DT, int VPT, bool VEC>
TW_DEV void load_weight(const void* w, int wtype, float fill, int d, int tid, int tpr, float (&v)[8 * VPT]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8 * VPT; ++i) v[i] = fill;
  } else if (wtype == DT) {
    RowMap<DT, VPT, VEC>::load(static_cast<const typename Elem<DT>::S*>(w), d, tid, tpr, v);
  } else {
    RowMap<TW_F32, VPT, VEC>::load(static_cast<const float*>(w), d, tid, tpr, v);
  }
}

// Sum over a team's threads, the same bits in each of them. `red` holds 32 floats; a
// caller alternates between two of them, so that one barrier per sum is enough.
TW_DEV float team_sum(float v, float* red, int team, int tpr) {
  v = warp_sum(v);
  if (tpr == 32) return v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) red[warp] = v;
  team_barrier(team + 1, tpr);
  return warp_sum(lane < (tpr >> 5) ? red[lane] : 0.f);
}
TW_DEV float2 team_sum2(float a, float b, float2* red, int team, int tpr) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (tpr == 32) return make_float2(a, b);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) red[warp] = make_float2(a, b);
  team_barrier(team + 1, tpr);
  const float2 p = lane < (tpr >> 5) ? red[lane] : make_float2(0.f, 0.f);
  return make_float2(warp_sum(p.x), warp_sum(p.y));
}

constexpr int kMaxTeams = 15;  // named barriers 1..15

template <int DT, int VPT, bool VEC>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormFwdArgs a) {
  using M = RowMap<DT, VPT, VEC>;
  using S = typename M::S;
  __shared__ float red[2][kMaxTeams][32];
  pdl_enter();
  const int tid = threadIdx.x, tpr = blockDim.x, team = threadIdx.y;
  const int row = blockIdx.x * blockDim.y + team;
  if (row >= a.T) return;
  const size_t r = static_cast<size_t>(row);
  float v[M::NE];
  M::load(static_cast<const S*>(a.x) + r * a.ldx, a.d, tid, tpr, v);
  if (a.res != nullptr) {
    float u[M::NE];
    M::load(static_cast<const S*>(a.res) + r * a.ldres, a.d, tid, tpr, u);
#pragma unroll
    for (int i = 0; i < M::NE; ++i) v[i] = Elem<DT>::get(Elem<DT>::put(v[i] + u[i]));
    if (a.sum != nullptr) M::store(static_cast<S*>(a.sum) + r * a.ldsum, a.d, tid, tpr, v);
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < M::NE; ++i) s += v[i];
  const float inv_d = 1.f / static_cast<float>(a.d);
  const float mean = team_sum(s, red[0][team], team, tpr) * inv_d;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < M::NE; ++i) {
    const float t = M::col(i, tid, tpr) < a.d ? v[i] - mean : 0.f;
    q = fmaf(t, t, q);
  }
  const float rstd = rsqrtf(team_sum(q, red[1][team], team, tpr) * inv_d + a.eps);
  float w[M::NE], b[M::NE];
  load_weight<DT, VPT, VEC>(a.w, a.wtype, 1.f, a.d, tid, tpr, w);
  load_weight<DT, VPT, VEC>(a.b, a.wtype, 0.f, a.d, tid, tpr, b);
#pragma unroll
  for (int i = 0; i < M::NE; ++i) v[i] = fmaf((v[i] - mean) * rstd, w[i], b[i]);
  M::store(static_cast<S*>(a.y) + r * a.ldy, a.d, tid, tpr, v);
  if (tid == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
}

template <int DT, int VPT, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const NormBwdArgs a) {
  using M = RowMap<DT, VPT, VEC>;
  using S = typename M::S;
  extern __shared__ float acc[];  // [2][d], teams joined in order (teams > 1 only)
  __shared__ float2 red[2][kMaxTeams][32];
  pdl_enter();
  const int tid = threadIdx.x, tpr = blockDim.x, team = threadIdx.y;
  float w[M::NE], dw[M::NE], db[M::NE];
  load_weight<DT, VPT, VEC>(a.w, a.wtype, 1.f, a.d, tid, tpr, w);
#pragma unroll
  for (int i = 0; i < M::NE; ++i) dw[i] = db[i] = 0.f;
  const float inv_d = 1.f / static_cast<float>(a.d);
  int flip = 0;
  for (int row = blockIdx.x * blockDim.y + team; row < a.T; row += gridDim.x * blockDim.y, flip ^= 1) {
    const size_t r = static_cast<size_t>(row);
    float x[M::NE], g[M::NE];
    M::load(static_cast<const S*>(a.x) + r * a.ldx, a.d, tid, tpr, x);
    M::load(static_cast<const S*>(a.dy) + r * a.lddy, a.d, tid, tpr, g);
    const float mean = a.mean[row], rstd = a.rstd[row];
    float c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int i = 0; i < M::NE; ++i) {
      x[i] = M::col(i, tid, tpr) < a.d ? (x[i] - mean) * rstd : 0.f;
      dw[i] = fmaf(g[i], x[i], dw[i]);
      db[i] += g[i];
      g[i] *= w[i];
      c1 += g[i];
      c2 = fmaf(g[i], x[i], c2);
    }
    const float2 c = team_sum2(c1, c2, red[flip][team], team, tpr);
    c1 = c.x * inv_d;
    c2 = c.y * inv_d;
#pragma unroll
    for (int i = 0; i < M::NE; ++i) g[i] = rstd * (g[i] - fmaf(x[i], c2, c1));
    if (a.dres != nullptr) {
      M::load(static_cast<const S*>(a.dres) + r * a.lddres, a.d, tid, tpr, x);
#pragma unroll
      for (int i = 0; i < M::NE; ++i) g[i] += x[i];
    }
    M::store(static_cast<S*>(a.dx) + r * a.lddx, a.d, tid, tpr, g);
  }
  if (a.part == nullptr) return;
  float* out = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.d;
  for (int t = 0; t + 1 < static_cast<int>(blockDim.y); ++t) {
    if (team == t) {
#pragma unroll
      for (int i = 0; i < M::NE; ++i) {
        const int c = M::col(i, tid, tpr);
        if (c < a.d) {
          acc[c] = t == 0 ? dw[i] : acc[c] + dw[i];
          acc[a.d + c] = t == 0 ? db[i] : acc[a.d + c] + db[i];
        }
      }
    }
    __syncthreads();
  }
  if (team == static_cast<int>(blockDim.y) - 1) {
#pragma unroll
    for (int i = 0; i < M::NE; ++i) {
      const int c = M::col(i, tid, tpr);
      if (c < a.d) {
        out[c] = team == 0 ? dw[i] : acc[c] + dw[i];
        out[a.d + c] = team == 0 ? db[i] : acc[a.d + c] + db[i];
      }
    }
  }
}

// dw, db = the partial sums of `n` CTAs, added in a fixed order.
__global__ void __launch_bounds__(512) norm_bwd_finish_kernel(const float* part, int n, int d, float* dw, float* db) {
  __shared__ float s[16][33];
  pdl_enter();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < 2 * d)
    for (int i = threadIdx.y; i < n; i += 16) v += part[static_cast<size_t>(i) * 2 * d + c];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || c >= 2 * d) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += s[i][threadIdx.x];
  if (c < d) {
    if (dw != nullptr) dw[c] = v;
  } else if (db != nullptr) {
    db[c - d] = v;
  }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t elem_size(int dtype) { return dtype == TW_F32 ? 4 : 2; }
bool stride16(int64_t ld, int dtype) { return ld * static_cast<int64_t>(elem_size(dtype)) % 16 == 0; }

struct Team {
  int tpr, teams;
};
// Warps for a row of d elements at 8 VPT elements a thread, and rows per CTA of about
// `threads` threads.
Team team_of(int d, int vpt, int threads, int T) {
  Team t;
  t.tpr = ((d + 8 * vpt - 1) / (8 * vpt) + 31) / 32 * 32;
  t.teams = std::max(1, std::min({threads / t.tpr, kMaxTeams, T}));
  return t;
}

template <int DT, int VPT, bool VEC>
cudaError_t norm_fwd(const NormFwdArgs& a, cudaStream_t s) {
  const Team t = team_of(a.d, VPT, 256, a.T);
  cudaError_t e = launch(norm_fwd_kernel<DT, VPT, VEC>, dim3((a.T + t.teams - 1) / t.teams), dim3(t.tpr, t.teams), 0, s, a);
  trace_mark(s, "norm_fwd");
  return e;
}

cudaError_t norm_bwd_finish(const NormBwdArgs& a, int partials, cudaStream_t s) {
  cudaError_t e = launch(norm_bwd_finish_kernel, dim3((2 * a.d + 31) / 32), dim3(32, 16), 0, s,
                         static_cast<const float*>(a.part), partials, a.d, a.dw, a.db);
  trace_mark(s, "norm_bwd_finish");
  return e;
}

template <int DT, int VPT, bool VEC, int MAXT>
cudaError_t norm_bwd(const NormBwdArgs& a, cudaStream_t s) {
  const Team t = team_of(a.d, VPT, MAXT, a.T);
  const int grid = std::min({(a.T + t.teams - 1) / t.teams, device_sm_count(), kNormPartials});
  const size_t smem = t.teams > 1 ? 2 * sizeof(float) * a.d : 0;
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024) {
    e = cudaFuncSetAttribute(norm_bwd_kernel<DT, VPT, VEC, MAXT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  e = launch(norm_bwd_kernel<DT, VPT, VEC, MAXT>, dim3(grid), dim3(t.tpr, t.teams), smem, s, a);
  trace_mark(s, "norm_bwd");
  if (e != cudaSuccess || a.part == nullptr) return e;
  return norm_bwd_finish(a, grid, s);
}

template <int DT, bool VEC>
cudaError_t norm_fwd_width(const NormFwdArgs& a, cudaStream_t s) {
  return a.d <= 1024 ? norm_fwd<DT, 1, VEC>(a, s) : norm_fwd<DT, 2, VEC>(a, s);
}
template <int DT, bool VEC>
cudaError_t norm_bwd_width(const NormBwdArgs& a, cudaStream_t s) {
  if (a.d <= 512) return norm_bwd<DT, 1, VEC, 512>(a, s);
  return a.d <= 8192 ? norm_bwd<DT, 2, VEC, 512>(a, s) : norm_bwd<DT, 2, VEC, 1024>(a, s);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwdArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int dt = a.dtype;
  const bool vec = a.d % 8 == 0 && on16(a.x) && on16(a.res) && on16(a.sum) && on16(a.y) && on16(a.w) && on16(a.b) &&
                   stride16(a.ldx, dt) && stride16(a.ldres, dt) && stride16(a.ldsum, dt) && stride16(a.ldy, dt);
  switch (dt) {
    case TW_F32: return vec ? norm_fwd_width<TW_F32, true>(a, s) : norm_fwd_width<TW_F32, false>(a, s);
    case TW_BF16: return vec ? norm_fwd_width<TW_BF16, true>(a, s) : norm_fwd_width<TW_BF16, false>(a, s);
    default: return vec ? norm_fwd_width<TW_F16, true>(a, s) : norm_fwd_width<TW_F16, false>(a, s);
  }
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t s) {
  if (a.T == 0) return a.dw != nullptr || a.db != nullptr ? norm_bwd_finish(a, 0, s) : cudaSuccess;  // sums over no rows
  const int dt = a.dtype;
  const bool vec = a.d % 8 == 0 && on16(a.x) && on16(a.dy) && on16(a.dres) && on16(a.dx) && on16(a.w) &&
                   stride16(a.ldx, dt) && stride16(a.lddy, dt) && stride16(a.lddres, dt) && stride16(a.lddx, dt);
  switch (dt) {
    case TW_F32: return vec ? norm_bwd_width<TW_F32, true>(a, s) : norm_bwd_width<TW_F32, false>(a, s);
    case TW_BF16: return vec ? norm_bwd_width<TW_BF16, true>(a, s) : norm_bwd_width<TW_BF16, false>(a, s);
    default: return vec ? norm_bwd_width<TW_F16, true>(a, s) : norm_bwd_width<TW_F16, false>(a, s);
  }
}

}  // namespace tw
