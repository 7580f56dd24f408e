// The kernels over rows of [T, d] that layer norm (tw_norm.cu) and root-mean-square norm
// (tw_rms_fwd.cu, tw_rms_fp8.cu, tw_rms_bwd.cu) are made of, and the choice of their form by
// the row's width. What the two norms compute, and what was measured, stands in those files.
#pragma once

#include <algorithm>

#include <cuda_fp8.h>

#include "tw_internal.h"
#include "tw_rows.cuh"

namespace tw {

namespace {

// What a forward kernel computes. The norms differ in the mean, which RMS norm does not
// take; the last two write e4m3 with an fp32 scale a row, or one for each 128 columns.
enum NormKind { LAYER_NORM = 0, RMS_NORM = 1, RMS_FP8_ROW = 2, RMS_FP8_GROUP = 3 };
constexpr int kFp8Group = 128;  // columns of a scale: whole vectors of 16 or 32 lanes
constexpr float kFp8Max = 448.f, kFp8LeastScale = 0x1p-126f;

// the larger; NaN where one of them is
TW_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// over groups of `lanes` lanes, of which those of `mask` are here
TW_DEV float warp_max_nan(float v, int lanes, unsigned mask = 0xFFFFFFFFu) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v = max_nan(v, __shfl_xor_sync(mask, v, o));
  return v;
}
TW_DEV float lanes_sum(float v, int lanes, unsigned mask) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v += __shfl_xor_sync(mask, v, o);
  return v;
}
// A team's lanes of its warp. Short rows' teams are less than a warp, whose teams may leave
// their rows' loop one after the other.
TW_DEV unsigned team_lanes(int tpr) {
  return tpr >= 32 ? 0xFFFFFFFFu : ((1u << (tpr & 31)) - 1u) << (threadIdx.y * tpr & 31);
}
// the scale that the largest magnitude fits with
TW_DEV float fp8_scale(float most) {
  const float s = most * (1.f / kFp8Max);
  return s < kFp8LeastScale ? kFp8LeastScale : s;
}
// 1 / scale (hardware approximation to about 1 ulp; e4m3 has 20 bits fewer)
TW_DEV float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// two values as e4m3, round to nearest even, NaN kept
TW_DEV uint32_t fp8x2(float2 v) { return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3); }

// How rows lie (VEC below). WHOLE: they begin on 16 bytes and hold whole vectors. ANYWHERE:
// anywhere, d is any, and a vector is put together from two (tw_rows.cuh). ALIKE: d is any,
// and a row lies alike in all matrices, `lead` elements behind 16 bytes. Vectors are then the
// aligned ones, whose elements before and behind the row read 0 and are not written; a team's
// rows are 8 (fp32: 4) apart, or a multiple, so that they have one lead, and weights and column
// sums keep their places in the threads. (RMS norm's alone: 65344 rows of 1027 bf16 forward 60
// us, ANYWHERE 79; backward 145 and 186, in fp32 161 and 265.)
enum Rows { ANYWHERE = 0, WHOLE = 1, ALIKE = 2 };

// Elements of a row owned by a thread, 8 VPT of them as packed pairs: vectors of 16 bytes in
// strides of the team, so that a warp's accesses are adjacent. What lies past the row reads 0.
// TPR: the team's threads where they are a constant of the kernel (offsets are then
// immediates), else 0.
template <int DT, int VPT, int VEC, int TPR>
struct RowMap {
  using S = typename Elem<DT>::S;
  static constexpr int NE = 8 * VPT, NP = NE / 2;
  static constexpr int E = Elem<DT>::E, NV = NE / E;  // elements of a vector, vectors
  int d, tid, tpr_, lead;
  bool edge;  // (ALIKE) the warp has a vector that is not whole: the others skip what those need
  TW_DEV RowMap(int d_, int tid_, int tpr, int lead_ = 0) : d(d_), tid(tid_), tpr_(tpr), lead(VEC == ALIKE ? lead_ : 0), edge(false) {
    if constexpr (VEC == ALIKE) {
      bool parts = false;
#pragma unroll
      for (int k = 0; k < NV; ++k) parts = parts || (has(k * E) && !whole(k));
      edge = __any_sync(0xFFFFFFFFu, parts);
    }
  }
  TW_DEV int tpr() const { return TPR > 0 ? TPR : tpr_; }
  TW_DEV int col(int i) const { return (i / E * tpr() + tid) * E + i % E - lead; }
  TW_DEV bool has(int i) const { return col(i / E * E) < d; }  // the element's vector is in the row, at least in part
  TW_DEV bool whole(int k) const { return VEC == WHOLE || (col(k * E) >= 0 && col(k * E) + E <= d); }  // vector k in all

  static TW_DEV void widen16(const uint4& w, float2* v) {
    float2 u[Elem<DT>::E / 2];
    Elem<DT>::pairs(w, u);
#pragma unroll
    for (int e = 0; e < Elem<DT>::E / 2; ++e) v[e] = u[e];
  }
  // careful: see load_any
  TW_DEV void load(const S* p, float2 (&v)[NP], bool careful = true) const {
    uint4 r[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = col(k * E);
      r[k] = make_uint4(0, 0, 0, 0);
      if constexpr (VEC != ANYWHERE) {
        if (c < d) r[k] = *reinterpret_cast<const uint4*>(p + c);
      } else {
        if (c < d) r[k] = load_any<DT>(p + c, d - c, careful);
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) widen16(r[k], v + k * E / 2);
  }
  // by whole warps
  TW_DEV void store(S* p, const float2 (&v)[NP]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 u[E / 2];
#pragma unroll
      for (int e = 0; e < E / 2; ++e) u[e] = v[k * E / 2 + e];
      const int c = col(k * E);
      if constexpr (VEC == ALIKE) {
        union {
          uint4 w;
          S e[E];
        } q;
        q.w = Elem<DT>::pack_pairs(u);
        if (!edge || whole(k)) {
          if (c < d) *reinterpret_cast<uint4*>(p + c) = q.w;
        } else if (c < d) {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (in(k * E + e)) p[c + e] = q.e[e];
        }
      } else if constexpr (VEC != ANYWHERE) {
        if (c < d) *reinterpret_cast<uint4*>(p + c) = Elem<DT>::pack_pairs(u);
      } else {
        store_any<DT>(p + c, Elem<DT>::pack_pairs(u), d - c, tid & 31);
      }
    }
  }
  // as e4m3 bytes; VEC: a vector's bytes at once
  TW_DEV void store_fp8(uint8_t* p, const float2 (&v)[NP]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = col(k * E);
      uint32_t w[E / 4];
#pragma unroll
      for (int e = 0; e < E / 4; ++e) w[e] = fp8x2(v[k * E / 2 + 2 * e]) | fp8x2(v[k * E / 2 + 2 * e + 1]) << 16;
      if (VEC == WHOLE || (VEC == ALIKE && (!edge || whole(k)) && (reinterpret_cast<uintptr_t>(p + c) & (E - 1)) == 0)) {
        if (c >= d) continue;
        if constexpr (E == 8)
          *reinterpret_cast<uint2*>(p + c) = make_uint2(w[0], w[1]);
        else
          *reinterpret_cast<uint32_t*>(p + c) = w[0];
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (in(k * E + e)) p[c + e] = static_cast<uint8_t>(w[e / 4] >> (8 * (e % 4)));
      }
    }
  }
  // a vector of d weights of the row's type or fp32 (fill where it is null)
  TW_DEV void weight(const void* w, int wtype, float fill, float2 (&v)[NP]) const {
    if (w == nullptr) {
#pragma unroll
      for (int i = 0; i < NP; ++i) v[i] = both(fill);
    } else if (VEC != ALIKE && wtype == DT) {
      load(static_cast<const S*>(w), v);
    } else if (wtype == DT) {
      const S* p = static_cast<const S*>(w);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        v[i].x = in(2 * i) ? Elem<DT>::get(p[col(2 * i)]) : 0.f;
        v[i].y = in(2 * i + 1) ? Elem<DT>::get(p[col(2 * i + 1)]) : 0.f;
      }
    } else {
      const float* p = static_cast<const float*>(w);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if constexpr (VEC == WHOLE) {
          v[i] = has(2 * i) ? *reinterpret_cast<const float2*>(p + col(2 * i)) : both(0.f);
        } else {
          v[i].x = in(2 * i) ? p[col(2 * i)] : 0.f;
          v[i].y = in(2 * i + 1) ? p[col(2 * i + 1)] : 0.f;
        }
      }
    }
  }
  // f(pair) for the pairs of vectors in the row, at least in part
  template <class F>
  TW_DEV void each(F f) const {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (has(k * E)) {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) f(k * E / 2 + e);
      }
  }
  TW_DEV bool in(int i) const { return col(i) < d && (VEC != ALIKE || col(i) >= 0); }
  // 0 in the places past the row of a vector that is in it in part
  TW_DEV void trim(float2 (&v)[NP]) const {
    if constexpr (VEC == WHOLE) return;
    if (VEC == ALIKE && !edge) return;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (has(k * E) && (VEC == ALIKE ? !whole(k) : !in(k * E + E - 1))) {
#pragma unroll
        for (int i = k * E / 2; i < (k + 1) * E / 2; ++i)
          v[i] = make_float2(in(2 * i) ? v[i].x : 0.f, in(2 * i + 1) ? v[i].y : 0.f);
      }
  }
};

// The rows around whose ends 16 bytes (E elements) may lie outside the matrix: the first and
// the last, and all where they lie closer together than that (a stride of 0 repeats a row).
TW_DEV bool end_row(int row, int T, int64_t ld, int E) { return row == 0 || row == T - 1 || ld < E; }

constexpr int kMaxTeams = 15;  // named barriers 1..15

template <bool RMS>
TW_DEV float2 centred(float2 x, float mean) {
  if constexpr (RMS)
    return x;
  else
    return add2(x, both(-mean));
}

// Sum over a team's threads, the same bits in each of them. `red` holds 32 values; a
// caller alternates between two of them, so that one barrier per sum is enough.
TW_DEV float team_sum(float v, float* red, int team, int tpr, int tid) {
  if (tpr < 32) return lanes_sum(v, tpr, team_lanes(tpr));
  v = warp_sum(v);
  if (tpr == 32) return v;
  const int lane = tid & 31, warp = tid >> 5, warps = tpr >> 5;
  if (lane == 0) red[warp] = v;
  team_barrier(team + 1, tpr);
  if (warps > 8) return warp_sum(lane < warps ? red[lane] : 0.f);
  v = red[0];
  for (int w = 1; w < warps; ++w) v += red[w];
  return v;
}
// The same for two sums, in two halves: every warp gives its part, and after the team's
// barrier each thread takes the total (tpr 32 and less: the part is the total).
template <bool ONE>  // ONE: a is 0
TW_DEV float2 give_sum2(float a, float b, float2* red, int tpr, int tid) {
  if (tpr < 32) return make_float2(ONE ? a : lanes_sum(a, tpr, team_lanes(tpr)), lanes_sum(b, tpr, team_lanes(tpr)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if constexpr (!ONE) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  if (tpr > 32 && (tid & 31) == 0) red[tid >> 5] = make_float2(a, b);
  return make_float2(a, b);
}
TW_DEV float2 take_sum2(float2 own, const float2* red, int team, int tpr, int tid) {
  if (tpr <= 32) return own;
  const int lane = tid & 31, warps = tpr >> 5;
  team_barrier(team + 1, tpr);
  if (warps > 8) {
    const float2 p = lane < warps ? red[lane] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(p.x), warp_sum(p.y));
  }
  float2 v = red[0];
  for (int w = 1; w < warps; ++w) v.x += red[w].x, v.y += red[w].y;
  return v;
}

// A sum and a maximum over a team's threads (NaN where one is), one barrier.
TW_DEV float2 team_sum_max(float s, float m, float2* red, int team, int tpr, int tid) {
  if (tpr < 32) return make_float2(lanes_sum(s, tpr, team_lanes(tpr)), warp_max_nan(m, tpr, team_lanes(tpr)));
  s = warp_sum(s);
  m = warp_max_nan(m, 32);
  if (tpr == 32) return make_float2(s, m);
  const int lane = tid & 31, warp = tid >> 5, warps = tpr >> 5;
  if (lane == 0) red[warp] = make_float2(s, m);
  team_barrier(team + 1, tpr);
  if (warps > 8) {
    const float2 p = lane < warps ? red[lane] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(p.x), warp_max_nan(p.y, 32));
  }
  float2 v = red[0];
  for (int w = 1; w < warps; ++w) v.x += red[w].x, v.y = max_nan(v.y, red[w].y);
  return v;
}

// A team's ring: DEPTH rows of up to three tensors (0: no ring). VEC: each thread copies and
// reads back its own NV vectors, so that the ring needs no barrier. Else the row's aligned 16
// bytes as they lie in memory, copied by the whole team and read, two for a vector, after
// its barrier.
template <int DT, int VPT, int VEC, int DEPTH, int TPR>
struct Ring {
  using M = RowMap<DT, VPT, VEC, TPR>;
  using S = typename M::S;
  static constexpr int E = M::E, NV = M::NV, kExtra = VEC ? 0 : 1;
  uint4* mine;
  int tensors;
  TW_DEV Ring(uint4* smem, int team, int tensors_, const M& m)
      : mine(smem + team * (DEPTH * tensors_ * (NV * m.tpr() + kExtra)) + (VEC ? m.tid : 0)), tensors(tensors_) {}
  TW_DEV uint4* place(const M& m, int stage, int t) const { return mine + (stage * tensors + t) * (NV * m.tpr() + kExtra); }
  static TW_DEV int lead_of(const S* row) { return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(S)); }
  // careful: see end_row
  TW_DEV void copy(const M& m, int stage, int t, const S* row, bool careful) const {
    uint4* to = place(m, stage, t);
    if constexpr (VEC != ANYWHERE) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!m.has(k * E)) continue;
        const S* p = row + m.col(k * E);
        if (VEC == ALIKE && careful && m.edge && !m.whole(k)) {
          S* q = reinterpret_cast<S*>(to + k * m.tpr());
          for (int e = 0; e < E; ++e)
            if (m.in(k * E + e)) q[e] = p[e];
        } else {
          cp_async16(to + k * m.tpr(), p);
        }
      }
    } else {
      const int lead = lead_of(row), end = lead + m.d;
      auto one = [&](int g) {
        if (g * E >= end) return;
        const S* p = row - lead + g * E;
        if (careful && ((g == 0 && lead > 0) || g * E + E > end)) {
          S* q = reinterpret_cast<S*>(to + g);
          for (int e = 0; e < E; ++e)
            if (g * E + e >= lead && g * E + e < end) q[e] = p[e];
        } else {
          cp_async16(to + g, p);
        }
      };
#pragma unroll
      for (int k = 0; k < NV; ++k) one(k * m.tpr() + m.tid);
      if (m.tid == 0) one(NV * m.tpr());
    }
  }
  TW_DEV void read(const M& m, int stage, int t, const S* row, float2 (&v)[M::NP]) const {
    const uint4* from = place(m, stage, t);
    if constexpr (VEC != ANYWHERE) {
#pragma unroll
      for (int k = 0; k < NV; ++k) M::widen16(m.has(k * E) ? from[k * m.tpr()] : make_uint4(0, 0, 0, 0), v + k * E / 2);
      m.trim(v);
    } else {
      const int lead = lead_of(row);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int g = k * m.tpr() + m.tid, left = m.d - g * E;
        uint4 r = make_uint4(0, 0, 0, 0);
        if (left > 0) r = first_of<DT>(shifted_from<DT>(from + g, lead), left);
        M::widen16(r, v + k * E / 2);
      }
    }
  }
};
template <int TPR>
TW_DEV void team_sync(int team) {
  if constexpr (TPR == 32)
    __syncwarp();
  else
    team_barrier(team + 1, TPR);
}

// CTAs an SM of a forward kernel of so many threads: about 800 threads, so that while a
// team waits for the two sums over its row, the other CTAs' rows go on.
// RMS norm's rows of whole vectors of 16 bits: 1024 threads, one sum a row leaves less to
// wait for (8191 x 8192 into e4m3 with a scale a row 36 us, at 800 threads 41; 16384 x 2048
// 22 against 23; but off 16 bytes 54 against 42, and fp32 gains nothing).
constexpr int fwd_ctas(int threads, bool more) {
  if (more) return threads > 512 ? 1 : 1024 / threads;
  return threads > 448 ? 1 : threads > 320 ? 2 : 800 / threads;
}
constexpr bool fwd_more(int kind, int dtype, bool vec, int depth) { return kind != LAYER_NORM && dtype != TW_F32 && vec && depth > 0; }

template <int DT, int VPT, int VEC, int DEPTH, int TPR, int MAXT, int KIND>
__global__ void __launch_bounds__(MAXT, fwd_ctas(MAXT, fwd_more(KIND, DT, VEC == WHOLE, DEPTH))) norm_fwd_kernel(const NormFwdArgs a) {
  constexpr bool RMS = KIND != LAYER_NORM;
  using M = RowMap<DT, VPT, VEC, TPR>;
  using S = typename M::S;
  constexpr int NP = M::NP;
  extern __shared__ uint4 smem[];
  __shared__ std::conditional_t<KIND == RMS_FP8_ROW, float2, float> red[2][kMaxTeams][32];
  pdl_enter();
  const int tid = threadIdx.x, tpr = TPR > 0 ? TPR : blockDim.x, team = threadIdx.y, teams = TPR > 0 ? MAXT / TPR : blockDim.y;
  const int stride = gridDim.x * teams;
  int row = blockIdx.x * teams + team;
  auto at = [](const void* p, int64_t ld, int r) { return static_cast<const S*>(p) + static_cast<size_t>(r) * ld; };
  const M m(a.d, tid, tpr, static_cast<int>((reinterpret_cast<uintptr_t>(at(a.x, a.ldx, row)) & 15u) / sizeof(S)));
  const Ring<DT, VPT, VEC, DEPTH, TPR> ring(smem, team, a.res != nullptr ? 2 : 1, m);
  auto fetch = [&](int stage, int r) {
    if (r < a.T) {
      ring.copy(m, stage, 0, at(a.x, a.ldx, r), end_row(r, a.T, a.ldx, M::E));
      if (a.res != nullptr) ring.copy(m, stage, 1, at(a.res, a.ldres, r), end_row(r, a.T, a.ldres, M::E));
    }
    cp_commit();
  };
  if constexpr (DEPTH > 0) {
#pragma unroll
    for (int s = 0; s < DEPTH; ++s) fetch(s, row + s * stride);
  }
  float2 w[NP], b[NP];
  m.weight(a.w, a.wtype, 1.f, w);
  if constexpr (!RMS) m.weight(a.b, a.wtype, 0.f, b);
  const float inv_d = 1.f / static_cast<float>(a.d);
  if constexpr (DEPTH > 0 && !VEC) {
    cp_wait<DEPTH - 1>();
    team_sync<TPR>(team);
  }
  [[maybe_unused]] int flip = 0;
  for (int stage = 0; row < a.T; row += stride) {
    float2 v[NP], u[NP];
    if constexpr (DEPTH > 0) {
      if constexpr (VEC != ANYWHERE) cp_wait<DEPTH - 1>();  // else before the last row's second sum
      ring.read(m, stage, 0, at(a.x, a.ldx, row), v);
      if (a.res != nullptr) ring.read(m, stage, 1, at(a.res, a.ldres, row), u);
    } else {
      m.load(at(a.x, a.ldx, row), v, end_row(row, a.T, a.ldx, M::E));
      if (a.res != nullptr) m.load(at(a.res, a.ldres, row), u, end_row(row, a.T, a.ldres, M::E));
    }
    const size_t r = static_cast<size_t>(row);
    if (a.res != nullptr) {
#pragma unroll
      for (int i = 0; i < NP; ++i) v[i] = Elem<DT>::rounded(add2(v[i], u[i]));
      if (a.sum != nullptr) m.store(static_cast<S*>(a.sum) + r * a.ldsum, v);
    }
    if constexpr (RMS) {
      // one barrier a row: after it the row has left its places for all of the team, and the
      // next row, whose copies every thread waits for before it, is there for all
      float2 q = both(0.f);
#pragma unroll
      for (int i = 0; i < NP; ++i) q = fma2(v[i], v[i], q);
      float most = 0.f, ssq;
      if constexpr (DEPTH > 0 && !VEC) {
        cp_wait<DEPTH - 2>();
        if constexpr (TPR == 32) __syncwarp();
      }
      if constexpr (KIND == RMS_FP8_ROW) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const float2 g = mul2(v[i], w[i]);
          most = max_nan(most, max_nan(fabsf(g.x), fabsf(g.y)));
        }
        const float2 sm = team_sum_max(q.x + q.y, most, red[flip][team], team, tpr, tid);
        ssq = sm.x, most = sm.y;
      } else {
        ssq = team_sum(q.x + q.y, red[flip][team], team, tpr, tid);
      }
      flip ^= 1;
      if constexpr (DEPTH > 0) {
        fetch(stage, row + DEPTH * stride);
        stage = stage + 1 == DEPTH ? 0 : stage + 1;
      }
      const float rstd = rsqrtf(ssq * inv_d + a.eps);
#pragma unroll
      for (int i = 0; i < NP; ++i) v[i] = mul2(mul2(v[i], both(rstd)), w[i]);
      if constexpr (KIND == RMS_NORM) {
        m.store(static_cast<S*>(a.y) + r * a.ldy, v);
      } else {
        uint8_t* q8 = static_cast<uint8_t*>(a.y) + r * a.ldy;
        if constexpr (KIND == RMS_FP8_ROW) {
          const float scale = fp8_scale(most * rstd);
          if (tid == 0) a.scales[row] = scale;
          const float inv = reciprocal(scale);
#pragma unroll
          for (int i = 0; i < NP; ++i) v[i] = mul2(v[i], both(inv));
        } else {
          constexpr int E = M::E, kLanes = kFp8Group / E;
          const int groups = (a.d + kFp8Group - 1) / kFp8Group;
#pragma unroll
          for (int k = 0; k < M::NV; ++k) {
            float g = 0.f;
#pragma unroll
            for (int e = k * E / 2; e < (k + 1) * E / 2; ++e) g = max_nan(g, max_nan(fabsf(v[e].x), fabsf(v[e].y)));
            const float scale = fp8_scale(warp_max_nan(g, kLanes, team_lanes(tpr)));
            const int c = m.col(k * E);
            if (c < a.d && c % kFp8Group == 0) a.scales[r * groups + c / kFp8Group] = scale;
            const float inv = reciprocal(scale);
#pragma unroll
            for (int e = k * E / 2; e < (k + 1) * E / 2; ++e) v[e] = mul2(v[e], both(inv));
          }
        }
        m.store_fp8(q8, v);
      }
      if (tid == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
    } else {
      float2 s = v[0];
#pragma unroll
      for (int i = 1; i < NP; ++i) s = add2(s, v[i]);
      const float mean = team_sum(s.x + s.y, red[0][team], team, tpr, tid) * inv_d;
      if constexpr (DEPTH > 0) {  // the row has left its places
        fetch(stage, row + DEPTH * stride);
        stage = stage + 1 == DEPTH ? 0 : stage + 1;
        if constexpr (!VEC) {  // the next row is here, and after the second sum's barrier for all
          cp_wait<DEPTH - 1>();
          if constexpr (TPR == 32) __syncwarp();
        }
      }
      float2 q = both(0.f);
#pragma unroll
      for (int i = 0; i < NP; ++i) v[i] = add2(v[i], both(-mean));
      m.trim(v);
      m.each([&](int i) { q = fma2(v[i], v[i], q); });
      const float rstd = rsqrtf(team_sum(q.x + q.y, red[1][team], team, tpr, tid) * inv_d + a.eps);
#pragma unroll
      for (int i = 0; i < NP; ++i) v[i] = fma2(mul2(v[i], both(rstd)), w[i], b[i]);
      m.store(static_cast<S*>(a.y) + r * a.ldy, v);
      if (tid == 0) {
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
      }
    }
  }
}

// One CTA of about 512 threads an SM, 16 elements of a row a thread: the column sums of dw
// and db, 32 registers a thread, are kept once for all of a team's rows and go to memory
// once an SM. 16384 x 2048 bf16 with dres, in microseconds: 512 threads and a ring of three
// rows 51.2, of four 57.6; 640 threads 79, 768 62, 1024 65.8; the saved statistics three
// rows ahead in registers 53.7; with the partial sums in the threads' order 47.4; one row
// ahead (below), a ring of four, 46.7, and 4096 x 8192, where one team has the SM to
// itself, 49.7 in place of 55.8.
template <int DT, int VPT, int VEC, int DEPTH, int TPR, int MAXT, bool RMS>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const NormBwdArgs a) {
  using M = RowMap<DT, VPT, VEC, TPR>;
  using S = typename M::S;
  constexpr int NP = M::NP;
  extern __shared__ uint4 smem[];  // the ring; then the teams' column sums
  __shared__ float2 red[2][kMaxTeams][32];
  pdl_enter();
  const int tid = threadIdx.x, tpr = TPR > 0 ? TPR : blockDim.x, team = threadIdx.y, teams = TPR > 0 ? MAXT / TPR : blockDim.y;
  const int stride = gridDim.x * teams;
  const int first = blockIdx.x * teams + team;
  int row = first;
  auto at = [](const void* p, int64_t ld, int r) { return static_cast<const S*>(p) + static_cast<size_t>(r) * ld; };
  const M m(a.d, tid, tpr, static_cast<int>((reinterpret_cast<uintptr_t>(at(a.x, a.ldx, row)) & 15u) / sizeof(S)));
  const Ring<DT, VPT, VEC, DEPTH, TPR> ring(smem, team, a.dres != nullptr ? 3 : 2, m);
  auto fetch = [&](int stage, int r) {
    if (r < a.T) {
      ring.copy(m, stage, 0, at(a.x, a.ldx, r), end_row(r, a.T, a.ldx, M::E));
      ring.copy(m, stage, 1, at(a.dy, a.lddy, r), end_row(r, a.T, a.lddy, M::E));
      if (a.dres != nullptr) ring.copy(m, stage, 2, at(a.dres, a.lddres, r), end_row(r, a.T, a.lddres, M::E));
    }
    cp_commit();
  };
  if constexpr (DEPTH > 0) {
#pragma unroll
    for (int s = 0; s < DEPTH; ++s) fetch(s, row + s * stride);
  }
  float2 w[NP], dw[NP], db[NP];
  m.weight(a.w, a.wtype, 1.f, w);
#pragma unroll
  for (int i = 0; i < NP; ++i) dw[i] = db[i] = both(0.f);
  const float inv_d = 1.f / static_cast<float>(a.d);
  // x becomes xh, g dy w; the thread's parts of the row's two sums, and its column sums.
  // Past the row g is 0, so what xh is there adds nothing.
  auto sums = [&](float2 (&x)[NP], float2 (&g)[NP], float mean, float rstd, float2* to) {
    float2 c1 = both(0.f), c2 = both(0.f);
    m.each([&](int i) {
      x[i] = mul2(centred<RMS>(x[i], mean), both(rstd));
      dw[i] = fma2(g[i], x[i], dw[i]);
      if constexpr (!RMS) db[i] = add2(db[i], g[i]);
      g[i] = mul2(g[i], w[i]);
      if constexpr (!RMS) c1 = add2(c1, g[i]);
      c2 = fma2(g[i], x[i], c2);
    });
    return give_sum2<RMS>(c1.x + c1.y, c2.x + c2.y, to, tpr, tid);
  };
  auto finish = [&](const float2 (&x)[NP], float2 (&g)[NP], const float2 (&more)[NP], float2 c, float rstd, int r) {
    [[maybe_unused]] const float2 k1 = both(-c.x * inv_d);
    const float2 k2 = both(-c.y * inv_d);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if constexpr (RMS)
        g[i] = mul2(fma2(x[i], k2, g[i]), both(rstd));
      else
        g[i] = mul2(add2(g[i], fma2(x[i], k2, k1)), both(rstd));
      if (a.dres != nullptr) g[i] = add2(g[i], more[i]);
    }
    m.store(static_cast<S*>(a.dx) + static_cast<size_t>(r) * a.lddx, g);
  };
  auto mean_of = [&](int r) { return !RMS && r < a.T ? a.mean[r] : 0.f; };
  auto rstd_of = [&](int r) { return r < a.T ? a.rstd[r] : 0.f; };
  float mean = mean_of(row), rstd = rstd_of(row);
  if constexpr (DEPTH >= 4) {
    // One row ahead: the team's barrier finds the parts of this row's sums long given, and
    // the next row's sums are taken before this row's dx, both from the ring. Without VEC the
    // barrier also says that the next row is there for all, and that the last one is read:
    // only then are its places filled again.
    float mean_next = mean_of(row + stride), rstd_next = rstd_of(row + stride);
    float2 part = both(0.f);
    if (row < a.T) {
      float2 x[NP], g[NP];
      cp_wait<DEPTH - 1>();
      if constexpr (!VEC) team_sync<TPR>(team);
      ring.read(m, 0, 0, at(a.x, a.ldx, row), x);
      ring.read(m, 0, 1, at(a.dy, a.lddy, row), g);
      part = sums(x, g, mean, rstd, red[0][team]);
    }
    for (int flip = 0, stage = 0; row < a.T; row += stride, flip ^= 1) {
      const int next = stage + 1 == DEPTH ? 0 : stage + 1;
      const float mean_2 = mean_of(row + 2 * stride), rstd_2 = rstd_of(row + 2 * stride);
      if constexpr (!VEC) {
        cp_wait<DEPTH - 3>();
        if constexpr (TPR == 32) __syncwarp();
      }
      const float2 c = take_sum2(part, red[flip][team], team, tpr, tid);
      if constexpr (!VEC) {
        if (row >= first + stride) fetch(stage == 0 ? DEPTH - 1 : stage - 1, row + (DEPTH - 1) * stride);
      }
      if (row + stride < a.T) {
        float2 x[NP], g[NP];
        if constexpr (VEC != ANYWHERE) cp_wait<DEPTH - 2>();
        ring.read(m, next, 0, at(a.x, a.ldx, row + stride), x);
        ring.read(m, next, 1, at(a.dy, a.lddy, row + stride), g);
        part = sums(x, g, mean_next, rstd_next, red[flip ^ 1][team]);
      }
      float2 x[NP], g[NP], more[NP];
      ring.read(m, stage, 0, at(a.x, a.ldx, row), x);
      ring.read(m, stage, 1, at(a.dy, a.lddy, row), g);
      if (a.dres != nullptr) ring.read(m, stage, 2, at(a.dres, a.lddres, row), more);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        x[i] = mul2(centred<RMS>(x[i], mean), both(rstd));
        g[i] = mul2(g[i], w[i]);
      }
      finish(x, g, more, c, rstd, row);
      if constexpr (VEC != ANYWHERE) fetch(stage, row + DEPTH * stride);
      stage = next;
      mean = mean_next, rstd = rstd_next;
      mean_next = mean_2, rstd_next = rstd_2;
    }
  } else {
    for (int flip = 0, stage = 0; row < a.T; row += stride, flip ^= 1) {
      float2 x[NP], g[NP], more[NP];
      if constexpr (DEPTH > 0) {
        cp_wait<DEPTH - 1>();
        static_assert(DEPTH == 0 || VEC, "rows read by others need the form above");
        ring.read(m, stage, 0, nullptr, x);
        ring.read(m, stage, 1, nullptr, g);
        if (a.dres != nullptr) ring.read(m, stage, 2, nullptr, more);
      } else {
        m.load(at(a.x, a.ldx, row), x, end_row(row, a.T, a.ldx, M::E));
        m.load(at(a.dy, a.lddy, row), g, end_row(row, a.T, a.lddy, M::E));
      }
      const float2 part = sums(x, g, mean, rstd, red[flip][team]);
      const float2 c = take_sum2(part, red[flip][team], team, tpr, tid);
      if constexpr (DEPTH > 0) {  // the row has left its places
        fetch(stage, row + DEPTH * stride);
        stage = stage + 1 == DEPTH ? 0 : stage + 1;
      } else if (a.dres != nullptr) {
        m.load(at(a.dres, a.lddres, row), more, end_row(row, a.T, a.lddres, M::E));
      }
      const float mean_next = mean_of(row + stride), rstd_next = rstd_of(row + stride);
      finish(x, g, more, c, rstd, row);
      mean = mean_next, rstd = rstd_next;
    }
  }
  if (a.part == nullptr) return;
  // The CTA's partial sums, [2][NE tpr] ([1] of RMS norm), in the order of the threads' own elements: a
  // column order would have every access of a warp hit 32 banks' worth of conflicts here
  // and 32 sectors there (it made the sums cost 8 us a call). The last kernel sorts.
  const int width = M::NE * tpr;
  constexpr int kSums = RMS ? 1 : 2;
  float* out = a.part + static_cast<size_t>(blockIdx.x) * kSums * width;
  float* acc = reinterpret_cast<float*>(smem) + team * kSums * width;
  if (teams == 1) acc = out;
  if (DEPTH > 0) {
    cp_wait<0>();
    __syncthreads();
  }
  if constexpr (VEC == ALIKE) {  // the places of the columns without a lead; lanes' are neighbours here too
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) {
      constexpr int E = M::E;
      const int back = m.lead > i % E ? 1 : 0, g = i / E * tpr + tid - back, e = i % E - m.lead + back * E;
      if (m.in(i)) acc[(g / tpr * E + e) * tpr + g % tpr] = i % 2 ? dw[i / 2].y : dw[i / 2].x;
    }
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    if constexpr (VEC == ALIKE) break;
    acc[2 * i * tpr + tid] = dw[i].x;
    acc[(2 * i + 1) * tpr + tid] = dw[i].y;
    if constexpr (!RMS) {
      acc[width + 2 * i * tpr + tid] = db[i].x;
      acc[width + (2 * i + 1) * tpr + tid] = db[i].y;
    }
  }
  if (teams == 1) return;
  __syncthreads();
  acc = reinterpret_cast<float*>(smem);
  for (int p = team * tpr + tid; p < kSums * width; p += teams * tpr) {
    float v = acc[p];
    for (int t = 1; t < teams; ++t) v += acc[t * kSums * width + p];
    out[p] = v;
  }
}

// The backward of a few rows in one launch. The sums over rows need the saved statistics
// only, not the rows' c1 and c2, so they are not kept waiting for them: the first row_ctas
// CTAs take dx, a row a team, and the others 256 columns each, whose rows they read once
// more (from L2) over 16 warps, joined in order.
constexpr int kFewThreads = 512, kFewWarps = kFewThreads / 32, kFewColumns = 256;

template <int DT, int VPT, int VEC, bool RMS>
__global__ void __launch_bounds__(kFewThreads) norm_bwd_few_kernel(const NormBwdArgs a, int tpr, int row_ctas) {
  using S = typename Elem<DT>::S;
  __shared__ float2 red[kMaxTeams + 1][32];
  __shared__ float sums[kFewWarps][2 * kFewColumns];
  pdl_enter();
  auto at = [](const void* p, int64_t ld, int r) { return static_cast<const S*>(p) + static_cast<size_t>(r) * ld; };
  if (static_cast<int>(blockIdx.x) < row_ctas) {
    using M = RowMap<DT, VPT, VEC, 0>;
    const int team = threadIdx.x / tpr, teams = min(kFewThreads / tpr, kMaxTeams);
    const int row = blockIdx.x * teams + team;
    if (team >= teams || row >= a.T) return;
    const M m(a.d, threadIdx.x - team * tpr, tpr);
    float2 x[M::NP], g[M::NP], w[M::NP];
    m.load(at(a.x, a.ldx, row), x, end_row(row, a.T, a.ldx, M::E));
    m.load(at(a.dy, a.lddy, row), g, end_row(row, a.T, a.lddy, M::E));
    const float mean = RMS ? 0.f : a.mean[row], rstd = a.rstd[row];
    m.weight(a.w, a.wtype, 1.f, w);
    float2 c1 = both(0.f), c2 = both(0.f);
    m.each([&](int i) {
      x[i] = mul2(centred<RMS>(x[i], mean), both(rstd));
      g[i] = mul2(g[i], w[i]);
      if constexpr (!RMS) c1 = add2(c1, g[i]);
      c2 = fma2(g[i], x[i], c2);
    });
    if (a.dres != nullptr) m.load(at(a.dres, a.lddres, row), w, end_row(row, a.T, a.lddres, M::E));
    const float2 c = take_sum2(give_sum2<RMS>(c1.x + c1.y, c2.x + c2.y, red[team], tpr, m.tid), red[team], team, tpr, m.tid);
    const float inv_d = 1.f / static_cast<float>(a.d);
    [[maybe_unused]] const float2 k1 = both(-c.x * inv_d);
    const float2 k2 = both(-c.y * inv_d);
#pragma unroll
    for (int i = 0; i < M::NP; ++i) {
      if constexpr (RMS)
        g[i] = mul2(fma2(x[i], k2, g[i]), both(rstd));
      else
        g[i] = mul2(add2(g[i], fma2(x[i], k2, k1)), both(rstd));
      if (a.dres != nullptr) g[i] = add2(g[i], w[i]);
    }
    m.store(static_cast<S*>(a.dx) + static_cast<size_t>(row) * a.lddx, g);
    return;
  }
  using M = RowMap<DT, 1, VEC, 32>;
  const int first = (blockIdx.x - row_ctas) * kFewColumns, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const M m(a.d - first, lane, 32);
  float2 dw[M::NP], db[M::NP];
#pragma unroll
  for (int i = 0; i < M::NP; ++i) dw[i] = db[i] = both(0.f);
#pragma unroll 4
  for (int row = warp; row < a.T; row += kFewWarps) {
    float2 x[M::NP], g[M::NP];
    m.load(at(a.x, a.ldx, row) + first, x, end_row(row, a.T, a.ldx, M::E));
    m.load(at(a.dy, a.lddy, row) + first, g, end_row(row, a.T, a.lddy, M::E));
    const float mean = RMS ? 0.f : a.mean[row], rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < M::NP; ++i) {
      dw[i] = fma2(g[i], mul2(centred<RMS>(x[i], mean), both(rstd)), dw[i]);
      if constexpr (!RMS) db[i] = add2(db[i], g[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < M::NP; ++i) {
    sums[warp][m.col(2 * i)] = dw[i].x, sums[warp][m.col(2 * i + 1)] = dw[i].y;
    if constexpr (!RMS)
      sums[warp][kFewColumns + m.col(2 * i)] = db[i].x, sums[warp][kFewColumns + m.col(2 * i + 1)] = db[i].y;
  }
  __syncthreads();
  if (RMS && threadIdx.x >= kFewColumns) return;
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < kFewWarps; ++k) v += sums[k][threadIdx.x];
  const int c = first + static_cast<int>(threadIdx.x) % kFewColumns;
  float* out = threadIdx.x < kFewColumns ? a.dw : a.db;
  if (c < a.d && out != nullptr) out[c] = v;
}

// dw, db = the partial sums of `n` CTAs, added in a fixed order. width, tpr, E: the order
// of a partial's places (RowMap::col); sums: 2, or 1 without db.
__global__ void __launch_bounds__(512) norm_bwd_finish_kernel(const float* part, int n, int sums, int d, int width, int tpr, int E,
                                                              float* dw, float* db) {
  __shared__ float s[16][33];
  pdl_enter();
  const int p = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
#pragma unroll 4
  for (int i = threadIdx.y; i < n; i += 16) v += part[static_cast<size_t>(i) * sums * width + p];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += s[i][threadIdx.x];
  const int q = p < width ? p : p - width, i = q / tpr, c = (i / E * tpr + q % tpr) * E + i % E;
  float* out = p < width ? dw : db;
  if (c < d && out != nullptr) out[c] = v;
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

template <class Kern, class Args>
cudaError_t launch_norm(Kern kern, int grid, const Team& t, size_t smem, const char* label, const Args& a,
                        cudaStream_t s) {
  cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  e = launch(kern, dim3(grid), dim3(t.tpr, t.teams), smem, s, a);
  trace_mark(s, label);
  return e;
}

// Rows through a ring of DEPTH: MAXT / TPR teams of TPR threads, 16 elements a thread.
size_t ring_bytes(int dtype, int vpt, const Team& t, int depth, int tensors, bool vec) {
  return t.teams * depth * tensors * (t.tpr * 8 * vpt * elem_size(dtype) + (vec ? 0 : 16));
}
// Of `want` CTAs (at most `most`) of so many teams: as many as make a team's rows a multiple of a
// vector's elements apart where they have to be.
int grid_of(int want, int most, int teams, int dtype, int vec) {
  if (vec != ALIKE) return std::min(want, most);
  int step = dtype == TW_F32 ? 4 : 8;
  while (step > 1 && teams % 2 == 0) step /= 2, teams /= 2;
  return std::max(step, std::min((want + step - 1) / step * step, most / step * step));
}
template <int KIND, int DT, int TPR, int MAXT, int VPT = 2, int VEC = WHOLE>
cudaError_t norm_fwd_ring(const NormFwdArgs& a, cudaStream_t s) {
  constexpr int kTeams = MAXT / TPR;
  const size_t smem = ring_bytes(DT, VPT, Team{TPR, kTeams}, 3, a.res != nullptr ? 2 : 1, VEC);
  // as many CTAs as stay resident
  const int fit = static_cast<int>(kSmemMost / (smem + 6 * 1024));
  const int per_sm = std::max(1, std::min(fwd_ctas(MAXT, fwd_more(KIND, DT, VEC == WHOLE, 3)), fit));
  return launch_norm(norm_fwd_kernel<DT, VPT, VEC, 3, TPR, MAXT, KIND>,
                     grid_of((a.T + kTeams - 1) / kTeams, device_sm_count() * per_sm, kTeams, DT, VEC), Team{TPR, kTeams}, smem,
                     "norm_fwd", a, s);
}
template <int KIND, int DT, int VPT, int VEC, int MAXT>
cudaError_t norm_fwd_direct(const NormFwdArgs& a, cudaStream_t s) {
  const Team t = team_of(a.d, VPT, MAXT <= 256 ? 256 : 32, a.T);
  return launch_norm(norm_fwd_kernel<DT, VPT, VEC, 0, 0, MAXT, KIND>,
                     std::min((a.T + t.teams - 1) / t.teams, device_sm_count() * 8), t, 0, "norm_fwd", a, s);
}

cudaError_t norm_bwd_finish(const NormBwdArgs& a, int sums, int partials, int width, int tpr, int E, cudaStream_t s) {
  cudaError_t e = launch(norm_bwd_finish_kernel, dim3(sums * width / 32), dim3(32, 16), 0, s,
                         static_cast<const float*>(a.part), partials, sums, a.d, width, tpr, E, a.dw, a.db);
  trace_mark(s, "norm_bwd_finish");
  return e;
}

template <bool RMS, int DT, int VPT, int VEC, int DEPTH, int TPR, int MAXT>
cudaError_t norm_bwd(const NormBwdArgs& a, const Team& t, cudaStream_t s) {
  using M = RowMap<DT, VPT, VEC, TPR>;
  constexpr int kSums = RMS ? 1 : 2;
  const int grid = grid_of((a.T + t.teams - 1) / t.teams, std::min(device_sm_count(), kNormPartials), t.teams, DT, VEC);
  const int width = M::NE * t.tpr;
  if (a.part != nullptr && static_cast<size_t>(kSums) * grid * width > norm_partial_floats(a.T, a.d, RMS)) return cudaErrorInvalidValue;
  const size_t smem = std::max(ring_bytes(DT, VPT, t, DEPTH, a.dres != nullptr ? 3 : 2, VEC),
                               t.teams > 1 ? kSums * sizeof(float) * t.teams * width : size_t{0});
  const cudaError_t e = launch_norm(norm_bwd_kernel<DT, VPT, VEC, DEPTH, TPR, MAXT, RMS>, grid, t, smem, "norm_bwd", a, s);
  return e != cudaSuccess || a.part == nullptr ? e : norm_bwd_finish(a, kSums, grid, width, t.tpr, M::E, s);
}
template <bool RMS, int DT, int VPT, int TPR, int MAXT, int DEPTH, int VEC = WHOLE>
cudaError_t norm_bwd_ring(const NormBwdArgs& a, cudaStream_t s) {
  return norm_bwd<RMS, DT, VPT, VEC, DEPTH, TPR, MAXT>(a, Team{TPR, MAXT / TPR}, s);
}
template <bool RMS, int DT, int VPT, int VEC, int MAXT>
cudaError_t norm_bwd_direct(const NormBwdArgs& a, cudaStream_t s) {
  return norm_bwd<RMS, DT, VPT, VEC, 0, 0, MAXT>(a, team_of(a.d, VPT, MAXT, a.T), s);
}

// Whether dx and an input matrix share memory.
bool overlap(const NormBwdArgs& a, const void* p, int64_t ld) {
  const size_t es = elem_size(a.dtype), rows = static_cast<size_t>(a.T) - 1;
  const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(a.dx);
  return x < y + es * (rows * a.lddx + a.d) && y < x + es * (rows * ld + a.d);
}

// Up to so many rows: one launch (norm_bwd_few_kernel). 77 rows of 2048 bf16 take 2.7 us
// against 6 in two; the two meet between 250 (512 columns) and 430 rows (8192), and at 200
// rows off 16 bytes.
constexpr int kFewRows = 320, kFewRowsOff16 = 160;
template <bool RMS, int DT, int VEC>
cudaError_t norm_bwd_few(const NormBwdArgs& a, cudaStream_t s) {
  const int vpt = a.d <= 4096 ? 1 : 2;
  const int tpr = ((a.d + 8 * vpt - 1) / (8 * vpt) + 31) / 32 * 32, teams = std::min(kFewThreads / tpr, kMaxTeams);
  const int row_ctas = (a.T + teams - 1) / teams;
  const int column_ctas = a.part == nullptr ? 0 : (a.d + kFewColumns - 1) / kFewColumns;
  const cudaError_t e = launch(vpt == 1 ? norm_bwd_few_kernel<DT, 1, VEC, RMS> : norm_bwd_few_kernel<DT, 2, VEC, RMS>,
                               dim3(row_ctas + column_ctas), dim3(kFewThreads), 0, s, a, tpr, row_ctas);
  trace_mark(s, "norm_bwd_few");
  return e;
}

// The least team that holds the row at 16 elements a thread, and three rows in the ring
// (the backward: four, in fp32 two). Rows that take a CTA's whole team: 8 elements a thread
// where that makes more warps without spills. Backward with dres, 33.5 M elements bf16: 5120
// columns 54.5 us (16 a thread 64.1), 5632 54.9 (61.9), but 6656 57.2 (52.3), 8192 79 (49.7);
// fp32, 16.8 M: 5632 49.8 (64.2), 8192 59.6 (48.2). Forward without residual: bf16 5632 37.4
// (27.5), 8192 33.2 (27.8); fp32 7168 23.2 (25.0).
template <int KIND, int DT, int VEC>
cudaError_t norm_fwd_width(const NormFwdArgs& a, cudaStream_t s) {
  if constexpr (VEC != ANYWHERE) {
    const int d = VEC == ALIKE ? a.d + Elem<DT>::E - 1 : a.d;
    if constexpr (VEC == WHOLE && KIND != LAYER_NORM) {  // several rows a warp
      if constexpr (KIND != RMS_FP8_GROUP) {  // (of 128 columns and less: by row)
        if (d <= 16 * 4) return norm_fwd_ring<KIND, DT, 4, 256>(a, s);
        if (d <= 16 * 8) return norm_fwd_ring<KIND, DT, 8, 256>(a, s);
      }
      if constexpr (KIND != RMS_FP8_GROUP || DT != TW_F32) {  // (16 lanes hold a group in 16 bits)
        if (d <= 16 * 16) return norm_fwd_ring<KIND, DT, 16, 256>(a, s);
      }
    }
    if (d <= 16 * 32) return norm_fwd_ring<KIND, DT, 32, 256, 2, VEC>(a, s);
    if (d <= 16 * 64) return norm_fwd_ring<KIND, DT, 64, 256, 2, VEC>(a, s);
    if (d <= 16 * 96) return norm_fwd_ring<KIND, DT, 96, 192, 2, VEC>(a, s);
    if (d <= 16 * 128) return norm_fwd_ring<KIND, DT, 128, 256, 2, VEC>(a, s);
    if (d <= 16 * 160) return norm_fwd_ring<KIND, DT, 160, 320, 2, VEC>(a, s);
    if (d <= 16 * 192) return norm_fwd_ring<KIND, DT, 192, 192, 2, VEC>(a, s);
    if (d <= 16 * 256) return norm_fwd_ring<KIND, DT, 256, 256, 2, VEC>(a, s);
    if (d <= 16 * 320) return norm_fwd_ring<KIND, DT, 320, 320, 2, VEC>(a, s);
    if (d <= 16 * 384) return norm_fwd_ring<KIND, DT, 384, 384, 2, VEC>(a, s);
    if constexpr (DT == TW_F32) {
      if (d <= 8 * 896) return norm_fwd_ring<KIND, DT, 896, 896, 1, VEC>(a, s);
      if (d <= 8 * 1024) return norm_fwd_ring<KIND, DT, 1024, 1024, 1, VEC>(a, s);
    } else {
      if (d <= 16 * 448) return norm_fwd_ring<KIND, DT, 448, 448, 2, VEC>(a, s);
      if (d <= 16 * 512) return norm_fwd_ring<KIND, DT, 512, 512, 2, VEC>(a, s);
    }
    return norm_fwd_direct<KIND, DT, 2, VEC == WHOLE ? WHOLE : ANYWHERE, 1024>(a, s);
  } else {
    if (a.d <= 16 * 32) return norm_fwd_ring<KIND, DT, 32, 256, 2, false>(a, s);
    if (a.d <= 16 * 64) return norm_fwd_ring<KIND, DT, 64, 256, 2, false>(a, s);
    if (a.d <= 16 * 96) return norm_fwd_ring<KIND, DT, 96, 192, 2, false>(a, s);
    if (a.d <= 16 * 128) return norm_fwd_ring<KIND, DT, 128, 256, 2, false>(a, s);
    if (a.d <= 16 * 192) return norm_fwd_ring<KIND, DT, 192, 192, 2, false>(a, s);
    if (a.d <= 16 * 256) return norm_fwd_ring<KIND, DT, 256, 256, 2, false>(a, s);
    if (a.d <= 16 * 320) return norm_fwd_ring<KIND, DT, 320, 320, 2, false>(a, s);
    if (a.d <= 16 * 384) return norm_fwd_ring<KIND, DT, 384, 384, 2, false>(a, s);
    if (a.d <= 16 * 512) return norm_fwd_ring<KIND, DT, 512, 512, 2, false>(a, s);
    return norm_fwd_direct<KIND, DT, 2, false, 1024>(a, s);
  }
}
template <bool RMS, int DT, int VEC>
cudaError_t norm_bwd_width(const NormBwdArgs& a, cudaStream_t s) {
  // (its column sums read x and dy while rows of dx are written: not in place of them)
  if (a.T <= (VEC == WHOLE ? kFewRows : kFewRowsOff16) && a.d <= 8192 && !overlap(a, a.x, a.ldx) && !overlap(a, a.dy, a.lddy))
    return norm_bwd_few<RMS, DT, VEC == WHOLE ? WHOLE : ANYWHERE>(a, s);
  if constexpr (VEC != ANYWHERE) {
    const int d = VEC == ALIKE ? a.d + Elem<DT>::E - 1 : a.d;
    constexpr int kDepth = DT == TW_F32 ? 2 : 4;
    if constexpr (VEC == WHOLE && RMS) {  // several rows a warp
      if (d <= 16 * 4) return norm_bwd_ring<RMS, DT, 2, 4, 512, kDepth>(a, s);
      if (d <= 16 * 8) return norm_bwd_ring<RMS, DT, 2, 8, 512, kDepth>(a, s);
      if (d <= 16 * 16) return norm_bwd_ring<RMS, DT, 2, 16, 512, kDepth>(a, s);
    }
    if (d <= 16 * 32) return norm_bwd_ring<RMS, DT, 2, 32, 480, kDepth, VEC>(a, s);
    if (d <= 16 * 64) return norm_bwd_ring<RMS, DT, 2, 64, 512, kDepth, VEC>(a, s);
    if (d <= 16 * 96) return norm_bwd_ring<RMS, DT, 2, 96, 480, kDepth, VEC>(a, s);
    if (d <= 16 * 128) return norm_bwd_ring<RMS, DT, 2, 128, 512, kDepth, VEC>(a, s);
    if (d <= 16 * 160) return norm_bwd_ring<RMS, DT, 2, 160, 480, kDepth, VEC>(a, s);
    if (d <= 16 * 256) return norm_bwd_ring<RMS, DT, 2, 256, 512, kDepth, VEC>(a, s);
    if (d <= 8 * 640) return norm_bwd_ring<RMS, DT, 1, 640, 640, kDepth, VEC>(a, s);
    if (d <= 8 * 704) return norm_bwd_ring<RMS, DT, 1, 704, 704, kDepth, VEC>(a, s);
    if constexpr (DT == TW_F32) {
      if (d <= 8 * 896) return norm_bwd_ring<RMS, DT, 1, 896, 896, kDepth, VEC>(a, s);
    }
    if (d <= 16 * 512) return norm_bwd_ring<RMS, DT, 2, 512, 512, kDepth, VEC>(a, s);
    return norm_bwd_direct<RMS, DT, 2, VEC == WHOLE ? WHOLE : ANYWHERE, 1024>(a, s);
  } else {
    constexpr int kVpt = DT == TW_F32 ? 1 : 2, kE = 8 * kVpt;
    if (a.d <= kE * 32) return norm_bwd_ring<RMS, DT, kVpt, 32, 480, 4, false>(a, s);
    if (a.d <= kE * 64) return norm_bwd_ring<RMS, DT, kVpt, 64, 512, 4, false>(a, s);
    if (a.d <= kE * 96) return norm_bwd_ring<RMS, DT, kVpt, 96, 480, 4, false>(a, s);
    if (a.d <= kE * 128) return norm_bwd_ring<RMS, DT, kVpt, 128, 512, 4, false>(a, s);
    if (a.d <= kE * 160) return norm_bwd_ring<RMS, DT, kVpt, 160, 480, 4, false>(a, s);
    if (a.d <= kE * 256) return norm_bwd_ring<RMS, DT, kVpt, 256, 512, 4, false>(a, s);
    if (a.d <= kE * 512) return norm_bwd_ring<RMS, DT, kVpt, 512, 512, 4, false>(a, s);
    return a.d <= 8192 ? norm_bwd_direct<RMS, DT, 1, false, 1024>(a, s) : norm_bwd_direct<RMS, DT, 2, false, 1024>(a, s);
  }
}

// Whether rows of stride ld from p on lie as x's do, each as many bytes behind 16 (p null: yes).
bool alike(const void* p, int64_t ld, const void* x, int64_t ldx, int dtype) {
  return p == nullptr || (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(x)) & 15u) == 0 && stride16(ld - ldx, dtype));
}

// By the type, and by how the rows lie: every one on 16 bytes (an 8-bit one on 8) and of whole
// vectors, or all alike, or not. (An 8-bit row's scales of 128 columns want whole vectors.)
template <int KIND, int DT>
cudaError_t norm_fwd_rows(const NormFwdArgs& a, cudaStream_t s) {
  bool vec = a.d % 8 == 0 && on16(a.x) && on16(a.res) && on16(a.sum) && on16(a.w) && on16(a.b) && stride16(a.ldx, DT) &&
             stride16(a.ldres, DT) && stride16(a.ldsum, DT);
  if constexpr (KIND == LAYER_NORM || KIND == RMS_NORM)
    vec = vec && on16(a.y) && stride16(a.ldy, DT);
  else
    vec = vec && (reinterpret_cast<uintptr_t>(a.y) & 7u) == 0 && a.ldy % 8 == 0;
  if (vec) return norm_fwd_width<KIND, DT, WHOLE>(a, s);
  if constexpr (KIND == RMS_NORM || KIND == RMS_FP8_ROW) {
    if (a.d <= 8192 - 8 && alike(a.res, a.ldres, a.x, a.ldx, DT) && alike(a.sum, a.ldsum, a.x, a.ldx, DT) &&
        (KIND == RMS_FP8_ROW || alike(a.y, a.ldy, a.x, a.ldx, DT)))
      return norm_fwd_width<KIND, DT, ALIKE>(a, s);
  }
  return norm_fwd_width<KIND, DT, ANYWHERE>(a, s);
}
template <int KIND>
cudaError_t norm_fwd(const NormFwdArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if constexpr (KIND == RMS_FP8_GROUP) {
    if (a.d <= kFp8Group) return norm_fwd<RMS_FP8_ROW>(a, s);
  }
  switch (a.dtype) {
    case TW_F32: return norm_fwd_rows<KIND, TW_F32>(a, s);
    case TW_BF16: return norm_fwd_rows<KIND, TW_BF16>(a, s);
    default: return norm_fwd_rows<KIND, TW_F16>(a, s);
  }
}

template <bool RMS, int DT>
cudaError_t norm_bwd_rows(const NormBwdArgs& a, cudaStream_t s) {
  const bool vec = a.d % 8 == 0 && on16(a.x) && on16(a.dy) && on16(a.dres) && on16(a.dx) && on16(a.w) &&
                   stride16(a.ldx, DT) && stride16(a.lddy, DT) && stride16(a.lddres, DT) && stride16(a.lddx, DT);
  if (vec) return norm_bwd_width<RMS, DT, WHOLE>(a, s);
  if constexpr (RMS) {
    // (512: the CTAs, rounded up, are not more than the rows, which the workspace has partials for)
    if (a.T >= 512 && a.d <= 8192 - 8 && alike(a.dy, a.lddy, a.x, a.ldx, DT) && alike(a.dres, a.lddres, a.x, a.ldx, DT) &&
        alike(a.dx, a.lddx, a.x, a.ldx, DT))
      return norm_bwd_width<RMS, DT, ALIKE>(a, s);
  }
  return norm_bwd_width<RMS, DT, ANYWHERE>(a, s);
}
template <bool RMS>
cudaError_t norm_bwd_any(const NormBwdArgs& a, cudaStream_t s) {
  if (a.T == 0) {  // sums over no rows
    const int width = (a.d + 31) / 32 * 32;
    return a.dw != nullptr || a.db != nullptr ? norm_bwd_finish(a, RMS ? 1 : 2, 0, width, width, 1, s) : cudaSuccess;
  }
  switch (a.dtype) {
    case TW_F32: return norm_bwd_rows<RMS, TW_F32>(a, s);
    case TW_BF16: return norm_bwd_rows<RMS, TW_BF16>(a, s);
    default: return norm_bwd_rows<RMS, TW_F16>(a, s);
  }
}

}  // namespace

}  // namespace tw
