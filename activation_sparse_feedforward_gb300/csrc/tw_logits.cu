// Operators on rows of logits [N, V]: the distillation loss with its gradient, and log
// probabilities of given tokens with the row's entropy and top alternatives.
//
// A row is held on chip. A cluster of 1 to 8 CTAs takes one row, each CTA a slice of it
// in shared memory, copied there by 16-byte asynchronous copies. Every sweep over the
// row after that (its maximum, its sums, the marking of listed tokens, the gradient)
// reads shared memory, so HBM is read once, and a thread reads back only the vectors it
// copied itself, so a sweep needs no barrier. The CTAs' partial statistics are joined
// through distributed shared memory: one launch, no workspace, no atomics on results.
//
// Softmax statistics are a maximum M of z and sums of 2^(c (z - M)), c = log2(e) /
// temperature; two such pairs join as M = max(M1, M2), S = S1 2^(c (M1-M)) + S2 2^(c (M2-M)).
// M is taken off before the scaling: c z alone would overflow, or lose the whole
// exponent to rounding, where a mask is the type's lowest value. A row, slice or thread
// with nothing but -inf has M = -inf and S = 0.
#include <cfloat>

#include <algorithm>

#include "tw_internal.h"
#include "tw_rows.cuh"

namespace tw {

namespace {

constexpr int kMaxThreads = 256;
constexpr int kMaxWarps = kMaxThreads / 32;  // 8, the most CTAs of a cluster too: partial
constexpr int kParts = 8;                    // statistics are joined over eight lanes
static_assert(kMaxWarps <= kParts, "one lane per warp's partial statistics");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

TW_DEV float neg_inf_f() { return __int_as_float(0xFF800000); }
// what to take off z: M, or 0 where there is nothing (so that -inf stays -inf)
TW_DEV float base_of(float M) { return M == neg_inf_f() ? 0.f : M; }
TW_DEV float exp_of(float z, float base, float c) { return exp2_fast((z - base) * c); }

// over groups of W lanes
template <int W = 32>
TW_DEV float warp_max(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
template <int W>
TW_DEV float group_sum(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
TW_DEV f32x2 exp2_pair(f32x2 t) {
  const float2 f = unpair(t);
  return pair(exp2_fast(f.x), exp2_fast(f.y));
}
TW_DEV float add_lanes(f32x2 v) {
  const float2 f = unpair(v);
  return f.x + f.y;
}

// ------------------------------------------------------------------ a CTA's slice of a row
// The row's address may have any element alignment: vectors are counted from the
// 16-byte boundary at or before it, so column c sits in vector (c + lead) / E. A vector
// that reaches outside the row is filled element by element, with -inf outside.
template <int DT>
struct Slice {
  using S = typename Elem<DT>::S;
  static constexpr int E = Elem<DT>::E;
  uint4* buf;
  int lead, V, first, n;  // n vectors from the row's vector `first`

  static TW_DEV int lead_of(const S* row) { return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(S)); }

  TW_DEV Slice(const S* row, int V_, int rank, int cluster, uint4* b) : buf(b), lead(lead_of(row)), V(V_) {
    const int vecs = (V + lead + E - 1) / E;
    const int per = (vecs + cluster - 1) / cluster;
    first = rank * per;
    n = max(0, min(per, vecs - first));
    // the first and the last vector may reach outside the row, all others are whole
    const S* src = row + col(0);
#pragma unroll 4
    for (int j = threadIdx.x; j < n; j += blockDim.x) {
      if ((first + j > 0 || lead == 0) && (first + j + 1 < vecs || (V + lead) % E == 0)) {
        cp_async16(buf + j, src + static_cast<ptrdiff_t>(j) * E);
      } else {
        const int c = col(j);
        S* e = reinterpret_cast<S*>(buf + j);
#pragma unroll
        for (int i = 0; i < E; ++i) e[i] = (c + i >= 0 && c + i < V) ? row[c + i] : Elem<DT>::neg_inf();
      }
    }
    cp_commit();
  }
  // first column of the slice's vector j
  TW_DEV int col(int j) const { return (first + j) * E - lead; }
  // the element of column c, or null when another CTA holds it
  TW_DEV S* at(int c) const {
    const int e = c + lead - first * E;
    return e >= 0 && e < n * E ? reinterpret_cast<S*>(buf) + e : nullptr;
  }
  // the largest of the thread's own vectors
  TW_DEV float own_max() const {
    float m = neg_inf_f();
#pragma unroll 4
    for (int j = threadIdx.x; j < n; j += blockDim.x) m = fmaxf(m, Elem<DT>::max16(buf[j]));
    return m;
  }
};

// ------------------------------------------------------------------ distillation
struct DistillStat {
  float M, rest, list;  // sums at the temperature over the unlisted and the listed tokens
  float s1;             // at temperature 1 over all (TWO only)
};

// Joins one DistillStat per lane over groups of W lanes (M = -inf, sums 0 in unused
// lanes); each lane of a group gets it.
template <bool TWO, int W>
TW_DEV DistillStat join(DistillStat a, float c0) {
  DistillStat r;
  r.M = warp_max<W>(a.M);
  const float base = base_of(r.M), f0 = exp_of(a.M, base, c0);
  r.rest = group_sum<W>(a.rest * f0);
  r.list = group_sum<W>(a.list * f0);
  r.s1 = TWO ? group_sum<W>(a.s1 * exp_of(a.M, base, kLog2e)) : 0.f;
  return r;
}

template <int DT>
TW_DEV float list_value(const void* p, size_t i, int dtype) {
  return dtype == TW_F32 ? static_cast<const float*>(p)[i] : Elem<DT>::get(static_cast<const typename Elem<DT>::S*>(p)[i]);
}
TW_DEV float teacher_logit(const void* p, size_t i, int dtype) {
  return dtype == TW_F16 ? list_value<TW_F16>(p, i, dtype) : list_value<TW_BF16>(p, i, dtype);
}

// One row per cluster. TWO: the hard-label term needs sums of its own (temperature not 1).
template <int DT, bool TWO>
__global__ void __launch_bounds__(kMaxThreads, 3) distill_kernel(const DistillArgs a, int cluster, int slice_bytes) {
  using El = Elem<DT>;
  using S = typename El::S;
  constexpr int E = El::E;
  extern __shared__ uint4 smem[];
  __shared__ float red[2][kMaxWarps];
  __shared__ DistillStat wstat[kMaxWarps], cstat;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
  const int rank = blockIdx.x % cluster;
  const size_t row = blockIdx.x / cluster;
  const int K = a.K;
  // the row's list: token, log2 P, P, z at the token, whether this thread's entry owns it
  int* l_idx = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(smem) + slice_bytes);
  float* l_lp = reinterpret_cast<float*>(l_idx + K);
  float* l_p = l_lp + K;
  float* l_z = l_p + K;
  pdl_enter();

  const S* z = static_cast<const S*>(a.z) + row * a.ldz;
  Slice<DT> sl(z, a.V, rank, cluster, smem);
  const float c0 = kLog2e / a.temperature;

  int label = a.labels != nullptr ? a.labels[row] : -1;
  if (label < -1 || label >= a.V) {
    if (tid == 0) raise_status(a.status, TW_EINVAL);
    label = -1;
  }
  const float z_label = label >= 0 ? El::get(z[label]) : 0.f;

  // the teacher's distribution over its list and the rest
  float tm = neg_inf_f();
  for (int k = tid; k < K; k += nt) {
    int i = a.t_idx[row * K + k];
    if (i < -1 || i >= a.V) {
      raise_status(a.status, TW_EINVAL);
      i = -1;
    }
    float t = i >= 0 ? teacher_logit(a.t_val, row * K + k, a.t_dtype) : neg_inf_f();
    if (t > neg_inf_f()) t = fmaxf(t / a.temperature, -FLT_MAX);  // a finite logit stays one
    l_idx[k] = i;
    l_lp[k] = t;
    l_z[k] = i >= 0 ? El::get(z[i]) : 0.f;
    tm = fmaxf(tm, t);
  }
  const float t_rest = a.t_rest != nullptr ? a.t_rest[row] : neg_inf_f();
  float p_rest = 0.f, lp_rest = neg_inf_f();
  bool some = false;
  if (K > 0 || a.t_rest != nullptr) {
    tm = warp_max(fmaxf(tm, t_rest));
    if (lane == 0) red[0][warp] = tm;
    __syncthreads();
    tm = base_of(warp_max(lane < warps ? red[0][lane] : neg_inf_f()));
    float ts = 0.f;
    for (int k = tid; k < K; k += nt) ts += exp_of(l_lp[k], tm, kLog2e);
    ts = warp_sum(ts);
    if (lane == 0) red[1][warp] = ts;
    __syncthreads();
    ts = warp_sum(lane < warps ? red[1][lane] : 0.f) + exp_of(t_rest, tm, kLog2e);
    some = ts != 0.f;  // NaN counts as some
    if (some) {
      const float inv = 1.f / ts, l2 = log2f(ts);
      for (int k = tid; k < K; k += nt) {
        const float t = (l_lp[k] - tm) * kLog2e;
        l_p[k] = exp2_fast(t) * inv;
        l_lp[k] = t - l2;
      }
      p_rest = exp_of(t_rest, tm, kLog2e) * inv;
      lp_rest = (t_rest - tm) * kLog2e - l2;
    }
  }

  // Listed tokens leave the row: the entry whose number survives in the token's slot
  // owns it (a token listed twice has one owner), and the slot becomes -inf.
  cp_wait<0>();
  __syncthreads();
  bool dup = false;
  if (some) {
    for (int k = tid; k < K; k += nt) {
      S* s = l_idx[k] >= 0 ? sl.at(l_idx[k]) : nullptr;
      if (s != nullptr) *s = static_cast<S>(k);
    }
    __syncthreads();
    for (int k = tid; k < K; k += nt) {
      const S* s = l_idx[k] >= 0 ? sl.at(l_idx[k]) : nullptr;
      const bool owner = s != nullptr && *s == static_cast<S>(k);
      if (s != nullptr && !owner) dup = true;
      if (!owner) l_idx[k] = -2 - l_idx[k];  // not this CTA's, or another entry's: -2 - token (padding: -1)
    }
    dup = __syncthreads_or(dup);
    for (int k = tid; k < K; k += nt)
      if (l_idx[k] >= 0) *sl.at(l_idx[k]) = El::neg_inf();
    __syncthreads();
  }

  // the row's statistics
  DistillStat st;
  {
    float m = sl.own_max();
    if (some)
      for (int k = tid; k < K; k += nt)
        if (l_idx[k] >= 0) m = fmaxf(m, l_z[k]);
    st.M = m;
    st.rest = st.list = st.s1 = 0.f;
    const float b = base_of(m);
    const f32x2 minus = both(-b), k0 = both(c0), k1 = both(kLog2e);
    f32x2 sum0 = both(0.f), sum1 = both(0.f);
#pragma unroll 2
    for (int j = tid; j < sl.n; j += nt) {
      f32x2 v[E / 2];
      El::pairs(sl.buf[j], v);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const f32x2 d = add2(v[e], minus);
        sum0 = add2(sum0, exp2_pair(mul2(d, k0)));
        if (TWO) sum1 = add2(sum1, exp2_pair(mul2(d, k1)));
      }
    }
    st.rest = add_lanes(sum0);
    if (TWO) st.s1 = add_lanes(sum1);
    if (some)
      for (int k = tid; k < K; k += nt)
        if (l_idx[k] >= 0) {
          st.list += exp_of(l_z[k], b, c0);
          if (TWO) st.s1 += exp_of(l_z[k], b, kLog2e);
        }
    st = join<TWO, 32>(st, c0);
    const DistillStat none = {neg_inf_f(), 0.f, 0.f, 0.f};
    if (lane == 0) wstat[warp] = st;
    __syncthreads();
    st = join<TWO, kParts>(lane % kParts < warps ? wstat[lane % kParts] : none, c0);
    if (cluster > 1) {
      if (tid == 0) cstat = st;
      cluster_sync();
      DistillStat p = none;
      if (lane % kParts < cluster) {
        const uint32_t at = peer_smem_addr(&cstat, lane % kParts);
        p.M = ld_cluster_f32(at);
        p.rest = ld_cluster_f32(at + 4);
        p.list = ld_cluster_f32(at + 8);
        p.s1 = ld_cluster_f32(at + 12);
      }
      st = join<TWO, kParts>(p, c0);
      cluster_arrive();  // waited for at the end: no CTA leaves while its cstat is read
    }
  }
  const float total = st.rest + st.list;
  const float b = base_of(st.M);
  const float s1 = TWO ? st.s1 : total;
  const bool nothing = !some && label < 0;  // no target: loss and gradient are 0 whatever the logits

  if (rank == 0 && a.loss != nullptr) {
    float kd = 0.f;
    const float l2 = log2f(total);
    if (some) {
      for (int k = tid; k < K; k += nt) {
        const float p = l_p[k];
        if (p != 0.f && l_idx[k] != -1) kd += p * (l_lp[k] - ((l_z[k] - b) * c0 - l2));
      }
    }
    kd = warp_sum(kd);
    if (lane == 0) red[0][warp] = kd;
    __syncthreads();
    if (tid == 0) {
      kd = 0.f;
      for (int w = 0; w < warps; ++w) kd += red[0][w];
      if (p_rest != 0.f) kd += p_rest * (lp_rest - (log2f(st.rest) - l2));
      float loss = a.kd_weight * a.temperature * a.temperature * kLn2 * kd;
      if (label >= 0) loss += a.ce_weight * kLn2 * (log2f(s1) - (z_label - b) * kLog2e);
      a.loss[row] = nothing ? 0.f : total == 0.f ? __int_as_float(0x7F800000) : loss;
    }
  }

  if (a.dz != nullptr) {
    S* dz = static_cast<S*>(a.dz) + row * a.lddz;
    const bool zero = nothing || total == 0.f;
    const float g = a.scale * (a.dloss != nullptr ? a.dloss[row] : 1.f);
    const float gk = g * a.kd_weight * a.temperature;
    const float gc = label >= 0 ? g * a.ce_weight : 0.f;
    float u = some ? gk / total : 0.f;  // factor of 2^(c0 (z - M)) on unlisted tokens
    if (p_rest != 0.f && st.rest != 0.f) u -= gk * p_rest / st.rest;
    const float w = label >= 0 ? gc / s1 : 0.f;
    if (!TWO) u += w;
    const bool vec = Slice<DT>::lead_of(dz) == sl.lead;
    const f32x2 minus = both(-b), k0 = both(c0), k1 = both(kLog2e), u2 = both(u), w2 = both(w);
#pragma unroll 2
    for (int j = tid; j < sl.n; j += nt) {
      f32x2 v[E / 2];
      El::pairs(sl.buf[j], v);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const f32x2 t = add2(v[e], minus);
        v[e] = mul2(u2, exp2_pair(mul2(t, k0)));
        if (TWO) fma2(v[e], w2, exp2_pair(mul2(t, k1)));
      }
      uint4 out = El::pack_pairs(v);
      if (zero) out = make_uint4(0, 0, 0, 0);
      const int c = sl.col(j);
      if (vec && c >= 0 && c + E <= a.V) {
        *reinterpret_cast<uint4*>(dz + c) = out;
      } else {
        const S* o = reinterpret_cast<const S*>(&out);
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (c + e >= 0 && c + e < a.V) dz[c + e] = o[e];
      }
    }
    __syncthreads();  // the listed tokens and the label overwrite what the sweep stored
    bool label_listed = false;
    if (some && !zero) {
      for (int k = tid; k < K; k += nt) {
        const int i = l_idx[k];
        if (i < 0) continue;
        float p = l_p[k];
        if (dup) {  // add up, in list order, every entry that names the same token
          p = 0.f;
          for (int q = 0; q < K; ++q)
            if (l_idx[q] == i || l_idx[q] == -2 - i) p += l_p[q];
        }
        float d = gk * (exp_of(l_z[k], b, c0) / total - p);
        if (label >= 0) d += w * exp_of(l_z[k], b, kLog2e);
        if (i == label) d -= gc, label_listed = true;
        dz[i] = El::put(d);
      }
    }
    if (a.labels != nullptr) {
      label_listed = __syncthreads_or(label_listed);
      if (tid == 0 && label >= 0 && !label_listed && !zero && sl.at(label) != nullptr) {
        float d = u * exp_of(z_label, b, c0) - gc;
        if (TWO) d = fmaf(w, exp_of(z_label, b, kLog2e), d);
        dz[label] = El::put(d);
      }
    }
  }
  if (cluster > 1) cluster_wait();
}

// ------------------------------------------------------------------ token log probabilities
struct ProbStat {
  float M, s, w;  // s = sum 2^t, w = sum 2^t t, t = c (z - M)
};
template <int W>
TW_DEV ProbStat join(ProbStat a, float c) {
  ProbStat r;
  r.M = warp_max<W>(a.M);
  const float d = (a.M - base_of(r.M)) * c, f = exp2_fast(d);
  r.s = group_sum<W>(a.s * f);
  r.w = group_sum<W>(f * fmaf(a.s, fmaxf(d, -1e30f), a.w));  // the bound keeps 0 (-inf) out
  return r;
}

// fp32 bits in an order of unsigned integers (-0 as 0), and a candidate's key: value
// first, then the lower token. Keys are distinct; 0 is below every key.
TW_DEV uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
TW_DEV float value_of(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o); }
typedef unsigned long long Key;
TW_DEV Key key_of(float v, int token) { return (static_cast<Key>(order_of(v)) << 32) | static_cast<uint32_t>(~token); }

constexpr int kCandidates = 1024;

// top[0..K) = the K largest of cand[0..n), descending, 0 past n. Distinct keys have
// distinct ranks: each thread counts the keys above its own. top is zeroed before.
TW_DEV void rank_select(const Key* cand, int n, Key* top, int K) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const Key k = cand[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += cand[j] > k ? 1 : 0;
    if (k != 0 && r < K) top[r] = k;
  }
}

// A threshold on the upper half of order_of that at least K (or all) of the CTA's n
// values reach, and not many more: a search bit by bit, by one warp.
TW_DEV uint32_t find_threshold(const uint16_t* high, int n, int K) {
  const int lane = threadIdx.x & 31;
  uint32_t h[kMaxThreads / 32];
#pragma unroll
  for (int i = 0; i < kMaxThreads / 32; ++i) h[i] = i * 32 + lane < n ? high[i * 32 + lane] : 0;
  uint32_t thr = 0;
  for (int b = 15; b >= 0; --b) {
    const uint32_t t = thr | (1u << b);
    int c = 0;
#pragma unroll
    for (int i = 0; i < kMaxThreads / 32; ++i) c += h[i] >= t ? 1 : 0;
    c = __reduce_add_sync(0xFFFFFFFFu, c);
    if (c >= K) {
      thr = t;
      if (c <= K + K / 2) break;
    }
  }
  return thr;
}

// The K largest keys of the CTA's slice, descending, into top (0 past the finite ones).
// A threshold that the largest elements of at least K threads reach leaves few
// candidates; a list that overflows (many ties, or the largest elements all with few
// threads) falls back to K sweeps for the next largest key. high: the upper half of the
// order of the thread's largest element, 0 when it has none; thr, count: set by the
// caller behind a barrier.
template <int DT>
TW_DEV void slice_top(const Slice<DT>& sl, uint32_t high, int K, Key* cand, Key* top, uint32_t thr, int* count,
                      Key* wkey) {
  using El = Elem<DT>;
  constexpr int E = El::E;
  const int tid = threadIdx.x, nt = blockDim.x;
  if (high != 0 && high >= thr) {
    for (int j = tid; j < sl.n; j += nt) {
      const uint4 w = sl.buf[j];
      const float m = El::max16(w);
      if (!(m > neg_inf_f()) || (order_of(m) >> 16) < thr) continue;
      float v[E];
      El::unpack(w, v);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (v[e] > neg_inf_f() && (order_of(v[e]) >> 16) >= thr) {
          const int p = atomicAdd(count, 1);
          if (p < kCandidates) cand[p] = key_of(v[e], sl.col(j) + e);
        }
    }
  }
  __syncthreads();
  const int n = *count;
  if (n <= kCandidates) {
    rank_select(cand, n, top, K);
    return;
  }
  Key last = ~0ull;
  for (int r = 0; r < K; ++r) {
    Key best = 0;
    for (int j = tid; j < sl.n; j += nt) {
      float v[E];
      El::unpack(sl.buf[j], v);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const Key k = v[e] > neg_inf_f() ? key_of(v[e], sl.col(j) + e) : 0;
        if (k < last && k > best) best = k;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
    if ((tid & 31) == 0) wkey[tid >> 5] = best;
    __syncthreads();
    best = 0;
    for (int w = 0; w < (nt >> 5); ++w) best = max(best, wkey[w]);
    if (tid == 0) top[r] = best;
    last = best;
    __syncthreads();
    if (best == 0) break;
  }
}

template <int DT>
__global__ void __launch_bounds__(kMaxThreads, 3) logprobs_kernel(const LogprobArgs a, int cluster, int slice_bytes) {
  using El = Elem<DT>;
  using S = typename El::S;
  constexpr int E = El::E;
  extern __shared__ uint4 smem[];
  __shared__ ProbStat wstat[kMaxWarps], cstat;
  __shared__ Key wkey[kMaxWarps];
  __shared__ uint16_t high_of[kMaxThreads];
  __shared__ uint32_t thr;
  __shared__ int count;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
  const int rank = blockIdx.x % cluster;
  const size_t row = blockIdx.x / cluster;
  const int K = a.K;
  Key* cand = reinterpret_cast<Key*>(reinterpret_cast<uint8_t*>(smem) + slice_bytes);
  Key* top = cand + (K > 0 ? kCandidates : 0);
  pdl_enter();

  const S* z = static_cast<const S*>(a.z) + row * a.ldz;
  Slice<DT> sl(z, a.V, rank, cluster, smem);
  const float c = kLog2e / a.temperature;
  cp_wait<0>();

  ProbStat st;
  const float mine = sl.own_max();
  st.M = mine;
  st.s = st.w = 0.f;
  {
    const float b = base_of(mine);
    const f32x2 minus = both(-b), k = both(c);
    f32x2 sum = both(0.f), weighted = both(0.f);
#pragma unroll 2
    for (int j = tid; j < sl.n; j += nt) {
      f32x2 v[E / 2];
      El::pairs(sl.buf[j], v);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const f32x2 t = mul2(add2(v[e], minus), k), p = exp2_pair(t);
        sum = add2(sum, p);
        const float2 f = unpair(t);
        fma2(weighted, p, pair(fmaxf(f.x, -1e30f), fmaxf(f.y, -1e30f)));  // -inf: 0 times a finite number
      }
    }
    st.s = add_lanes(sum);
    st.w = add_lanes(weighted);
  }
  st = join<32>(st, c);
  if (lane == 0) wstat[warp] = st;
  const uint32_t high = mine > neg_inf_f() ? order_of(mine) >> 16 : 0;
  if (K > 0) high_of[tid] = static_cast<uint16_t>(high);
  __syncthreads();
  // warp 0: the slice's statistics, and the threshold of its alternatives
  const ProbStat none = {neg_inf_f(), 0.f, 0.f};
  if (warp == 0) {
    st = join<kParts>(lane % kParts < warps ? wstat[lane % kParts] : none, c);
    if (lane == 0) cstat = st;
    if (K > 0) {
      const uint32_t t = find_threshold(high_of, nt, K);
      if (lane == 0) thr = t, count = 0;
      for (int k = lane; k < K; k += 32) top[k] = 0;
    }
  }
  if (K > 0) {
    __syncthreads();
    slice_top<DT>(sl, high, K, cand, top, thr, &count, wkey);
  }
  if (cluster > 1) {
    cluster_sync();
    if (rank == 0) {
      if (warp == 0) {
        ProbStat p = none;
        if (lane % kParts < cluster) {
          const uint32_t at = peer_smem_addr(&cstat, lane % kParts);
          p.M = ld_cluster_f32(at);
          p.s = ld_cluster_f32(at + 4);
          p.w = ld_cluster_f32(at + 8);
        }
        st = join<kParts>(p, c);
      }
      for (int i = tid; i < cluster * K; i += nt) cand[i] = ld_cluster_u64(peer_smem_addr(top + i % K, i / K));
    }
    cluster_sync();  // every list has been read: the CTAs may leave, rank 0 may overwrite its own
    if (rank != 0) return;
    if (K > 0) {
      for (int k = tid; k < K; k += nt) top[k] = 0;
      __syncthreads();
      rank_select(cand, cluster * K, top, K);
    }
  }
  if (K > 0) __syncthreads();
  if (warp != 0) return;

  const float bm = base_of(st.M), l2 = log2f(st.s);
  const bool empty = st.s == 0.f;  // every logit -inf
  auto logprob = [&](float v) { return empty ? neg_inf_f() : kLn2 * ((v - bm) * c - l2); };
  for (int i = lane; i < a.n_tokens; i += 32) {
    const int t = a.tokens[row * a.n_tokens + i];
    float lp = 0.f;
    if (t >= 0 && t < a.V)
      lp = logprob(El::get(z[t]));
    else if (t != -1)
      raise_status(a.status, TW_EINVAL);
    a.logprob[row * a.n_tokens + i] = lp;
  }
  if (tid == 0 && a.entropy != nullptr) a.entropy[row] = empty ? 0.f : kLn2 * (l2 - st.w / st.s);
  const bool bad = !(st.s < __int_as_float(0x7F800000));  // a NaN or an infinity in the row
  for (int k = lane; k < K; k += 32) {
    const Key key = top[k];
    a.top_idx[row * K + k] = key == 0 || bad ? -1 : static_cast<int>(~static_cast<uint32_t>(key));
    a.top_logprob[row * K + k] = bad ? __int_as_float(0x7FC00000) : key == 0 ? neg_inf_f() : logprob(value_of(key >> 32));
  }
}

// ------------------------------------------------------------------ launch shapes
struct RowShape {
  int cluster, threads, slice_bytes;
};

// A slice of at most 64 KB keeps three CTAs on an SM, so that one's copies run under
// the others' sweeps. Fewer rows than SMs: more CTAs a row, down to 8 KB each.
RowShape row_shape(int64_t N, int V, int dtype, int top_k) {
  const int E = dtype == TW_F32 ? 4 : 8;
  const int vecs = (V + 2 * E - 2) / E;  // at any alignment
  RowShape r;
  r.cluster = 1;
  auto bytes = [&] { return 16 * ((vecs + r.cluster - 1) / r.cluster); };
  while (r.cluster < 8 && bytes() > 64 * 1024) r.cluster *= 2;
  while (r.cluster < 8 && N * r.cluster * 2 <= device_sm_count() && bytes() > 8 * 1024) r.cluster *= 2;
  r.slice_bytes = bytes();
  // eight vectors a thread; two threads an alternative, so that a threshold which top_k
  // threads reach is passed by few elements
  r.threads = std::max({64, (r.slice_bytes / 16 / 8 + 31) / 32 * 32, 2 * ((top_k + 31) / 32 * 32)});
  r.threads = std::min(r.threads, kMaxThreads);
  return r;
}

template <class Kern, class Args>
cudaError_t launch_rows(Kern kern, const Args& a, const RowShape& r, size_t smem, const char* label, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.N) * r.cluster), block(r.threads);
  e = r.cluster == 1 ? launch(kern, grid, block, smem, s, a, r.cluster, r.slice_bytes)
                     : launch_clustered(kern, grid, block, smem, r.cluster, s, a, r.cluster, r.slice_bytes);
  trace_mark(s, label);
  return e;
}

template <int DT>
cudaError_t distill(const DistillArgs& a, cudaStream_t s) {
  const RowShape r = row_shape(a.N, a.V, DT, 0);
  const size_t smem = r.slice_bytes + 16 * static_cast<size_t>(a.K);
  return a.labels != nullptr && a.temperature != 1.f ? launch_rows(distill_kernel<DT, true>, a, r, smem, "distill", s)
                                                     : launch_rows(distill_kernel<DT, false>, a, r, smem, "distill", s);
}

template <int DT>
cudaError_t logprobs(const LogprobArgs& a, cudaStream_t s) {
  const RowShape r = row_shape(a.N, a.V, DT, a.K);
  const size_t smem = r.slice_bytes + (a.K > 0 ? sizeof(Key) * static_cast<size_t>(kCandidates + a.K) : 0);
  return launch_rows(logprobs_kernel<DT>, a, r, smem, "token_logprobs", s);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t s) {
  if (a.N == 0) return cudaSuccess;
  return a.dtype == TW_F32 ? distill<TW_F32>(a, s) : a.dtype == TW_BF16 ? distill<TW_BF16>(a, s) : distill<TW_F16>(a, s);
}

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t s) {
  if (a.N == 0) return cudaSuccess;
  return a.dtype == TW_F32 ? logprobs<TW_F32>(a, s) : a.dtype == TW_BF16 ? logprobs<TW_BF16>(a, s) : logprobs<TW_F16>(a, s);
}

}  // namespace tw
