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

// Threads of every CTA here: a constant, so that a thread's vectors lie at constant
// distances (a run-time count cost an integer instruction or two an element).
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kParts = 8;  // per-warp or per-CTA statistics of the log probabilities, joined over eight lanes
static_assert(kWarps <= kParts && kMaxCluster <= kParts, "one lane per part");
static_assert(kWarps * kMaxCluster <= 64, "two lanes' worth of per-warp statistics in a cluster");
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

TW_DEV float2 exp2_pair(float2 t) { return make_float2(exp2_fast(t.x), exp2_fast(t.y)); }
TW_DEV float add_lanes(float2 v) { return v.x + v.y; }
// v^POW, POW 2 or 4
template <int POW>
TW_DEV float2 power(float2 v) {
  const float2 q = mul2(v, v);
  return POW == 4 ? mul2(q, q) : q;
}

// ------------------------------------------------------------------ a CTA's part of a row
// The row's address may have any element alignment: vectors are counted from the
// 16-byte boundary at or before it, so column c sits in vector (c + lead) / E. Only the
// row's first and last vector may reach outside it; those are read element by element,
// with -inf outside.
template <int DT>
struct Part {
  using S = typename Elem<DT>::S;
  static constexpr int E = Elem<DT>::E;
  const S* row;
  int lead, V, first, n;  // n vectors from the row's vector `first`
  int lo, hi;             // those of them that are whole: [lo, hi)

  static TW_DEV int lead_of(const S* row) { return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(S)); }

  TW_DEV Part(const S* row_, int V_, int rank, int cluster) : row(row_), lead(lead_of(row_)), V(V_) {
    const int vecs = (V + lead + E - 1) / E;
    const int per = (vecs + cluster - 1) / cluster;
    first = rank * per;
    n = max(0, min(per, vecs - first));
    lo = first == 0 && lead > 0 ? 1 : 0;
    hi = min(n, (V + lead) / E - first);
  }
  // first column of the part's vector j
  TW_DEV int col(int j) const { return (first + j) * E - lead; }
  TW_DEV bool whole(int j) const { return j >= lo && j < hi; }
  TW_DEV const S* at(int j) const { return row + col(j); }
  TW_DEV uint4 edge(int j) const {
    union {
      S e[E];
      uint4 w;
    } u;
    const int c = col(j);
#pragma unroll
    for (int i = 0; i < E; ++i) u.e[i] = (c + i >= 0 && c + i < V) ? row[c + i] : Elem<DT>::neg_inf();
    return u.w;
  }
};

// The same part copied to shared memory: a thread copies, and then sweeps, the whole
// vectors lo + threadIdx.x, lo + threadIdx.x + kThreads, ...; the edges are the CTA's
// first and last thread's.
template <int DT>
struct Slice : Part<DT> {
  using P = Part<DT>;
  using typename P::S;
  using P::E;
  uint4* buf;

  TW_DEV Slice(const S* row, int V, int rank, int cluster, uint4* b) : P(row, V, rank, cluster), buf(b) {
      uint4* dst = buf + this->lo + threadIdx.x;
    const uint4* src = reinterpret_cast<const uint4*>(P::at(this->lo)) + threadIdx.x;
    int j = this->lo + threadIdx.x;
#pragma unroll 4
    for (; j < this->hi; j += kThreads, dst += kThreads, src += kThreads) cp_async16(dst, src);
    if (first_edge()) buf[0] = P::edge(0);
    if (last_edge()) buf[this->n - 1] = P::edge(this->n - 1);
    cp_commit();
  }
  // whether this thread holds the slice's first (last) vector as one that is not whole
  TW_DEV bool first_edge() const { return threadIdx.x == 0 && this->lo > 0; }
  TW_DEV bool last_edge() const { return threadIdx.x == kThreads - 1 && this->hi < this->n && this->n > this->lo; }
  // the element of column c, or null when another CTA holds it
  TW_DEV S* element(int c) const {
    const int e = c + this->lead - this->first * E;
    return e >= 0 && e < this->n * E ? reinterpret_cast<S*>(buf) + e : nullptr;
  }
};

// ------------------------------------------------------------------ exponentials of a sweep
// A sweep takes 2^(c (z - m)) of many z for one m. Where c m is of ordinary size that is
// one fused multiply-add and one exponential, 2^(c z - k) with k = c m rounded, and the
// sweep's sums are corrected once by 2^(k - c m), whose exponent the fused operation
// gives exactly. Past 2^20 the rounding of k would leave more than a fraction of the
// exponent (a mask of the type's lowest value ends there), and m is taken off z first.
struct Scale {
  float m, c, k;
  bool fused;
  TW_DEV Scale(float max, float c_) : m(base_of(max)), c(c_), k(m * c_) { fused = fabsf(k) < 1048576.f; }
  TW_DEV float shift() const { return fused ? -fmaf(m, c, -k) : 0.f; }  // k - c m
  // what the exponent c z - k grows by when `to` is used in place of this one
  TW_DEV float move(const Scale& to) const { return fmaf(m - to.m, c, shift() - to.shift()); }
  template <bool FUSED>
  TW_DEV float2 exponent(float2 z) const {
    if (FUSED) return fma2(z, both(c), both(-k));
    return mul2(add2(z, both(-m)), both(c));
  }
};

constexpr int kBatch = 4;  // vectors a thread takes at a time

// f(j, all) for the thread's vectors j, j + kThreads, ... of [lo, hi) in batches of
// kBatch; all: a constant, whether the whole batch is below hi.
struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };
template <class F>
TW_DEV void in_batches(int lo, int hi, F f) {
  int j = lo + threadIdx.x;
  for (; j + (kBatch - 1) * kThreads < hi; j += kBatch * kThreads) f(j, Yes());
  if (j < hi) f(j, No());
}

// A thread's online sums over its vectors, in batches. The reference m follows the
// running maximum, but only when that is more than kSlack above it (in nats at
// temperature 1): sums are rescaled a few times a row, and no term exceeds e^kSlack.
constexpr float kSlack = 8.f;

template <int DT>
struct Running {
  typename Elem<DT>::Max top;
  float limit = -__builtin_huge_valf();
  // Takes a batch into the maximum; true when the reference has to
  // move to it.
  TW_DEV bool grow(const uint4 (&r)[kBatch], float slack) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top.add(r[i]);
    const float m = top.get();
    if (!(m > limit)) return false;
    limit = m + slack;
    return true;
  }
};
// a batch of nothing but -inf
template <int DT>
TW_DEV uint4 no_vector() {
  constexpr uint32_t v = DT == TW_F32 ? 0xFF800000u : DT == TW_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
  return make_uint4(v, v, v, v);
}

// ------------------------------------------------------------------ distillation
// The hard-label term wants sums of e^z at temperature 1. How a kernel gets them beside
// the sums of p = e^(z / temperature): HARD = kNoSum where there are no labels or the
// temperature is 1; 2 or 4 where the temperature is that: p^2 or p^4, products in place
// of a second exponential an element in each sweep (4096 x 131072 bf16 at temperature 2:
// the exponentials alone would keep their unit busy for three quarters of the floor);
// kOwnSum at any other temperature.
constexpr int kNoSum = 0, kOwnSum = 1;

struct DistillStat {
  float M, rest, list;  // sums at the temperature over the unlisted and the listed tokens
  float s1;             // at temperature 1 over all (not with kNoSum)
};

// The scale at temperature 1 beside `a` at the temperature. (c is log2(e) / HARD, an
// exact division, so HARD times c, k and the shift are exact too.)
template <int HARD>
TW_DEV Scale hard_scale(const Scale& a) {
  Scale b(a.m, kLog2e);
  if (HARD == 2 || HARD == 4) b.k = HARD * a.k, b.fused = a.fused;
  return b;
}


// Joins one DistillStat per lane (M = -inf, sums 0 in unused lanes); all lanes get it.
template <int HARD>
TW_DEV DistillStat join(DistillStat a, float c0) {
  DistillStat r;
  r.M = warp_max(a.M);
  const float base = base_of(r.M), f0 = exp_of(a.M, base, c0);
  r.rest = warp_sum(a.rest * f0);
  r.list = warp_sum(a.list * f0);
  r.s1 = HARD != kNoSum ? warp_sum(a.s1 * exp_of(a.M, base, kLog2e)) : 0.f;
  return r;
}
template <int HARD>
TW_DEV DistillStat join_two(DistillStat a, DistillStat b, float c0) {
  DistillStat r;
  r.M = fmaxf(a.M, b.M);
  const float base = base_of(r.M), fa = exp_of(a.M, base, c0), fb = exp_of(b.M, base, c0);
  r.rest = a.rest * fa + b.rest * fb;
  r.list = a.list * fa + b.list * fb;
  r.s1 = HARD != kNoSum ? a.s1 * exp_of(a.M, base, kLog2e) + b.s1 * exp_of(b.M, base, kLog2e) : 0.f;
  return r;
}

// The thread's own vectors of the slice in one sweep: their largest element m, and the
// sums of their exponentials relative to it at the scales c0 and log2(e).
template <int DT, int HARD, bool FUSED>
TW_DEV void add_exps(const uint4 (&r)[kBatch], const Scale& a, const Scale& b, float2& s0, float2& s1) {
  using El = Elem<DT>;
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    float2 v[El::E / 2];
    El::pairs(r[i], v);
#pragma unroll
    for (int e = 0; e < El::E / 2; ++e) {
      const float2 p = exp2_pair(a.exponent<FUSED>(v[e]));
      s0 = add2(s0, p);
      if (HARD == kOwnSum) s1 = add2(s1, exp2_pair(b.exponent<FUSED>(v[e])));
      if (HARD == 2) s1 = fma2(p, p, s1);
      if (HARD == 4) {
        const float2 q = mul2(p, p);
        s1 = fma2(q, q, s1);
      }
    }
  }
}
template <int DT, int HARD>
TW_DEV void own_sums(const Slice<DT>& sl, float c0, float& m, float& sum0, float& sum1) {
  Running<DT> run;
  const float slack = kSlack * fminf(1.f, kLog2e / c0);
  float2 s0 = both(0.f), s1 = both(0.f);
  Scale a(neg_inf_f(), c0), b(neg_inf_f(), kLog2e);
  bool fused = true, some = false;
  auto batch = [&](const uint4 (&r)[kBatch]) {
    if (run.grow(r, slack)) {
      Scale a2(run.top.get(), c0), b2 = hard_scale<HARD>(a2);
      a2.fused = b2.fused = fused = a2.fused && b2.fused;
      s0 = some ? mul2(s0, both(exp2_fast(a.move(a2)))) : both(0.f);
      if (HARD != kNoSum) s1 = some ? mul2(s1, both(exp2_fast(b.move(b2)))) : both(0.f);
      a = a2, b = b2, some = true;
    }
    if (fused)
      add_exps<DT, HARD, true>(r, a, b, s0, s1);
    else
      add_exps<DT, HARD, false>(r, a, b, s0, s1);
  };
  in_batches(sl.lo, sl.hi, [&](int j, auto all) {
    uint4 r[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) r[i] = all.value || j + i * kThreads < sl.hi ? sl.buf[j + i * kThreads] : no_vector<DT>();
    batch(r);
  });
  if (sl.first_edge() || sl.last_edge()) {
    const uint4 r[kBatch] = {sl.first_edge() ? sl.buf[0] : no_vector<DT>(), sl.last_edge() ? sl.buf[sl.n - 1] : no_vector<DT>(),
                             no_vector<DT>(), no_vector<DT>()};
    batch(r);
  }
  m = run.top.get();
  const float base = base_of(m);
  sum0 = add_lanes(s0) * exp2_fast(fmaf(a.m - base, c0, a.shift()));
  sum1 = HARD != kNoSum ? add_lanes(s1) * exp2_fast(fmaf(b.m - base, kLog2e, b.shift())) : 0.f;
}

template <int DT>
TW_DEV float value_at(const void* p, size_t i) {
  return Elem<DT>::get(static_cast<const typename Elem<DT>::S*>(p)[i]);
}
TW_DEV float teacher_logit(const DistillArgs& a, size_t e) {
  return a.t_dtype == TW_F32 ? value_at<TW_F32>(a.t_val, e) : a.t_dtype == TW_BF16 ? value_at<TW_BF16>(a.t_val, e)
                                                                                  : value_at<TW_F16>(a.t_val, e);
}

// What a row is to learn, beside its list.
struct Target {
  bool some;              // the teacher has mass
  float p_rest, lp_rest;  // P and log2 P of the rest
  int label;
  float up;               // the upstream gradient
};

// The rare part of the marking, by the whole CTA: entries that found -inf at their token.
// The lowest of those whose token no other entry took owns it (its logit is masked);
// the others learn the logit from the owner.
template <int DT>
TW_DEV void owners(const Slice<DT>& sl, int K, int* l_idx, float* l_z, int label, int* label_entry) {
  __syncthreads();
  uint32_t owns = 0;  // a bit for each of the thread's entries: at most 1024 / 64
  int n = 0;
  for (int k = threadIdx.x; k < K; k += kThreads, ++n) {
    const int i = -2 - l_idx[k];
    bool own = i >= 0 && sl.element(i) != nullptr;
    for (int q = 0; own && q < K; ++q) {
      if (l_idx[q] == i) l_z[k] = l_z[q], own = false;
      if (q < k && l_idx[q] == -2 - i) own = false;
    }
    owns |= own ? 1u << n : 0u;
  }
  __syncthreads();
  n = 0;
  for (int k = threadIdx.x; k < K; k += kThreads, ++n)
    if (owns >> n & 1u) {
      l_idx[k] = -2 - l_idx[k];
      if (l_idx[k] == label) *label_entry = k;
    }
  __syncthreads();
}

// u 2^(c0 (z - M)) (+ w 2^(log2(e) (z - M))) of one vector
template <int DT, int HARD, bool FUSED>
TW_DEV uint4 gradient(const uint4& r, const Scale& a, const Scale& b, float u, float w) {
  using El = Elem<DT>;
  float2 v[El::E / 2];
  El::pairs(r, v);
#pragma unroll
  for (int e = 0; e < El::E / 2; ++e) {
    const float2 z = v[e], p = exp2_pair(a.exponent<FUSED>(z));
    v[e] = mul2(both(u), p);
    if (HARD == kOwnSum) v[e] = fma2(both(w), exp2_pair(b.exponent<FUSED>(z)), v[e]);
    if (HARD == 2 || HARD == 4) v[e] = fma2(both(w), power<HARD>(p), v[e]);
  }
  return El::pack_pairs(v);
}
// f of each of the thread's vectors, stored at its columns of dz.
template <int DT, class F>
TW_DEV void store_slice(const Slice<DT>& sl, typename Elem<DT>::S* dz, F f) {
  using S = typename Elem<DT>::S;
  constexpr int E = Elem<DT>::E;
  auto singly = [&](int j) {
    const uint4 g = f(sl.buf[j]);
    const S* o = reinterpret_cast<const S*>(&g);
    const int c = sl.col(j);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (c + e >= 0 && c + e < sl.V) dz[c + e] = o[e];
  };
  if (Part<DT>::lead_of(dz) == sl.lead) {  // the same alignment as z's row
    uint4* out = reinterpret_cast<uint4*>(dz + sl.col(0));
    in_batches(sl.lo, sl.hi, [&](int j, auto all) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (all.value || j + i * kThreads < sl.hi) out[j + i * kThreads] = f(sl.buf[j + i * kThreads]);
    });
  } else {
    for (int j = sl.lo + threadIdx.x; j < sl.hi; j += kThreads) singly(j);
  }
  if (sl.first_edge()) singly(0);
  if (sl.last_edge()) singly(sl.n - 1);
}

// One row per cluster. What the CTAs tell each other is pushed into the receiver's shared
// memory before a cluster barrier: every warp's statistics to every CTA, every warp's
// share of the loss to rank 0.
template <int DT, int HARD>
__global__ void __launch_bounds__(kThreads, 3) distill_kernel(const DistillArgs a, int cluster, int slice_bytes, int ahead) {
  using El = Elem<DT>;
  using S = typename El::S;
  extern __shared__ uint4 smem[];
  __shared__ float4 stats[kMaxCluster * kWarps];
  __shared__ float shares[kMaxCluster * kWarps];
  __shared__ Target target;
  __shared__ int label_entry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster;
  const size_t row = blockIdx.x / cluster;
  const int K = a.K;
  // the row's list: the token (after the marking -2 - token where the entry does not own
  // its place in this CTA's slice), log2 P, P, and z at the token (until the marking: the
  // teacher's logit)
  int* l_idx = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(smem) + slice_bytes);
  float* l_lp = reinterpret_cast<float*>(l_idx + K);
  float* l_p = l_lp + K;
  float* l_z = l_p + K;
  pdl_enter();
  if (cluster > 1) cluster_arrive_relaxed();  // waited for before the first push: every CTA has started

  // Warp 0 takes the row's target while the slice is on its way: its loads go before the
  // slice's, and the other warps keep out of its way (all of them taking it for
  // themselves cost 1 us a row in issue slots).
  const float c0 = kLog2e / a.temperature;
  const size_t list = row * K;
  const S* z = static_cast<const S*>(a.z) + row * a.ldz;
  int label = -1, i_first = -1;
  float t_rest = neg_inf_f(), up = 1.f, t_first = neg_inf_f();
  if (warp == 0) {
    if (a.labels != nullptr) label = a.labels[row];
    if (a.t_rest != nullptr) t_rest = a.t_rest[row];
    if (a.dloss != nullptr) up = a.dloss[row];
    if (lane < K) i_first = a.t_idx[list + lane], t_first = teacher_logit(a, list + lane);
  }
  Slice<DT> sl(z, a.V, rank, cluster, smem);
  if (warp == 0) {
    if (label < -1 || label >= a.V) {
      if (lane == 0) raise_status(a.status, TW_EINVAL);
      label = -1;
    }
    float tm = t_rest;
    for (int k = lane; k < K; k += 32) {
      int i = k == lane ? i_first : a.t_idx[list + k];
      float t = k == lane ? t_first : teacher_logit(a, list + k);
      if (i < 0 || i >= a.V) {
        if (i != -1) raise_status(a.status, TW_EINVAL);
        i = -1;
        t = neg_inf_f();
      }
      if (t > neg_inf_f()) t = fmaxf(t / a.temperature, -FLT_MAX);  // a finite logit stays one
      l_idx[k] = i;
      l_z[k] = t;
      tm = fmaxf(tm, t);
    }
    tm = base_of(warp_max(tm));
    float ts = 0.f;
    for (int k = lane; k < K; k += 32) {
      const float e = exp_of(l_z[k], tm, kLog2e);
      l_p[k] = e;
      ts += e;
    }
    const float e_rest = exp_of(t_rest, tm, kLog2e);
    ts = warp_sum(ts) + e_rest;
    const float inv = 1.f / ts, l2 = log2f(ts);
    for (int k = lane; k < K; k += 32) {
      l_p[k] *= inv;
      l_lp[k] = (l_z[k] - tm) * kLog2e - l2;
    }
    if (lane == 0) {
      target.some = ts != 0.f;  // NaN counts as some
      target.p_rest = target.some ? e_rest * inv : 0.f;
      target.lp_rest = (t_rest - tm) * kLog2e - l2;
      target.label = label;
      target.up = up * a.scale;
      label_entry = -1;
    }
  }
  // the lists of a row that a later CTA takes: cold, their loads were the longest step
  // before the sums
  if (rank == 0 && warp == kWarps - 1 && row + ahead < static_cast<size_t>(a.N)) {
    const size_t e = (row + ahead) * K;
    const int size = a.t_dtype == TW_F32 ? 4 : 2;
    for (int k = lane * 32; k < K; k += 32 * 32) {
      prefetch_line(a.t_idx + e + k);
      prefetch_line(static_cast<const uint8_t*>(a.t_val) + (e + k) * size);
    }
    if (lane == 0 && a.t_rest != nullptr) prefetch_line(a.t_rest + row + ahead);
    if (lane == 0 && a.labels != nullptr) prefetch_line(a.labels + row + ahead);
    if (lane == 0 && a.dloss != nullptr) prefetch_line(a.dloss + row + ahead);
  }

  // Listed tokens leave the row: an entry takes the token's logit and puts -inf in its
  // place. Whoever finds -inf there comes second (a token listed twice), or the logit was
  // masked: owners() sorts that out.
  cp_wait<0>();
  __syncthreads();
  label = target.label;
  const bool some = target.some;
  bool dup = false;
  if (some) {
    for (int k = tid; k < K; k += kThreads) {
      const int i = l_idx[k];
      S* s = i >= 0 ? sl.element(i) : nullptr;
      const float v = s != nullptr ? El::get(El::exchange(s, El::neg_inf())) : 0.f;
      l_z[k] = v;
      const bool owner = s != nullptr && v != neg_inf_f();
      if (s != nullptr && !owner) dup = true;
      if (!owner) l_idx[k] = -2 - i;  // padding: -1
      if (owner && i == label) label_entry = k;
    }
    dup = __syncthreads_or(dup);
    if (dup) owners(sl, K, l_idx, l_z, label, &label_entry);
  }

  // the row's statistics
  DistillStat st;
  {
    float m;
    own_sums<DT, HARD>(sl, c0, m, st.rest, st.s1);
    if (some) {  // the list's tokens that this thread owns join its maximum
      const float was = m;
      for (int k = tid; k < K; k += kThreads)
        if (l_idx[k] >= 0) m = fmaxf(m, l_z[k]);
      if (m != was) {
        st.rest *= exp_of(was, base_of(m), c0);
        if (HARD != kNoSum) st.s1 *= exp_of(was, base_of(m), kLog2e);
      }
    }
    st.M = m;
    st.list = 0.f;
    const float b = base_of(m);
    if (some)
      for (int k = tid; k < K; k += kThreads)
        if (l_idx[k] >= 0) {
          st.list += exp_of(l_z[k], b, c0);
          if (HARD != kNoSum) st.s1 += exp_of(l_z[k], b, kLog2e);
        }
    st = join<HARD>(st, c0);
    const float4 mine = make_float4(st.M, st.rest, st.list, st.s1);
    if (cluster > 1) {
      cluster_wait();
      if (lane < cluster) st_cluster_v4(peer_smem_addr(&stats[rank * kWarps + warp], lane), mine);
      cluster_barrier();
    } else {
      if (lane == 0) stats[warp] = mine;
      __syncthreads();
    }
    const DistillStat none = {neg_inf_f(), 0.f, 0.f, 0.f};
    const int parts = cluster * kWarps;
    auto part = [&](int i) {
      if (i >= parts) return none;
      const float4 s = stats[i];
      return DistillStat{s.x, s.y, s.z, s.w};
    };
    st = part(lane);
    if (parts > 32) st = join_two<HARD>(st, part(lane + 32), c0);
    st = join<HARD>(st, c0);
  }
  const float total = st.rest + st.list;
  const float b = base_of(st.M);
  const float s1 = HARD != kNoSum ? st.s1 : total;
  const bool nothing = !some && label < 0;  // no target: loss and gradient are 0 whatever the logits
  const bool holds_label = label >= 0 && sl.element(label) != nullptr;
  const float z_label = !holds_label ? 0.f : label_entry >= 0 ? l_z[label_entry] : El::get(*sl.element(label));

  // the loss, in units of log2: each entry's term by the thread that found it in its slice
  if (a.loss != nullptr) {
    float share = 0.f;
    if (some) {
      const float l2 = log2f(total), f = a.kd_weight * a.temperature * a.temperature;
      for (int k = tid; k < K; k += kThreads) {
        const int i = l_idx[k] >= 0 ? l_idx[k] : -2 - l_idx[k];
        const float p = l_p[k];
        if (i >= 0 && sl.element(i) != nullptr && p != 0.f) share += p * (l_lp[k] - ((l_z[k] - b) * c0 - l2));
      }
      if (rank == 0 && tid == 0 && target.p_rest != 0.f) share += target.p_rest * (target.lp_rest - (log2f(st.rest) - l2));
      share *= f;
    }
    if (holds_label && tid == 0) share += a.ce_weight * (log2f(s1) - (z_label - b) * kLog2e);
    share = warp_sum(share);
    if (lane == 0) {
      if (cluster > 1)
        st_cluster_f32(peer_smem_addr(&shares[rank * kWarps + warp], 0), share);
      else
        shares[warp] = share;
    }
  }
  if (cluster > 1) cluster_arrive();  // waited for at the end

  if (a.dz != nullptr) {
    S* dz = static_cast<S*>(a.dz) + row * a.lddz;
    const bool zero = nothing || total == 0.f;
    const float gk = target.up * a.kd_weight * a.temperature;
    const float gc = label >= 0 ? target.up * a.ce_weight : 0.f;
    float u = some ? gk / total : 0.f;  // factor of 2^(c0 (z - M)) on unlisted tokens
    if (target.p_rest != 0.f && st.rest != 0.f) u -= gk * target.p_rest / st.rest;
    const float w = label >= 0 ? gc / s1 : 0.f;
    if (HARD == kNoSum) u += w;
    Scale sa(st.M, c0), sb = hard_scale<HARD>(sa);
    const bool fused = sa.fused && sb.fused;
    const float uf = fused ? u * exp2_fast(sa.shift()) : u, wf = fused ? w * exp2_fast(sb.shift()) : w;
    if (zero)
      store_slice<DT>(sl, dz, [](const uint4&) { return make_uint4(0, 0, 0, 0); });
    else if (fused)
      store_slice<DT>(sl, dz, [&](const uint4& r) { return gradient<DT, HARD, true>(r, sa, sb, uf, wf); });
    else
      store_slice<DT>(sl, dz, [&](const uint4& r) { return gradient<DT, HARD, false>(r, sa, sb, uf, wf); });
    __syncthreads();  // the listed tokens and the label overwrite what the sweep stored
    if (some && !zero) {
      for (int k = tid; k < K; k += kThreads) {
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
        if (i == label) d -= gc;
        dz[i] = El::put(d);
      }
    }
    if (tid == 0 && holds_label && label_entry < 0 && !zero) {
      float d = u * exp_of(z_label, b, c0) - gc;
      if (HARD != kNoSum) d = fmaf(w, exp_of(z_label, b, kLog2e), d);
      dz[label] = El::put(d);
    }
  }

  if (cluster > 1)
    cluster_wait();
  else if (a.dz == nullptr)
    __syncthreads();
  if (rank == 0 && warp == 0 && a.loss != nullptr) {
    const int parts = cluster * kWarps;
    float loss = (lane < parts ? shares[lane] : 0.f) + (lane + 32 < parts ? shares[lane + 32] : 0.f);
    loss = kLn2 * warp_sum(loss);
    if (lane == 0) a.loss[row] = nothing ? 0.f : total == 0.f ? __int_as_float(0x7F800000) : loss;
  }
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

constexpr int kCandidates = 1024, kMaxAlternatives = 128;
static_assert(kMaxAlternatives * kMaxCluster <= kCandidates, "a cluster's lists fit");

// top[0..K) = the K largest of cand[0..n), descending, 0 past n. Distinct keys have
// distinct ranks: each thread counts the keys above its own. top is zeroed before; cand
// has room for one more.
TW_DEV void rank_select(Key* cand, int n, Key* top, int K) {
  const ulonglong2* two = reinterpret_cast<const ulonglong2*>(cand);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Key k = cand[i];
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < n / 2; ++j) {
      const ulonglong2 c = two[j];
      r += (c.x > k ? 1 : 0) + (c.y > k ? 1 : 0);
    }
    if (n & 1) r += cand[n - 1] > k ? 1 : 0;
    if (k != 0 && r < K) top[r] = k;
  }
}

// A threshold that at least K of the CTA's values (below 2^16; one a thread) reach, and
// not many more: bit by bit from the highest, a barrier that counts each. 0 where fewer
// than K are not 0.
TW_DEV uint32_t find_threshold(uint32_t v, int K) {
  uint32_t thr = 0;
  for (int b = 15; b >= 0; --b) {
    const uint32_t t = thr | 1u << b;
    const int c = __syncthreads_count(v >= t);
    if (c >= K) {
      thr = t;
      if (c <= K + K / 2 + 2) break;
    }
  }
  return thr;
}

// f(vector, index) for each of the thread's whole vectors, and for the edges, which the
// CTA's first and last thread take.
template <int DT, class F>
TW_DEV void each_vector(const Part<DT>& p, F f) {
#pragma unroll 4
  for (int j = p.lo + threadIdx.x; j < p.hi; j += kThreads) f(*reinterpret_cast<const uint4*>(p.at(j)), j);
  if (threadIdx.x == 0 && p.lo > 0) f(p.edge(0), 0);
  if (threadIdx.x == kThreads - 1 && p.hi < p.n && p.n > p.lo) f(p.edge(p.n - 1), p.n - 1);
}

// The K largest keys of the CTA's part, descending, into top (0 past the finite ones).
// A threshold that the largest elements of at least K threads reach leaves few
// candidates, all in those threads' vectors. The whole CTA reads these once more (from
// L2), a vector a thread: left to their owners, one lane of a warp would walk a row's
// worth of latencies. A list that overflows (many ties, or the largest elements all with
// few threads) falls back to K sweeps for the next largest key. high: the upper half of
// the order of the thread's largest element, 0 when it has none; count (two zeros) and top
// (zeros): set by the caller behind a barrier; above: room for a thread number each.
template <int DT>
TW_DEV void part_top(const Part<DT>& p, uint32_t high, int K, Key* cand, Key* top, uint32_t thr, int* count,
                     uint16_t* above, Key* wkey) {
  using El = Elem<DT>;
  constexpr int E = El::E;
  const int tid = threadIdx.x;
  auto collect = [&](const uint4& w, int j) {
    const float m = El::max16(w);
    if (!(m > neg_inf_f()) || (order_of(m) >> 16) < thr) return;
    float v[E];
    El::unpack(w, v);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (v[e] > neg_inf_f() && (order_of(v[e]) >> 16) >= thr) {
        const int at = atomicAdd(count, 1);
        if (at < kCandidates) cand[at] = key_of(v[e], p.col(j) + e);
      }
  };
  if (high != 0 && high >= thr) above[atomicAdd(count + 1, 1)] = static_cast<uint16_t>(tid);
  if (tid == 0 && p.lo > 0) collect(p.edge(0), 0);
  if (tid == kThreads - 1 && p.hi < p.n && p.n > p.lo) collect(p.edge(p.n - 1), p.n - 1);
  __syncthreads();
  const int rounds = (p.hi - p.lo + kThreads - 1) / kThreads, work = count[1] * rounds;
  for (int i = tid; i < work; i += kThreads) {
    const int j = p.lo + above[i / rounds] + (i % rounds) * kThreads;
    if (j < p.hi) collect(*reinterpret_cast<const uint4*>(p.at(j)), j);
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
    each_vector(p, [&](const uint4& w, int j) {
      float v[E];
      El::unpack(w, v);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const Key k = v[e] > neg_inf_f() ? key_of(v[e], p.col(j) + e) : 0;
        if (k < last && k > best) best = k;
      }
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
    if ((tid & 31) == 0) wkey[tid >> 5] = best;
    __syncthreads();
    best = 0;
    for (int w = 0; w < kWarps; ++w) best = max(best, wkey[w]);
    if (tid == 0) top[r] = best;
    last = best;
    __syncthreads();
    if (best == 0) break;
  }
}

// One vector's share of the sums s = sum 2^t and w = sum 2^t t.
template <int DT, bool FUSED>
TW_DEV void add_terms(const uint4& r, const Scale& a, float2& s, float2& w) {
  using El = Elem<DT>;
  float2 v[El::E / 2];
  El::pairs(r, v);
#pragma unroll
  for (int e = 0; e < El::E / 2; ++e) {
    const float2 t = a.exponent<FUSED>(v[e]), p = exp2_pair(t);
    s = add2(s, p);
    w = fma2(p, make_float2(fmaxf(t.x, -1e30f), fmaxf(t.y, -1e30f)), w);  // -inf: 0 times a finite number
  }
}

// Batches a thread has on their way, in its own places of a ring in shared memory
// (kBatch kDepth vectors a thread: 48 KB at 256 threads, four CTAs an SM). Registers held
// one batch ahead: 8192 x 65536 bf16 took 194 us, 333 rows of 100003 fp16 28 us.
constexpr int kDepth = 3;
constexpr int kRingBytes = 16 * kDepth * kBatch * kThreads;

// The thread's share of the part in one sweep: its largest element and its sums relative
// to that.
template <int DT>
TW_DEV ProbStat own_probs(const Part<DT>& p, float c, uint4* ring) {
  Running<DT> run;
  const float slack = kSlack * fminf(1.f, kLog2e / c);
  float2 s = both(0.f), w = both(0.f);
  Scale a(neg_inf_f(), c);
  bool some = false;
  const int tid = threadIdx.x;
  auto batch = [&](const uint4 (&r)[kBatch]) {
    if (run.grow(r, slack)) {
      const Scale to(run.top.get(), c);
      const float d = fmaxf(a.move(to), -1e30f);  // finite: s and w become 0, not NaN
      const float2 f = both(some ? exp2_fast(d) : 0.f);
      w = mul2(fma2(s, both(some ? d : 0.f), w), f);
      s = mul2(s, f);
      a = to, some = true;
    }
    if (a.fused) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) add_terms<DT, true>(r[i], a, s, w);
    } else {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) add_terms<DT, false>(r[i], a, s, w);
    }
  };
  const uint4* src = reinterpret_cast<const uint4*>(p.at(0));
  constexpr int kStep = kBatch * kThreads, kStage = kStep;  // vectors from a batch, a stage to the next
  auto load = [&](uint4* to, int j) {
    if (j + kStep - kThreads < p.hi) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) cp_async16(to + i * kThreads, src + j + i * kThreads);
    } else {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (j + i * kThreads < p.hi) cp_async16(to + i * kThreads, src + j + i * kThreads);
    }
    cp_commit();
  };
  int j = p.lo + tid;
  uint4 *const begin = ring + tid, *at = begin;
#pragma unroll
  for (int d = 0; d < kDepth; ++d) load(begin + d * kStage, j + d * kStep);
  for (; j < p.hi; j += kStep) {
    cp_wait<kDepth - 1>();
    uint4 r[kBatch];
    if (j + kStep - kThreads < p.hi) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) r[i] = at[i * kThreads];
    } else {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) r[i] = j + i * kThreads < p.hi ? at[i * kThreads] : no_vector<DT>();
    }
    batch(r);
    load(at, j + kDepth * kStep);
    at = at == begin + (kDepth - 1) * kStage ? begin : at + kStage;
  }
  cp_wait<0>();
  if (p.lo > 0 || p.hi < p.n) {  // the edges: one vector of the first thread, one of the last
    uint4 r[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) r[i] = no_vector<DT>();
    if (tid == 0 && p.lo > 0) r[0] = p.edge(0);
    if (tid == kThreads - 1 && p.hi < p.n && p.n > p.lo) r[1] = p.edge(p.n - 1);
    batch(r);
  }
  ProbStat st;
  st.M = run.top.get();
  const float d = fmaf(a.m - base_of(st.M), c, a.shift()), f = exp2_fast(d);
  st.s = add_lanes(s);
  st.w = f * fmaf(st.s, d, add_lanes(w));
  st.s *= f;
  return st;
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const LogprobArgs a, int cluster) {
  using El = Elem<DT>;
  using S = typename El::S;
  extern __shared__ uint4 smem[];  // the ring, then the candidates
  __shared__ Key top[kMaxAlternatives];
  __shared__ ProbStat wstat[kWarps], cstat;
  __shared__ Key wkey[kWarps];
  __shared__ uint16_t above[kThreads];
  __shared__ int count[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster;
  const size_t row = blockIdx.x / cluster;
  const int K = a.K;
  Key* cand = reinterpret_cast<Key*>(smem);
  if (tid < 2) count[tid] = 0;
  for (int k = tid; k < K; k += kThreads) top[k] = 0;
  pdl_enter();

  const S* z = static_cast<const S*>(a.z) + row * a.ldz;
  const Part<DT> part(z, a.V, rank, cluster);
  const float c = kLog2e / a.temperature;
  // the first given tokens' logits come while the row does
  int t_first = -1;
  float z_first = 0.f;
  const bool answers = rank == 0 && warp == 0;
  if (answers && lane < a.n_tokens) {
    t_first = a.tokens[row * a.n_tokens + lane];
    if (t_first >= 0 && t_first < a.V) z_first = El::get(z[t_first]);
  }
  ProbStat st = own_probs(part, c, smem);
  const float mine = st.M;
  st = join<32>(st, c);
  if (lane == 0) wstat[warp] = st;
  const uint32_t high = mine > neg_inf_f() ? order_of(mine) >> 16 : 0;
  const uint32_t thr = K > 0 ? find_threshold(high, K) : 0;
  __syncthreads();
  // warp 0: the part's statistics
  const ProbStat none = {neg_inf_f(), 0.f, 0.f};
  if (warp == 0) {
    st = join<kParts>(lane % kParts < kWarps ? wstat[lane % kParts] : none, c);
    if (lane == 0) cstat = st;
  }
  if (K > 0) {
    part_top<DT>(part, high, K, cand, top, thr, count, above, wkey);
  }
  if (cluster > 1) {
    cluster_barrier();
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
      if (K > 0) {  // of the lists' keys, those that the largest K-th of a list does not rule out
        if (tid == 0) count[0] = 0;
        Key least = 0;
        for (int r = 0; r < cluster; ++r) least = max(least, ld_cluster_u64(peer_smem_addr(top + K - 1, r)));
        __syncthreads();
        for (int i = tid; i < cluster * K; i += kThreads) {
          const Key k = ld_cluster_u64(peer_smem_addr(top + i % K, i / K));
          if (k != 0 && k >= least) cand[atomicAdd(count, 1)] = k;
        }
      }
    }
    cluster_barrier();  // every list has been read: the CTAs may leave, rank 0 may overwrite its own
    if (rank != 0) return;
    if (K > 0) {
      for (int k = tid; k < K; k += kThreads) top[k] = 0;
      __syncthreads();
      rank_select(cand, count[0], top, K);
    }
  }
  if (K > 0) __syncthreads();
  if (warp != 0) return;

  const float bm = base_of(st.M), l2 = log2f(st.s);
  const bool empty = st.s == 0.f;  // every logit -inf
  auto logprob = [&](float v) { return empty ? neg_inf_f() : kLn2 * ((v - bm) * c - l2); };
  for (int i = lane; i < a.n_tokens; i += 32) {
    const int t = i == lane ? t_first : a.tokens[row * a.n_tokens + i];
    float lp = 0.f;
    if (t >= 0 && t < a.V)
      lp = logprob(i == lane ? z_first : El::get(z[t]));
    else if (t != -1)
      raise_status(a.status, TW_EINVAL);
    a.logprob[row * a.n_tokens + i] = lp;
  }
  if (tid == 0 && a.entropy != nullptr) {
    const float h = empty ? 0.f : kLn2 * (l2 - st.w / st.s);
    a.entropy[row] = h < 0.f ? 0.f : h;  // rounding may go below; NaN stays
  }
  const bool bad = !(st.s < __int_as_float(0x7F800000));  // a NaN or an infinity in the row
  for (int k = lane; k < K; k += 32) {
    const Key key = top[k];
    a.top_idx[row * K + k] = key == 0 || bad ? -1 : static_cast<int>(~static_cast<uint32_t>(key));
    a.top_logprob[row * K + k] = bad ? __int_as_float(0x7FC00000) : key == 0 ? neg_inf_f() : logprob(value_of(key >> 32));
  }
}

// ------------------------------------------------------------------ launch shapes
struct RowShape {
  int cluster, part_bytes;
};

// The most 16-byte vectors a row of V elements covers, at any alignment.
int row_vectors(int V, int dtype) {
  const int E = dtype == TW_F32 ? 4 : 8;
  return (V + 2 * E - 2) / E;
}

// CTAs a row (1 to 8): as few as keep a part at `most` bytes, and, while all rows
// together make fewer than `fill` CTAs, as many as keep it at `least`. Eight vectors a
// thread.
RowShape row_shape(int64_t N, int V, int dtype, int most, int64_t fill, int least) {
  const int64_t bytes = 16 * static_cast<int64_t>(row_vectors(V, dtype));
  auto parts = [&](int64_t size) { return (bytes + size - 1) / size; };
  const int64_t few = std::min<int64_t>(8, parts(most));
  const int64_t many = std::min<int64_t>({8, parts(least), fill / N});
  RowShape r;
  r.cluster = static_cast<int>(std::max(few, many));
  r.part_bytes = 16 * ((row_vectors(V, dtype) + r.cluster - 1) / r.cluster);
  return r;
}

template <class... KArgs, class... Args>
cudaError_t launch_rows(void (*kern)(KArgs...), int64_t N, const RowShape& r, size_t smem, const char* label,
                        cudaStream_t s, Args... args) {
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(N * r.cluster)), block(kThreads);
  e = r.cluster == 1 ? launch(kern, grid, block, smem, s, args...)
                     : launch_clustered(kern, grid, block, smem, r.cluster, s, args...);
  trace_mark(s, label);
  return e;
}

// A slice of at most 72 KB keeps three CTAs on an SM, so that one's copies run under
// the others' sweeps. Fewer rows than SMs: more CTAs a row, down to 8 KB each.
template <int DT>
cudaError_t distill(const DistillArgs& a, cudaStream_t s) {
  const RowShape r = row_shape(a.N, a.V, DT, 72 * 1024, device_sm_count(), 8 * 1024);
  const size_t smem = r.part_bytes + 16 * static_cast<size_t>(a.K);
  const int ahead = 3 * device_sm_count() / r.cluster;
  auto run = [&](auto kern) { return launch_rows(kern, a.N, r, smem, "distill", s, a, r.cluster, r.part_bytes, ahead); };
  if (a.labels == nullptr || a.temperature == 1.f) return run(distill_kernel<DT, kNoSum>);
  if (a.temperature == 2.f) return run(distill_kernel<DT, 2>);
  if (a.temperature == 4.f) return run(distill_kernel<DT, 4>);
  return run(distill_kernel<DT, kOwnSum>);
}

// A row needs no place on chip: one CTA takes it, more where there are few rows. Two
// threads an alternative, so that a threshold which K threads reach is passed by few
// elements.
template <int DT>
cudaError_t logprobs(const LogprobArgs& a, cudaStream_t s) {
  const RowShape r = row_shape(a.N, a.V, DT, 1 << 30, 4 * device_sm_count(), 8 * 1024);
  const size_t smem = std::max<size_t>(kRingBytes, a.K > 0 ? sizeof(Key) * kCandidates : 0);
  return launch_rows(logprobs_kernel<DT>, a.N, r, smem, "token_logprobs", s, a, r.cluster);
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
