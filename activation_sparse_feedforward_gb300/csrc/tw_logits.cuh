// Device code that the operators on rows of logits share (tw_logits.cu: one row per
// cluster, and the log probabilities; tw_distill_rows.cuh: short rows, one per CTA): parts of a
// row, softmax statistics, and the distillation's target, loss and gradient.
//
// Softmax statistics are a maximum M of z and sums of 2^(c (z - M)), c = log2(e) /
// temperature; two such pairs join as M = max(M1, M2), S = S1 2^(c (M1-M)) + S2 2^(c (M2-M)).
// M is taken off before the scaling: c z alone would overflow, or lose the whole
// exponent to rounding, where a mask is the type's lowest value. A row, part or thread
// with nothing but -inf has M = -inf and S = 0. The distillation keeps a pair for the listed
// tokens and one for the others, whose mass and gradient are needed by themselves.
#pragma once

#include <cfloat>

#include "tw_internal.h"
#include "tw_rows.cuh"

namespace tw {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

TW_DEV float neg_inf_f() { return __int_as_float(0xFF800000); }
// what to take off z: M, or 0 where there is nothing (so that -inf stays -inf)
TW_DEV float base_of(float M) { return M == neg_inf_f() ? 0.f : M; }
TW_DEV float exp_of(float z, float base, float c) { return exp2_fast((z - base) * c); }

// over groups of W lanes
template <int W = 32>
TW_DEV float warp_max(float v) {
  if constexpr (W == 32) {  // one instruction; a NaN loses to a number, as with fmaxf
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  } else {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
  }
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
  // Whether this thread of NT holds the part's first (last) vector as one that is not whole.
  template <int NT>
  TW_DEV bool first_edge() const { return threadIdx.x == 0 && lo > 0; }
  template <int NT>
  TW_DEV bool last_edge() const { return threadIdx.x == NT - 1 && hi < n && n > lo; }
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

// f(j, all) for the thread's vectors j, j + NT, ... of [lo, hi), NT the CTA's threads, in
// batches of kBatch; all: a constant, whether the whole batch is below hi.
struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };
template <int NT, class F>
TW_DEV void in_batches(int lo, int hi, F f) {
  int j = lo + threadIdx.x;
  for (; j + (kBatch - 1) * NT < hi; j += kBatch * NT) f(j, Yes());
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
  // Takes a batch into the maximum; true when the reference has to move to it.
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

// ------------------------------------------------------------------ a row through a ring
// A row's whole vectors through shared memory: every thread keeps kDepth batches on their
// way in places of its own, so the ring needs no barrier.
template <int DT, int NT, int DEPTH>
struct RowRing {
  static constexpr int kStep = kBatch * NT;  // vectors from a batch to the thread's next
  static constexpr int kBytes = 16 * DEPTH * kStep;
  uint4* begin;
  TW_DEV explicit RowRing(uint4* smem) : begin(smem + threadIdx.x) {}
  TW_DEV void load(const Part<DT>& p, uint4* to, int j) const {
    const uint4* src = reinterpret_cast<const uint4*>(p.at(0));
    if (j + kStep - NT < p.hi) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) cp_async16(to + i * NT, src + j + i * NT);
    } else {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (j + i * NT < p.hi) cp_async16(to + i * NT, src + j + i * NT);
    }
    cp_commit();
  }
  TW_DEV void start(const Part<DT>& p) const {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(p, begin + d * kStep, p.lo + threadIdx.x + d * kStep);
  }
  // f(batch, first vector's index) for all of the started row's whole vectors
  template <class F>
  TW_DEV void sweep(const Part<DT>& p, F f) const {
    uint4* at = begin;
    for (int j = p.lo + threadIdx.x; j < p.hi; j += kStep) {
      cp_wait<DEPTH - 1>();
      uint4 r[kBatch];
      if (j + kStep - NT < p.hi) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) r[i] = at[i * NT];
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) r[i] = j + i * NT < p.hi ? at[i * NT] : no_vector<DT>();
      }
      f(r, j);
      load(p, at, j + DEPTH * kStep);
      at = at == begin + (DEPTH - 1) * kStep ? begin : at + kStep;
    }
    cp_wait<0>();
  }
};

// ------------------------------------------------------------------ distillation
// The hard-label term wants sums of e^z at temperature 1. How a kernel gets them beside
// the sums of p = e^(z / temperature): HARD = kNoSum where there are no labels or the
// temperature is 1; 2 or 4 where the temperature is that: p^2 or p^4, products in place
// of a second exponential an element in each sweep (4096 x 131072 bf16 at temperature 2:
// the exponentials alone would keep their unit busy for three quarters of the floor);
// kOwnSum at any other temperature.
constexpr int kNoSum = 0, kOwnSum = 1;

// The listed and the unlisted tokens' sums each have a reference of their own: against the
// row's largest logit the unlisted ones' would be 0 where the list lies far above them, and
// log q_rest and q / q_rest with it.
struct SoftSum {
  float M, s;  // the largest logit, and the sum at the temperature against it
  float s1;    // the sum at temperature 1 (not with kNoSum)
  static TW_DEV SoftSum none() { return {neg_inf_f(), 0.f, 0.f}; }
};

// The scale at temperature 1 beside `a` at the temperature. (c is log2(e) / HARD, an
// exact division, so HARD times c, k and the shift are exact too.)
template <int HARD>
TW_DEV Scale hard_scale(const Scale& a) {
  Scale b(a.m, kLog2e);
  if (HARD == 2 || HARD == 4) b.k = HARD * a.k, b.fused = a.fused;
  return b;
}

// Joins one SoftSum per lane of groups of W lanes; all of them get it.
template <int HARD, int W = 32>
TW_DEV SoftSum join(SoftSum a, float c0) {
  SoftSum r;
  r.M = warp_max<W>(a.M);
  const float base = base_of(r.M);
  r.s = group_sum<W>(a.s * exp_of(a.M, base, c0));
  r.s1 = HARD != kNoSum ? group_sum<W>(a.s1 * exp_of(a.M, base, kLog2e)) : 0.f;
  return r;
}
template <int HARD>
TW_DEV SoftSum join_two(SoftSum a, SoftSum b, float c0) {
  SoftSum r;
  r.M = fmaxf(a.M, b.M);
  const float base = base_of(r.M);
  r.s = a.s * exp_of(a.M, base, c0) + b.s * exp_of(b.M, base, c0);
  r.s1 = HARD != kNoSum ? a.s1 * exp_of(a.M, base, kLog2e) + b.s1 * exp_of(b.M, base, kLog2e) : 0.f;
  return r;
}
// A row's statistics.
struct DistillStat {
  float M, total;        // the largest logit of all, and the sum over all against it
  float rest_top, rest;  // the unlisted tokens' largest logit and sum
  float rest_near;       // that sum against M
  float s1;              // at temperature 1 over all, against M (total with kNoSum, where that is wanted)
};
template <int HARD>
TW_DEV DistillStat row_stat_of(const SoftSum& rest, const SoftSum& list, float c0) {
  DistillStat r;
  const SoftSum all = join_two<HARD>(rest, list, c0);
  r.M = all.M, r.total = all.s;
  r.rest_top = rest.M, r.rest = rest.s;
  r.rest_near = rest.s * exp_of(rest.M, base_of(all.M), c0);
  r.s1 = HARD != kNoSum ? all.s1 : all.s;
  return r;
}

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
// The sums of a thread's vectors, taken in batches: of p at the scale c0 and, where the
// hard-label term needs its own, at log2(e), relative to the largest element in the end.
template <int DT, int HARD>
struct Sums {
  Running<DT> run;
  float c0;
  Scale a;
  float2 s0, s1;
  TW_DEV explicit Sums(float c) : c0(c), a(neg_inf_f(), c), s0(both(0.f)), s1(both(0.f)) {}
  TW_DEV float slack() const { return kSlack * fminf(1.f, kLog2e / c0); }
  // the scale of s1 beside `of` for s0
  TW_DEV Scale hard(const Scale& of) const {
    Scale b = hard_scale<HARD>(of);
    b.fused = of.fused;
    return b;
  }
  TW_DEV Scale scale_at(float m) const {
    Scale to(m, c0);
    if (HARD == kOwnSum) to.fused = to.fused && Scale(m, kLog2e).fused;
    return to;
  }
  TW_DEV void add(const uint4 (&r)[kBatch]) {
    const bool some = run.limit > neg_inf_f();
    if (run.grow(r, slack())) {
      const Scale to = scale_at(run.top.get());
      // a factor of 0, not a sum set to 0, where only -inf came before: a NaN among them stays
      s0 = mul2(s0, both(some ? exp2_fast(a.move(to)) : 0.f));
      if (HARD != kNoSum) s1 = mul2(s1, both(some ? exp2_fast(hard(a).move(hard(to))) : 0.f));
      a = to;
    }
    if (a.fused)
      add_exps<DT, HARD, true>(r, a, hard(a), s0, s1);
    else
      add_exps<DT, HARD, false>(r, a, hard(a), s0, s1);
  }
  TW_DEV SoftSum get() const {
    SoftSum r;
    r.M = run.top.get();
    const float base = base_of(r.M);
    const Scale b = hard(a);
    r.s = add_lanes(s0) * exp2_fast(fmaf(a.m - base, c0, a.shift()));
    r.s1 = HARD != kNoSum ? add_lanes(s1) * exp2_fast(fmaf(b.m - base, kLog2e, b.shift())) : 0.f;
    return r;
  }
};

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
  bool some;          // the teacher has mass
  float sum, p_rest;  // sum over its classes of e^(logit - the largest), and P of the rest
  int label;
  float up;           // the upstream gradient
  float z_label;      // z at the label (kept by the kernels that need it)
};
// A row's list in shared memory: the token (after the marking -2 - token where the entry
// does not own its place), the teacher's logit over the temperature (after
// teacher_distribution less the largest), P, and z at the token.
struct List {
  int* idx;
  float *lp, *p, *z;
  TW_DEV List(void* at, int K) : idx(static_cast<int*>(at)) {
    lp = reinterpret_cast<float*>(idx + K);
    p = lp + K;
    z = p + K;
  }
};
constexpr int kListBytes = 16;  // an entry

// The rare part of the marking, by the whole CTA of NT threads: of the entries that name one
// token (here(token): in this CTA's part of the row) the lowest owns it, whichever thread
// came to the token first, so that sums are taken in one order; the others learn the token's
// logit from whom had it. Entries that found a masked token have no owner among them yet.
template <int NT, class H>
TW_DEV void lowest_own(const List& l, int K, int label, int* label_entry, H here) {
  static_assert(1024 / NT <= 32, "a bit for each of a thread's entries");
  auto token = [&](int k) { return l.idx[k] >= 0 ? l.idx[k] : -2 - l.idx[k]; };
  __syncthreads();
  uint32_t owns = 0;
  int n = 0;
  for (int k = threadIdx.x; k < K; k += NT, ++n) {
    const int i = token(k);
    bool own = i >= 0 && here(i);
    for (int q = 0; i >= 0 && q < K; ++q) {
      const int at = l.idx[q];
      if (at == i && q != k) l.z[k] = l.z[q];
      if (q < k && (at == i || at == -2 - i)) own = false;
    }
    owns |= own ? 1u << n : 0u;
  }
  __syncthreads();
  n = 0;
  for (int k = threadIdx.x; k < K; k += NT, ++n) {
    const int i = token(k);
    const bool own = owns >> n & 1u;
    l.idx[k] = own ? i : -2 - i;
    if (own && i == label) *label_entry = k;
  }
  __syncthreads();
}

// By one warp: the sums of the tokens that the list owns (l.idx >= 0); all lanes get them.
// A lane holds its first FIRST entries' logits between the sweep for the largest and the
// sums (0: where registers are short).
template <int HARD, int FIRST>
TW_DEV SoftSum list_sums(const List& l, int K, float c0) {
  constexpr int kUnroll = FIRST > 0 ? 4 : 2;
  const int lane = threadIdx.x & 31;
  auto owned = [&](int k) { return k < K && l.idx[k] >= 0 ? l.z[k] : neg_inf_f(); };
  SoftSum r = SoftSum::none();
  float z[FIRST + 1];  // (+ 1: not empty)
#pragma unroll
  for (int n = 0; n < FIRST; ++n) r.M = fmaxf(r.M, z[n] = owned(lane + 32 * n));
#pragma unroll kUnroll
  for (int k = lane + 32 * FIRST; k < K; k += 32) r.M = fmaxf(r.M, owned(k));
  r.M = warp_max(r.M);
  const float base = base_of(r.M);
  auto add = [&](float v) {
    r.s += exp_of(v, base, c0);
    if (HARD != kNoSum) r.s1 += exp_of(v, base, kLog2e);
  };
#pragma unroll
  for (int n = 0; n < FIRST; ++n) add(z[n]);
#pragma unroll kUnroll
  for (int k = lane + 32 * FIRST; k < K; k += 32) add(owned(k));
  r.s = warp_sum(r.s);
  if (HARD != kNoSum) r.s1 = warp_sum(r.s1);
  return r;
}

// By one warp: the teacher's distribution over the list, whose logits are in l.lp, and the
// rest, into l.p and the target.
TW_DEV void teacher_distribution(const List& l, int K, float t_rest, Target* target) {
  const int lane = threadIdx.x & 31;
  float tm = t_rest;
  for (int k = lane; k < K; k += 32) tm = fmaxf(tm, l.lp[k]);
  tm = base_of(warp_max(tm));
  float ts = 0.f;
  for (int k = lane; k < K; k += 32) {
    const float e = exp_of(l.lp[k], tm, kLog2e);
    l.p[k] = e;
    ts += e;
  }
  const float e_rest = exp_of(t_rest, tm, kLog2e);
  ts = warp_sum(ts) + e_rest;
  const float inv = 1.f / ts;
  for (int k = lane; k < K; k += 32) {
    l.p[k] *= inv;
    l.lp[k] -= tm;
  }
  if (lane == 0) {
    target->some = ts != 0.f;  // NaN counts as some
    target->p_rest = ts != 0.f ? e_rest * inv : 0.f;
    target->sum = ts;
  }
}

// One warp takes a row's target: load() before the row's own loads, which would hold these
// up, finish() while the row is on its way.
struct TargetLoads {
  static constexpr int kFirst = 4;  // entries a lane loads at once: lists of up to 128
  int label = -1, i_first[kFirst];
  float t_rest = neg_inf_f(), up = 1.f, t_first[kFirst];
  TW_DEV void load(const DistillArgs& a, size_t row) {
    const int lane = threadIdx.x & 31;
    if (a.labels != nullptr) label = a.labels[row];
    if (a.t_rest != nullptr) t_rest = a.t_rest[row];
    if (a.dloss != nullptr) up = a.dloss[row];
#pragma unroll
    for (int n = 0; n < kFirst; ++n) {
      const int k = lane + 32 * n;
      i_first[n] = k < a.K ? a.t_idx[row * a.K + k] : -1;
      t_first[n] = k < a.K ? teacher_logit(a, row * a.K + k) : 0.f;
    }
  }
  TW_DEV void finish(const DistillArgs& a, size_t row, const List& l, Target* target) {
    const int lane = threadIdx.x & 31, K = a.K;
    if (label < -1 || label >= a.V) {
      if (lane == 0) raise_status(a.status, TW_EINVAL);
      label = -1;
    }
    auto entry = [&](int k, int i, float t) {
      if (i < 0 || i >= a.V) {
        if (i != -1) raise_status(a.status, TW_EINVAL);
        i = -1;
        t = neg_inf_f();
      }
      l.idx[k] = i;
      l.lp[k] = t > neg_inf_f() ? fmaxf(t / a.temperature, -FLT_MAX) : t;  // a finite logit stays one
    };
#pragma unroll
    for (int n = 0; n < kFirst; ++n)
      if (lane + 32 * n < K) entry(lane + 32 * n, i_first[n], t_first[n]);
    for (int k = lane + 32 * kFirst; k < K; k += 32) entry(k, a.t_idx[row * K + k], teacher_logit(a, row * K + k));
    teacher_distribution(l, K, t_rest, target);
    if (lane == 0) {
      target->label = label;
      target->up = up * a.scale;
    }
  }
};
// By one warp: asks for the target of a row that is taken later. Cold, these loads were
// the longest step before the sums.
TW_DEV void prefetch_target(const DistillArgs& a, size_t row) {
  const int lane = threadIdx.x & 31, size = a.t_dtype == TW_F32 ? 4 : 2;
  for (int k = lane * 32; k < a.K; k += 32 * 32) {
    prefetch_line(a.t_idx + row * a.K + k);
    prefetch_line(static_cast<const uint8_t*>(a.t_val) + (row * a.K + k) * size);
  }
  if (lane == 0 && a.t_rest != nullptr) prefetch_line(a.t_rest + row);
  if (lane == 0 && a.labels != nullptr) prefetch_line(a.labels + row);
  if (lane == 0 && a.dloss != nullptr) prefetch_line(a.dloss + row);
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
// Stores f of the vectors [lo, hi) of a part, which get(j) reads, at their columns of a row
// that lies otherwise against 16 bytes: each vector stored is put together from two, by
// both(j, shift). (One element at a time, 3358 x 120602 bf16 took 965 us, most of it partial
// writes in L2; this 396.)
template <int DT, int NT, class G, class B, class F>
TW_DEV void store_shifted(const Part<DT>& p, typename Elem<DT>::S* dz, int lo, int hi, G get, B both, F f) {
  using S = typename Elem<DT>::S;
  constexpr int E = Elem<DT>::E;
  const int shift = (p.lead - Part<DT>::lead_of(dz)) & (E - 1), first = p.col(lo) + shift;
  auto singly = [&](const uint4& r, int c, int from, int to) {  // elements [from, to) of r, whose first is column c
    const uint4 v = f(r);
    const S* o = reinterpret_cast<const S*>(&v);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e >= from && e < to && c + e >= 0 && c + e < p.V) dz[c + e] = o[e];
  };
#pragma unroll 2
  for (int i = threadIdx.x; i < hi - lo - 1; i += NT) {
    const uint4 r = both(lo + i, shift);
    const int c = first + i * E;
    if (c >= 0 && c + E <= p.V)
      *reinterpret_cast<uint4*>(dz + c) = f(r);
    else
      singly(r, c, 0, E);
  }
  if (lo >= hi) return;
  if (threadIdx.x == 0) singly(get(lo), p.col(lo), 0, shift);
  if (threadIdx.x == NT - 1) singly(get(hi - 1), p.col(hi - 1), shift, E);
}

// A row's loss from its statistics: the terms of the entries for which here(k, token)
// holds, by the threads that fill them; the rest's and the label's by the threads told so.
// tau (log P - log q), in the logits' own units so that a mask of the type's lowest value
// stays finite, is taken from the logits' distances to their largest and from quotients of
// the sums: all are small where teacher and student agree, while each logarithm by itself
// rounds at its own size.
template <class F>
TW_DEV float loss_share(const DistillArgs& a, const DistillStat& st, const List& l, const Target& t, int threads,
                        bool takes_rest, bool takes_label, float z_label, F here) {
  const float tau = a.temperature, b = base_of(st.M);
  float share = 0.f;
  if (t.some) {
    const float ratio = tau * logf(st.total / t.sum);
    for (int k = threadIdx.x; k < a.K; k += threads) {
      const int i = l.idx[k] >= 0 ? l.idx[k] : -2 - l.idx[k];
      const float p = l.p[k];
      if (i >= 0 && p != 0.f && here(i)) share += p * (fmaf(tau, l.lp[k], b - l.z[k]) + ratio);
    }
    if (takes_rest && t.p_rest != 0.f) {
      // the quotient against M while it has all its digits, else the distance beside it
      const bool near = st.rest_near >= 0x1p-60f;
      const float d = tau * logf(t.p_rest * st.total / (near ? st.rest_near : st.rest));
      share += t.p_rest * (near ? d : d + (st.M - st.rest_top));
    }
    share *= a.kd_weight * tau;
  }
  if (takes_label) share += a.ce_weight * (b - z_label + logf(st.s1));
  return share;
}

// The gradient's factors of a row (see the header): u 2^(c0 (z - m)) + w e^(z - m) on
// unlisted tokens, and the values that overwrite it at the list and the label. m is the
// unlisted tokens' largest logit where the teacher has a rest, so that P_rest q / q_rest is
// a sum of factors of at most 1 whatever the list's logits are; else the row's largest.
template <int HARD>
struct Gradient {
  bool rest;  // the teacher has a rest, and the student tokens for it
  float b, c0, total, gk, gc, u, w;
  Scale sa, sb;
  float uf, wf;  // u and w against the scales' own references
  bool fused, zero;
  TW_DEV Gradient(const DistillArgs& a, const DistillStat& st, float c0_, const Target& t)
      : rest(t.p_rest != 0.f && st.rest != 0.f), b(base_of(st.M)), c0(c0_), total(st.total),
        sa(rest ? st.rest_top : st.M, c0_), sb(hard_scale<HARD>(sa)) {
    zero = (!t.some && t.label < 0) || total == 0.f;
    gk = t.up * a.kd_weight * a.temperature;
    gc = t.label >= 0 ? t.up * a.ce_weight : 0.f;
    u = t.some ? gk / total : 0.f;
    w = t.label >= 0 ? gc / st.s1 : 0.f;
    if (rest) {
      u = u * exp_of(sa.m, b, c0) - gk * t.p_rest / st.rest;
      w *= exp_of(sa.m, b, kLog2e);
    }
    if (HARD == kNoSum) u += w;
    fused = sa.fused && sb.fused;
    uf = fused ? u * exp2_fast(sa.shift()) : u;
    wf = fused ? w * exp2_fast(sb.shift()) : w;
  }
  // at entry k, which owns token l.idx[k]; dup: entries may name a token twice
  TW_DEV float listed(const DistillStat& st, const List& l, int K, int k, int label, bool dup) const {
    const int i = l.idx[k];
    float p = l.p[k];
    if (dup) {  // add up, in list order, every entry that names the same token
      p = 0.f;
      for (int q = 0; q < K; ++q)
        if (l.idx[q] == i || l.idx[q] == -2 - i) p += l.p[q];
    }
    float d = gk * (exp_of(l.z[k], b, c0) / total - p);
    if (label >= 0) d += gc / st.s1 * exp_of(l.z[k], b, kLog2e);
    return i == label ? d - gc : d;
  }
  // at the label, which is not listed
  TW_DEV float at_label(float z) const {
    const float d = u * exp_of(z, sa.m, c0) - gc;
    return HARD != kNoSum ? fmaf(w, exp_of(z, sa.m, kLog2e), d) : d;
  }
  // f(vector -> gradient) chosen by the row's case
  template <int DT, class F>
  TW_DEV void with(F f) const {
    if (zero)
      f([](const uint4&) { return make_uint4(0, 0, 0, 0); });
    else if (fused)
      f([&](const uint4& r) { return gradient<DT, HARD, true>(r, sa, sb, uf, wf); });
    else
      f([&](const uint4& r) { return gradient<DT, HARD, false>(r, sa, sb, uf, wf); });
  }
};

// ------------------------------------------------------------------ host side
// The most 16-byte vectors a row of V elements covers, at any alignment.
inline int row_vectors(int V, int dtype) {
  const int E = dtype == TW_F32 ? 4 : 8;
  return (V + 2 * E - 2) / E;
}
// The kernels' HARD for a call.
inline int hard_form(const DistillArgs& a) {
  if (a.labels == nullptr || a.temperature == 1.f) return kNoSum;
  return a.temperature == 2.f ? 2 : a.temperature == 4.f ? 4 : kOwnSum;
}

}  // namespace

}  // namespace tw
