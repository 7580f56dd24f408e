// Operators on rows of logits [N, V]: the distillation loss with its gradient, and log
// probabilities of given tokens with the row's entropy and top alternatives.
//
//  log probabilities  One CTA a row (a cluster of up to eight where there are few rows), the
//                     row through a ring of asynchronous copies, read once.
//  distillation       A cluster of up to eight CTAs a row, each with a slice of it in shared
//                     memory, so that HBM is read once. Many short rows, and the loss
//                     alone: one small CTA a row, which reads it a second time from L2 for
//                     the gradient (tw_distill_rows.cuh).
//
// Bound: HBM, one read of the logits and, with a gradient, one write. Measured on one GB300
// against the copy rate (6681 GB/s): log probabilities 8192 x 65536 bf16 with five
// alternatives 167 us (0.96); distillation 4096 x 131072 bf16, K = 64, temperature 2, rest
// and labels 428 us (0.75), fp32 1023 x 50011, K = 33, 92 us (0.67). What keeps the
// distillation from the copy rate are the steps between a slice's sweeps: of the 11.9 us a
// CTA takes for 64 KB (three on an SM, with time stamps) 3.7 pass until the copies are issued
// and the target taken, 0.6 with the listed entries, 2.1 with the sums, 1.8 with joining the
// cluster's statistics and 3.1 with the gradient.
//
// Both join partial statistics through distributed shared memory: one launch, no
// workspace, no atomics on results.
#include <algorithm>

#include "tw_logits.cuh"

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

// ------------------------------------------------------------------ distillation, one row per cluster
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
  TW_DEV bool first_edge() const { return P::template first_edge<kThreads>(); }
  TW_DEV bool last_edge() const { return P::template last_edge<kThreads>(); }
  // the element of column c, or null when another CTA holds it
  TW_DEV S* element(int c) const {
    const int e = c + this->lead - this->first * E;
    return e >= 0 && e < this->n * E ? reinterpret_cast<S*>(buf) + e : nullptr;
  }
};

// The thread's own vectors of the slice in one sweep.
template <int DT, int HARD>
TW_DEV SoftSum own_sums(const Slice<DT>& sl, float c0) {
  Sums<DT, HARD> sums(c0);
  in_batches<kThreads>(sl.lo, sl.hi, [&](int j, auto all) {
    uint4 r[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) r[i] = all.value || j + i * kThreads < sl.hi ? sl.buf[j + i * kThreads] : no_vector<DT>();
    sums.add(r);
  });
  if (sl.first_edge() || sl.last_edge()) {
    const uint4 r[kBatch] = {sl.first_edge() ? sl.buf[0] : no_vector<DT>(), sl.last_edge() ? sl.buf[sl.n - 1] : no_vector<DT>(),
                             no_vector<DT>(), no_vector<DT>()};
    sums.add(r);
  }
  return sums.get();
}

// f of the slice's vectors, stored at their columns of dz; each thread takes its own where
// dz's row lies against 16 bytes as z's does.
template <int DT, class F>
TW_DEV void store_slice(const Slice<DT>& sl, typename Elem<DT>::S* dz, F f) {
  using S = typename Elem<DT>::S;
  constexpr int E = Elem<DT>::E;
  if (Part<DT>::lead_of(dz) != sl.lead) {
    store_shifted<DT, kThreads>(sl, dz, 0, sl.n, [&](int j) { return sl.buf[j]; },
                                [&](int j, int shift) { return shifted_from<DT>(sl.buf + j, shift); }, f);
    return;
  }
  auto singly = [&](int j) {
    const uint4 g = f(sl.buf[j]);
    const S* o = reinterpret_cast<const S*>(&g);
    const int c = sl.col(j);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (c + e >= 0 && c + e < sl.V) dz[c + e] = o[e];
  };
  uint4* out = reinterpret_cast<uint4*>(dz + sl.col(0));
  in_batches<kThreads>(sl.lo, sl.hi, [&](int j, auto all) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (all.value || j + i * kThreads < sl.hi) out[j + i * kThreads] = f(sl.buf[j + i * kThreads]);
  });
  if (sl.first_edge()) singly(0);
  if (sl.last_edge()) singly(sl.n - 1);
}

// One row per cluster, its slices in shared memory. What the CTAs tell each other is pushed
// into the receiver's shared memory before a cluster barrier: every warp's statistics to
// every CTA, every warp's share of the loss to rank 0.
template <int DT, int HARD>
__global__ void __launch_bounds__(kThreads, 3) distill_kernel(const DistillArgs a, int cluster, int slice_bytes, int ahead) {
  using El = Elem<DT>;
  using S = typename El::S;
  extern __shared__ uint4 smem[];
  __shared__ float4 stats[kMaxCluster * kWarps];
  __shared__ float4 lists[kMaxCluster];
  __shared__ float shares[kMaxCluster * kWarps];
  __shared__ Target target;
  __shared__ int label_entry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster;
  const size_t row = blockIdx.x / cluster;
  const int K = a.K;
  const List l(reinterpret_cast<uint8_t*>(smem) + slice_bytes, K);
  pdl_enter();
  if (cluster > 1) cluster_arrive_relaxed();  // waited for before the first push: every CTA has started

  // Warp 0 takes the row's target while the slice is on its way; the other warps keep out
  // of its way (all of them taking it for themselves cost 1 us a row in issue slots).
  const float c0 = kLog2e / a.temperature;
  const S* z = static_cast<const S*>(a.z) + row * a.ldz;
  TargetLoads loads;
  if (warp == 0) loads.load(a, row);
  const Slice<DT> sl(z, a.V, rank, cluster, smem);
  if (warp == 0) {
    loads.finish(a, row, l, &target);
    if (lane == 0) label_entry = -1;
  }
  if (rank == 0 && warp == kWarps - 1 && row + ahead < static_cast<size_t>(a.N)) prefetch_target(a, row + ahead);

  // Listed tokens leave the row: an entry takes the token's logit and puts -inf in its
  // place. Whoever finds -inf there comes second (a token listed twice), or the logit was
  // masked: lowest_own() sorts that out.
  cp_wait<0>();
  __syncthreads();
  const int label = target.label;
  const bool some = target.some;
  bool dup = false;
  if (some) {
    for (int k = tid; k < K; k += kThreads) {
      const int i = l.idx[k];
      S* s = i >= 0 ? sl.element(i) : nullptr;
      const float v = s != nullptr ? El::get(El::exchange(s, El::neg_inf())) : 0.f;
      l.z[k] = v;
      const bool owner = s != nullptr && v != neg_inf_f();
      if (s != nullptr && !owner) dup = true;
      if (!owner) l.idx[k] = -2 - i;  // padding: -1
      if (owner && i == label) label_entry = k;
    }
    dup = __syncthreads_or(dup);
    if (dup) lowest_own<kThreads>(l, K, label, &label_entry, [&](int i) { return sl.element(i) != nullptr; });
  }

  // the row's statistics: every warp's sums of its own tokens, and first the last warp's of the list
  const SoftSum none = SoftSum::none();
  auto packed = [](const SoftSum& v) { return make_float4(v.M, v.s, v.s1, 0.f); };
  auto unpacked = [](const float4& v) { return SoftSum{v.x, v.y, v.z}; };
  const bool takes_list = warp == kWarps - 1;
  const SoftSum own_list = takes_list && some ? list_sums<HARD, 4>(l, K, c0) : none;
  const SoftSum own = join<HARD>(own_sums<DT, HARD>(sl, c0), c0);
  if (cluster > 1) {
    cluster_wait();
    if (lane < cluster) {
      st_cluster_v4(peer_smem_addr(&stats[rank * kWarps + warp], lane), packed(own));
      if (takes_list) st_cluster_v4(peer_smem_addr(&lists[rank], lane), packed(own_list));
    }
    cluster_barrier();
  } else {
    if (lane == 0) {
      stats[warp] = packed(own);
      if (takes_list) lists[0] = packed(own_list);
    }
    __syncthreads();
  }
  const int parts = cluster * kWarps;
  auto part = [&](int i) { return i < parts ? unpacked(stats[i]) : none; };
  SoftSum rest = part(lane);
  if (parts > 32) rest = join_two<HARD>(rest, part(lane + 32), c0);
  rest = join<HARD>(rest, c0);
  SoftSum list = none;
  if (some) {
    const int r = lane % kMaxCluster;
    list = cluster == 1 ? unpacked(lists[0]) : join<HARD, kMaxCluster>(r < cluster ? unpacked(lists[r]) : none, c0);
  }
  const DistillStat st = row_stat_of<HARD>(rest, list, c0);

  const bool holds_label = label >= 0 && sl.element(label) != nullptr;
  const float z_label = !holds_label ? 0.f : label_entry >= 0 ? l.z[label_entry] : El::get(*sl.element(label));
  if (a.loss != nullptr) {
    float share = loss_share(a, st, l, target, kThreads, rank == 0 && tid == 0, holds_label && tid == 0, z_label,
                             [&](int i) { return sl.element(i) != nullptr; });
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
    const Gradient<HARD> g(a, st, c0, target);
    g.template with<DT>([&](auto f) { store_slice<DT>(sl, dz, f); });
    __syncthreads();  // the listed tokens and the label overwrite what the sweep stored
    if (some && !g.zero) {
      for (int k = tid; k < K; k += kThreads)
        if (l.idx[k] >= 0) dz[l.idx[k]] = El::put(g.listed(st, l, K, k, label, dup));
    }
    if (tid == 0 && holds_label && label_entry < 0 && !g.zero) dz[label] = El::put(g.at_label(z_label));
  }

  if (cluster > 1)
    cluster_wait();
  else if (a.dz == nullptr)
    __syncthreads();
  if (rank == 0 && warp == 0 && a.loss != nullptr) {
    float loss = (lane < parts ? shares[lane] : 0.f) + (lane + 32 < parts ? shares[lane + 32] : 0.f);
    loss = warp_sum(loss);
    if (lane == 0) a.loss[row] = !some && label < 0 ? 0.f : st.total == 0.f ? __int_as_float(0x7F800000) : loss;
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
template <int NT>
TW_DEV void rank_select(Key* cand, int n, Key* top, int K) {
  const ulonglong2* two = reinterpret_cast<const ulonglong2*>(cand);
  for (int i = threadIdx.x; i < n; i += NT) {
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
template <int DT, int NT, class F>
TW_DEV void each_vector(const Part<DT>& p, F f) {
#pragma unroll 4
  for (int j = p.lo + threadIdx.x; j < p.hi; j += NT) f(*reinterpret_cast<const uint4*>(p.at(j)), j);
  if (p.template first_edge<NT>()) f(p.edge(0), 0);
  if (p.template last_edge<NT>()) f(p.edge(p.n - 1), p.n - 1);
}

// A thread's batches of a part in chunks, whose largest elements are kept apart: the
// alternatives are then looked for in a few chunks, not in all of a thread's vectors
// (2048 rows of 131072 bf16 with 32 alternatives took 157 us, without any 82).
constexpr int kChunks = 8;
template <int DT, int NT>
TW_DEV int chunk_batches(const Part<DT>& p) {
  const int batches = (p.hi - p.lo + kBatch * NT - 1) / (kBatch * NT);
  return max(1, (batches + kChunks - 1) / kChunks);
}

// The K largest keys of the CTA's part, descending, into top (0 past the finite ones).
// thr is reached by the largest elements of at least K threads, and so leaves few
// candidates, all in the chunks of threads whose largest element reaches it. The whole CTA
// reads these once more (from L2), a vector a thread: left to their owners, one lane of a
// warp would walk a row's worth of latencies. A list that overflows (many ties, or the
// largest elements all in few chunks) falls back to K sweeps for the next largest key.
// highs: the thread's own column of its chunks' largest elements, NT apart, as upper halves
// of their order (0: none); count (two zeros) and top (zeros): set by the caller behind a
// barrier; above: room for a number of each chunk.
template <int DT, int NT>
TW_DEV void part_top(const Part<DT>& p, const uint16_t* highs, int K, Key* cand, Key* top, uint32_t thr, int* count,
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
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const uint32_t high = highs[c * NT];
    if (high != 0 && high >= thr) above[atomicAdd(count + 1, 1)] = static_cast<uint16_t>(c * NT + tid);
  }
  if (p.template first_edge<NT>()) collect(p.edge(0), 0);
  if (p.template last_edge<NT>()) collect(p.edge(p.n - 1), p.n - 1);
  __syncthreads();
  const int each = chunk_batches<DT, NT>(p) * kBatch, work = count[1] * each;
#pragma unroll 4
  for (int i = tid; i < work; i += NT) {
    const int from = above[i / each];
    const int j = p.lo + from % NT + (from / NT * each + i % each) * NT;
    if (j < p.hi) collect(*reinterpret_cast<const uint4*>(p.at(j)), j);
  }
  __syncthreads();
  const int n = *count;
  if (n <= kCandidates) {
    rank_select<NT>(cand, n, top, K);
    return;
  }
  Key last = ~0ull;
  for (int r = 0; r < K; ++r) {
    Key best = 0;
    each_vector<DT, NT>(p, [&](const uint4& w, int j) {
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
    for (int w = 0; w < NT / 32; ++w) best = max(best, wkey[w]);
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

// Three batches a thread on their way: 48 KB an SM's quarter. (8192 x 65536 bf16 with five
// alternatives 167 us. When the ring took the place of one batch ahead in registers, before
// the chunks and the smaller CTAs, that went from 194 us to 178.)
template <int DT, int NT>
using ProbRing = RowRing<DT, NT, 3>;

// The thread's share of the part in one sweep: its largest element and its sums relative
// to that. highs (null: not wanted): see part_top.
template <int DT, int NT>
TW_DEV ProbStat own_probs(const Part<DT>& p, float c, const ProbRing<DT, NT>& ring, uint16_t* highs) {
  Running<DT> run;
  float largest = neg_inf_f();  // of the chunks that are done
  const float slack = kSlack * fminf(1.f, kLog2e / c);
  float2 s = both(0.f), w = both(0.f);
  Scale a(neg_inf_f(), c);
  bool some = false;
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
  auto high_of = [](float v) { return v > neg_inf_f() ? static_cast<uint16_t>(order_of(v) >> 16) : uint16_t{0}; };
  int left = highs != nullptr ? chunk_batches<DT, NT>(p) : 0, chunk = 0;
  const int per = left;
  if (highs != nullptr) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) highs[c * NT] = 0;
  }
  // the edges, one vector of the first thread and one of the last, come while the row does
  const bool first = p.template first_edge<NT>(), last = p.template last_edge<NT>();
  const uint4 e0 = first ? p.edge(0) : no_vector<DT>(), e1 = last ? p.edge(p.n - 1) : no_vector<DT>();
  ring.sweep(p, [&](const uint4 (&r)[kBatch], int) {
    batch(r);
    if (highs != nullptr) {  // kept as the chunk goes: the last one may be short
      const float m = run.top.get();
      highs[chunk * NT] = high_of(m);
      if (--left == 0) {
        largest = fmaxf(largest, m);
        run.top = typename Elem<DT>::Max();
        left = per, ++chunk;
      }
    }
  });
  if (first || last) {
    const uint4 r[kBatch] = {e0, e1, no_vector<DT>(), no_vector<DT>()};
    batch(r);
  }
  ProbStat st;
  st.M = fmaxf(largest, run.top.get());
  const float d = fmaf(a.m - base_of(st.M), c, a.shift()), f = exp2_fast(d);
  st.s = add_lanes(s);
  st.w = f * fmaf(st.s, d, add_lanes(w));
  st.s *= f;
  return st;
}

// NT threads (64, 128 or 256); 1024 / NT CTAs an SM.
template <int DT, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) logprobs_kernel(const LogprobArgs a, int cluster) {
  using El = Elem<DT>;
  using S = typename El::S;
  constexpr int kWarps = NT / 32;
  extern __shared__ uint4 smem[];  // the ring, then the candidates and the chunks above the threshold
  __shared__ Key top[kMaxAlternatives];
  __shared__ ProbStat wstat[kWarps], cstat;
  __shared__ Key wkey[kWarps];
  __shared__ uint16_t highs[kChunks * NT];
  __shared__ int count[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster;
  const size_t row = blockIdx.x / cluster;
  const int K = a.K;
  Key* cand = reinterpret_cast<Key*>(smem);
  uint16_t* above = reinterpret_cast<uint16_t*>(cand + kCandidates);
  if (tid < 2) count[tid] = 0;
  for (int k = tid; k < K; k += NT) top[k] = 0;
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
  const ProbRing<DT, NT> ring(smem);
  ring.start(part);
  ProbStat st = own_probs<DT, NT>(part, c, ring, K > 0 ? highs + tid : nullptr);
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
  if (K > 0) part_top<DT, NT>(part, highs + tid, K, cand, top, thr, count, above, wkey);
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
        for (int i = tid; i < cluster * K; i += NT) {
          const Key k = ld_cluster_u64(peer_smem_addr(top + i % K, i / K));
          if (k != 0 && k >= least) cand[atomicAdd(count, 1)] = k;
        }
      }
    }
    cluster_barrier();  // every list has been read: the CTAs may leave, rank 0 may overwrite its own
    if (rank != 0) return;
    if (K > 0) {
      for (int k = tid; k < K; k += NT) top[k] = 0;
      __syncthreads();
      rank_select<NT>(cand, count[0], top, K);
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

// CTAs a row (1 to 8): as few as keep a part at `most` bytes, and, while all rows
// together make fewer than `fill` CTAs, as many as keep it at `least`.
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

// Whether, and with CTAs of how many threads, one small CTA takes a row and reads it a
// second time from L2 for the gradient (tw_distill_rows.cuh). Short rows are bound by the
// steps between their sweeps, so many small CTAs an SM beat a few that hold rows on chip;
// long ones would not stay in L2. Fraction of the copy rate at K = 64, temperature 2, with
// rest and labels, 64 threads / 128 threads / one row per cluster, 134 to 402 MB of logits:
// rows of 8 KB (bf16) 0.43 / 0.34 / 0.16, 16 KB 0.57 / 0.49 / 0.30, 32 KB 0.69 / 0.64 / 0.49,
// 48 KB 0.69 / 0.74 / 0.61; fp32 of 32 KB 0.76 / 0.76 / 0.57, 48 KB 0.66 / 0.84 / 0.73, 64 KB
// 0.60 / 0.77 / 0.81. At 32 KB a cluster is
// faster up to two rows an SM, and 64 threads slower up to sixteen. The loss alone needs no
// second sweep, so it takes long rows too once they fill the device: 4096 x 128000 bf16 162
// us (cluster 291), 320 x 64000 13.7 (15.5), 160 x 128000 16.8 (16.3), 640 x 32000 15.3 (14.1).
int distill_rows_threads(const DistillArgs& a) {
  const int64_t kb = static_cast<int64_t>(row_vectors(a.V, a.dtype)) / 64, sms = device_sm_count();
  if (kb <= 24 && a.N >= 16 * sms) return 64;
  if (a.dz == nullptr && kb > 52) return (kb >= 100 && a.N >= sms && kb * a.N >= 256 * sms) || a.N >= 8 * sms ? 128 : 0;
  return kb <= 52 && a.N >= 2 * sms ? 128 : 0;
}

template <class... KArgs, class... Args>
cudaError_t launch_rows(void (*kern)(KArgs...), int64_t N, const RowShape& r, int threads, size_t smem,
                        const char* label, cudaStream_t s, Args... args) {
  cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(N * r.cluster)), block(threads);
  e = r.cluster == 1 ? launch(kern, grid, block, smem, s, args...)
                     : launch_clustered(kern, grid, block, smem, r.cluster, s, args...);
  trace_mark(s, label);
  return e;
}

// One row per cluster: slices of at most 72 KB keep three CTAs on an SM, so that one's
// copies run under the others' sweeps. Fewer rows than SMs: more CTAs a row, down to 8 KB
// each.
template <int DT>
cudaError_t distill(const DistillArgs& a, cudaStream_t s) {
  const RowShape r = row_shape(a.N, a.V, DT, 72 * 1024, device_sm_count(), 8 * 1024);
  const size_t smem = r.part_bytes + kListBytes * static_cast<size_t>(a.K);
  const int ahead = 3 * device_sm_count() / r.cluster;
  auto run = [&](auto kern) {
    return launch_rows(kern, a.N, r, kThreads, smem, "distill", s, a, r.cluster, r.part_bytes, ahead);
  };
  switch (hard_form(a)) {
    case kNoSum: return run(distill_kernel<DT, kNoSum>);
    case 2: return run(distill_kernel<DT, 2>);
    case 4: return run(distill_kernel<DT, 4>);
    default: return run(distill_kernel<DT, kOwnSum>);
  }
}

template <int DT, int NT>
cudaError_t logprobs(const LogprobArgs& a, const RowShape& r, cudaStream_t s) {
  const size_t lists = a.K > 0 ? sizeof(Key) * kCandidates + sizeof(uint16_t) * kChunks * NT : 0;
  return launch_rows(logprobs_kernel<DT, NT>, a.N, r, NT, std::max<size_t>(ProbRing<DT, NT>::kBytes, lists),
                     "token_logprobs", s, a, r.cluster);
}

// A row needs no place on chip: one CTA takes it, more where there are few rows. Many
// short rows: smaller CTAs, as many more of them an SM, so that the steps after one row's
// sweep run under the others' sweeps; but with few threads an alternative the threshold
// lets many elements pass. Fraction of the copy rate with 5 alternatives (32), 64 / 128 /
// 256 threads: bf16 rows of 16 KB 0.47 / 0.38 / 0.24 (0.23 / 0.29 / 0.21), 32 KB 0.66 /
// 0.56 / 0.40 (0.37 / 0.46 / 0.36), 64 KB 0.82 / 0.78 / 0.61 (0.43 / 0.66 / 0.56), 128 KB
// - / 0.90 / 0.82 (- / 0.69 / 0.77); without any, 64 threads reach it from 32 KB.
template <int DT>
cudaError_t logprobs_any(const LogprobArgs& a, cudaStream_t s) {
  const int sms = device_sm_count();
  const RowShape r = row_shape(a.N, a.V, DT, 1 << 30, 4 * sms, 8 * 1024);
  const int kb = row_vectors(a.V, DT) / 64;
  if (kb <= 48 && a.K <= 16 && a.N >= 16 * sms) return logprobs<DT, 64>(a, r, s);
  if (((kb <= 72 && a.K <= 32) || (kb <= 140 && a.K <= 8)) && a.N >= 8 * sms) return logprobs<DT, 128>(a, r, s);
  return logprobs<DT, 256>(a, r, s);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t s) {
  if (a.N == 0) return cudaSuccess;
  switch (distill_rows_threads(a)) {
    case 64: return launch_distill_rows_64(a, s);
    case 128: return launch_distill_rows_128(a, s);
  }
  return a.dtype == TW_F32 ? distill<TW_F32>(a, s) : a.dtype == TW_BF16 ? distill<TW_BF16>(a, s) : distill<TW_F16>(a, s);
}

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t s) {
  if (a.N == 0) return cudaSuccess;
  return a.dtype == TW_F32    ? logprobs_any<TW_F32>(a, s)
         : a.dtype == TW_BF16 ? logprobs_any<TW_BF16>(a, s)
                              : logprobs_any<TW_F16>(a, s);
}

}  // namespace tw
