// Token embedding, forward and backward (tw_embedding_fwd, tw_embedding_bwd).
//
//   y[t] = scale E[tok_t]                               (0 for a token of -1)
//   dE[v] = scale sum_{t: tok_t = v} dy[t]  (+ dE[v])   in the order of t, fp32
//
// The forward is a gather of rows, 16 bytes a lane. The backward adds no row to another by
// atomics: it sorts the positions by token, stably, and sums each token's rows in that
// order, so the same call gives the same bits. Both are bound by HBM; the gradient written
// whole is mostly the zeros of the tokens that do not occur.
//
// Measured on one GB300 against the copy rate (6777 GB/s): forward of 16384 tokens, 2048
// columns, fp32 table of 131072 rows, bf16 out 21.0 us for 123 MB (0.87); the gradient of the
// same, written whole, 166 us for 1.14 GB (a memset of the table alone takes 140); added to a
// table of 5003 x 1027, 40009 positions of fp16, 51 us for 117 MB (0.34: the sort takes 10, the
// sums of rows in no order 33, the join 8).
#include <algorithm>
#include <type_traits>

#include "tw_internal.h"
#include "tw_rows.cuh"

namespace tw {

namespace {

// ------------------------------------------------------------------ forward
// A CTA takes 512 vectors of 16 bytes of y, four a thread, all on their way at once: of several
// rows where they are short (32768 rows of 64 bf16 4.9 us, a CTA each 34; 16384 of 2048 19.9
// against 22.3; of 1027 fp16 20 against 28). Two vectors a thread are as fast where rows are
// whole vectors, one a thread takes 1.2 to 1.9 times as long.
constexpr int kFwdThreads = 128, kFwdVecs = 4;

// per_row: threads' vectors of a row (off 16 bytes whole warps of them, since store_any wants a
// warp's in one row); rows: of a CTA
template <int DT, int WT, bool VEC>
__global__ void __launch_bounds__(kFwdThreads) embed_fwd_kernel(const EmbedFwdArgs a, int per_row, int rows) {
  using S = typename Elem<DT>::S;
  constexpr int E = Elem<DT>::E;
  pdl_enter();
  const int t0 = blockIdx.x * rows, first = blockIdx.y * kFwdThreads * kFwdVecs;
  int at[kFwdVecs], col[kFwdVecs], tok[kFwdVecs];  // row (-1: none), column, token
#pragma unroll
  for (int k = 0; k < kFwdVecs; ++k) {
    const int i = threadIdx.x + k * kFwdThreads, r = rows == 1 ? 0 : i / per_row;
    at[k] = r < rows && t0 + r < a.T ? t0 + r : -1;
    col[k] = (first + i - r * per_row) * E;
    tok[k] = at[k] >= 0 ? a.tokens[at[k]] : -1;
  }
  constexpr int EW = Elem<WT>::E, NW = E / EW;  // the table's vectors of one of y
  uint4 v[kFwdVecs][NW];
#pragma unroll
  for (int k = 0; k < kFwdVecs; ++k) {
    const bool valid = tok[k] >= 0 && tok[k] < a.V;
    if (!valid && tok[k] != -1) raise_status(a.status, TW_EINVAL);
    const bool careful = tok[k] == 0 || tok[k] == a.V - 1 || a.ldw < 8;
    const auto* row = static_cast<const typename Elem<WT>::S*>(a.w) + static_cast<size_t>(valid ? tok[k] : 0) * a.ldw;
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      const int c = col[k] + q * EW;
      v[k][q] = make_uint4(0, 0, 0, 0);
      if (valid && c < a.d) v[k][q] = VEC ? __ldg(reinterpret_cast<const uint4*>(row + c)) : load_any<WT>(row + c, a.d - c, careful);
    }
  }
#pragma unroll
  for (int k = 0; k < kFwdVecs; ++k) {
    if (at[k] < 0) continue;  // (off 16 bytes the whole warp)
    float2 u[E / 2];
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      float x[EW];
      Elem<WT>::unpack(v[k][q], x);
#pragma unroll
      for (int i = 0; i < EW / 2; ++i) u[q * EW / 2 + i] = make_float2(x[2 * i] * a.scale, x[2 * i + 1] * a.scale);
    }
    const uint4 w = Elem<DT>::pack_pairs(u);
    S* y = static_cast<S*>(a.y) + static_cast<size_t>(at[k]) * a.ldy + col[k];
    if (VEC) {
      if (col[k] < a.d) *reinterpret_cast<uint4*>(y) = w;
    } else {
      store_any<DT>(y, w, a.d - col[k], threadIdx.x & 31);
    }
  }
}

// ------------------------------------------------------------------ backward: rows into registers
// A lane's 8 of a warp's 256 columns of dy's rows, summed into acc in order. VEC: 8 adjacent
// ones, 16 bytes at a time. Else 32 columns apart, so that a warp's accesses are adjacent by
// the element: rows off 16 bytes put together from aligned vectors (tw_rows.cuh) took twice
// the instructions.
constexpr int kCols = 8, kWarpCols = 32 * kCols;

template <int DT, bool VEC>
struct RowSum {
  using S = typename Elem<DT>::S;
  static constexpr int E = VEC ? Elem<DT>::E : 1, NV = kCols / E;
  static constexpr int kStride = VEC ? 1 : 32;  // from a lane's column to its next
  using W = std::conditional_t<VEC, uint4, S>;  // what one load brings
  const EmbedBwdArgs& a;
  int c;        // the lane's first column
  float acc[kCols];
  TW_DEV RowSum(const EmbedBwdArgs& a_, int first) : a(a_), c(first + static_cast<int>(threadIdx.x & 31) * (VEC ? kCols : 1)) {
    clear();
  }
  TW_DEV void clear() {
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
  }
  TW_DEV int col(int i) const { return c + i * kStride; }
  TW_DEV void load(int pos, W (&w)[NV]) const {
    const S* row = static_cast<const S*>(a.dy) + static_cast<size_t>(pos) * a.lddy;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (VEC)
        w[k] = col(k * E) < a.d ? __ldg(reinterpret_cast<const uint4*>(row + col(k * E))) : make_uint4(0, 0, 0, 0);
      else
        w[k] = col(k) < a.d ? __ldg(row + col(k)) : Elem<DT>::put(0.f);
    }
  }
  TW_DEV void add(const W (&w)[NV]) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (VEC) {
        float u[E];
        Elem<DT>::unpack(w[k], u);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[k * E + i] += u[i];
      } else {
        acc[k] += Elem<DT>::get(w[k]);
      }
    }
  }
  // the sum so far to, and another added from, a part of a run: 256 columns a warp, in the
  // lanes' order
  TW_DEV void keep(float* part) const {
    float4* to = reinterpret_cast<float4*>(part) + 2 * (threadIdx.x & 31);
    to[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    to[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
  TW_DEV void join(const float4& p, const float4& q) {
    acc[0] += p.x, acc[1] += p.y, acc[2] += p.z, acc[3] += p.w;
    acc[4] += q.x, acc[5] += q.y, acc[6] += q.z, acc[7] += q.w;
  }
  // n parts, `step` floats apart, in order; N on their way at once
  template <int N>
  TW_DEV void join(const float* part, int n, size_t step) {
    const float4* from = reinterpret_cast<const float4*>(part) + 2 * (threadIdx.x & 31);
    for (int i = 0; i < n; i += N) {
      float4 p[N], q[N];
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (i + k < n) p[k] = from[(i + k) * step / 4], q[k] = from[(i + k) * step / 4 + 1];
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (i + k < n) join(p[k], q[k]);
    }
  }
  // the finished sum of token v, into its row
  TW_DEV void put(int v) const {
    float* out = a.dw + static_cast<size_t>(v) * a.lddw;
    if (VEC && a.vec_out) {
      float4 o[kCols / 4];
#pragma unroll
      for (int k = 0; k < kCols / 4; ++k)
        o[k] = a.add && c + 4 * k < a.d ? reinterpret_cast<const float4*>(out + c)[k] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kCols / 4; ++k)
        if (c + 4 * k < a.d)
          reinterpret_cast<float4*>(out + c)[k] =
              make_float4(fmaf(a.scale, acc[4 * k], o[k].x), fmaf(a.scale, acc[4 * k + 1], o[k].y),
                          fmaf(a.scale, acc[4 * k + 2], o[k].z), fmaf(a.scale, acc[4 * k + 3], o[k].w));
    } else {
      float o[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) o[i] = a.add && col(i) < a.d ? out[col(i)] : 0.f;
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (col(i) < a.d) out[col(i)] = fmaf(a.scale, acc[i], o[i]);
    }
  }
};

// Asks for a warp's columns of row v, which a sum will be added to, in L2.
TW_DEV void prefetch_out(const EmbedBwdArgs& a, int v, int block) {
  const char* out = reinterpret_cast<const char*>(a.dw + static_cast<size_t>(v) * a.lddw + block);
  const int bytes = 4 * min(kWarpCols, a.d - block);
  for (int b = 0; b < bytes; b += 128) prefetch_line(out + b);
  prefetch_line(out + bytes - 1);
}

// Zeros into row v's columns, by `threads` threads.
TW_DEV void zero_row(const EmbedBwdArgs& a, int v, int tid, int threads) {
  float* out = a.dw + static_cast<size_t>(v) * a.lddw;
  if (a.vec_out) {
    for (int c = tid * 4; c < a.d; c += threads * 4) __stcs(reinterpret_cast<float4*>(out + c), make_float4(0.f, 0.f, 0.f, 0.f));
  } else {
    for (int c = tid; c < a.d; c += threads) __stcs(out + c, 0.f);
  }
}

constexpr int kThreads = 256, kWarps = kThreads / 32;  // of the kernels below

// ------------------------------------------------------------------ backward of few tokens
// One launch and no sort: the CTA of position i looks through the tokens; where its own
// occurs before i it has nothing to do, else it sums all rows of the token. The CTAs behind
// those zero the rows of the tokens that do not occur, kFillRows each.
constexpr int kFewTokens = 512, kFillRows = 8;

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) embed_bwd_few_kernel(const EmbedBwdArgs a) {
  __shared__ int tok[kFewTokens];
  __shared__ unsigned same[kFewTokens / 32];
  pdl_enter();
  const int tid = threadIdx.x;
  for (int i = tid; i < a.T; i += kThreads) tok[i] = a.tokens[i];
  for (int i = tid; i < kFewTokens / 32; i += kThreads) same[i] = 0u;
  __syncthreads();
  const int words = (a.T + 31) / 32;
  if (static_cast<int>(blockIdx.x) >= a.T) {  // zeros
    if (blockIdx.y > 0) return;
    const int lo = (blockIdx.x - a.T) * kFillRows, rows = min(kFillRows, a.V - lo);
    for (int i = tid; i < a.T; i += kThreads) {
      const unsigned r = static_cast<unsigned>(tok[i]) - static_cast<unsigned>(lo);
      if (r < static_cast<unsigned>(rows)) atomicOr(&same[r >> 5], 1u << (r & 31));
    }
    __syncthreads();
    for (int r = 0; r < rows; ++r)
      if (!((same[r >> 5] >> (r & 31)) & 1u)) zero_row(a, lo + r, tid, kThreads);
    return;
  }
  const int me = blockIdx.x, mine = tok[me];
  if (mine < 0 || mine >= a.V) {
    if (mine != -1 && tid == 0 && blockIdx.y == 0) raise_status(a.status, TW_EINVAL);
    return;
  }
  for (int i = tid; i < words * 32; i += kThreads) {
    const unsigned m = __ballot_sync(0xFFFFFFFFu, i < a.T && tok[i] == mine);
    if ((i & 31) == 0) same[i >> 5] = m;
  }
  __syncthreads();
  for (int w = 0; w < me >> 5; ++w)
    if (same[w] != 0u) return;
  if (same[me >> 5] & ((1u << (me & 31)) - 1u)) return;
  constexpr int kBatch = 8;  // rows on their way at once
  RowSum<DT, VEC> sum(a, (blockIdx.y * kWarps + (tid >> 5)) * kWarpCols);
  if (sum.c >= a.d) return;
  typename RowSum<DT, VEC>::W w[kBatch][RowSum<DT, VEC>::NV];
  int n = 0;
  for (int word = me >> 5; word < words; ++word)
    for (unsigned m = same[word]; m != 0u;) {  // up to kBatch rows on their way at once
      n = 0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (m != 0u) {
          sum.load(word * 32 + __ffs(m) - 1, w[k]);
          m &= m - 1u;
          ++n;
        }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k < n) sum.add(w[k]);
    }
  sum.put(mine);
}

// ------------------------------------------------------------------ backward: sort
// Positions in the order of (token, position). Each CTA owns `range` tokens (about V / 152, at
// most kMostRange) and needs nothing from the others: it reads all tokens, each warp a stretch,
// counts those below its own (where its part of the result begins) and lists its own in order.
// After a prefix sum over (token, warp) each warp goes through its list and puts it down. A
// warp whose list is full (a stretch of the CTA's tokens alone) reads its stretch again in its
// place. Bound by the instructions of looking at all tokens, some 65 a warp for 128 of them:
// 40009 tokens of 5003 10 us (20 where every group of 128 with one of the CTA's was gone through
// twice, by shuffles), 16384 of 131072 6 us.
constexpr int kSortWarps = 32, kSortThreads = 32 * kSortWarps, kMostRange = 1024, kAhead = 4, kList = 256;

TW_DEV int warp_sum_int(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const EmbedBwdArgs a) {
  // [kSortWarps][range] counts, [range + 1]: where a token's positions begin, [kSortWarps][kList]
  extern __shared__ int count[];
  __shared__ int scan[kSortWarps], below[kSortWarps];
  pdl_enter();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, range = a.range;
  const int lo = blockIdx.x * range;
  const unsigned own_range = min(range, a.V - lo), before = (1u << lane) - 1u;
  // a warp's stretch: groups of 128 positions, four adjacent ones a lane
  const int stretch = (a.T + 4 * kSortThreads - 1) / (4 * kSortThreads) * 128;
  const int begin = min(a.T, warp * stretch), end = min(a.T, begin + stretch);
  const bool whole = (reinterpret_cast<uintptr_t>(a.tokens) & 15u) == 0;
  int4 t[kAhead];
  auto read = [&](int base) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = base + 128 * k + 4 * lane;
      const int* p = a.tokens + i;
      if (whole && i + 4 <= end)
        t[k] = __ldg(reinterpret_cast<const int4*>(p));
      else
        t[k] = make_int4(i < end ? p[0] : -1, i + 1 < end ? p[1] : -1, i + 2 < end ? p[2] : -1, i + 3 < end ? p[3] : -1);
    }
  };
  // (unsigned: any int may stand among the tokens)
  auto own = [&](int v) { return static_cast<unsigned>(v) - static_cast<unsigned>(lo) < own_range; };
  read(begin);
  for (int i = tid; i < kSortWarps * range; i += kSortThreads) count[i] = 0;
  __syncthreads();
  int* mine = count + warp * range;
  int* start = count + kSortWarps * range;
  unsigned* list = reinterpret_cast<unsigned*>(start + range + 1) + warp * kList;  // token - lo | position - begin << 10
  static_assert(kMostRange <= 1 << 10 && (1 << 22) / kSortWarps <= 1 << 22, "an entry's fields");
  int less = 0, listed = 0;  // (listed > kList: not all are)
  bool bad = false;
  for (int base = begin; base < end; base += 128 * kAhead) {
    if (base > begin) read(base);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const unsigned l = lo;
      less += (static_cast<unsigned>(t[k].x) < l) + (static_cast<unsigned>(t[k].y) < l) + (static_cast<unsigned>(t[k].z) < l) +
              (static_cast<unsigned>(t[k].w) < l);
      const bool o[4] = {own(t[k].x), own(t[k].y), own(t[k].z), own(t[k].w)};
      if (!__any_sync(0xFFFFFFFFu, o[0] || o[1] || o[2] || o[3])) continue;
      int at = listed;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const unsigned owned = __ballot_sync(0xFFFFFFFFu, o[q]);
        at += __popc(owned & before);
        listed += __popc(owned);
      }
      if (listed > kList) {
        listed = kList + 1;
        continue;
      }
      const int v[4] = {t[k].x, t[k].y, t[k].z, t[k].w};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (o[q]) list[at++] = static_cast<unsigned>(v[q] - lo) | static_cast<unsigned>(base - begin + 128 * k + 4 * lane + q) << 10;
    }
    if (blockIdx.x == 0) {
      auto out = [&](int v) { return v < -1 || v >= a.V; };
#pragma unroll
      for (int k = 0; k < kAhead; ++k) bad |= out(t[k].x) || out(t[k].y) || out(t[k].z) || out(t[k].w);
    }
  }
  if (bad) raise_status(a.status, TW_EINVAL);
  // what the warp owns, 32 in order at a time, to act(token - lo, position, how many of the token
  // lie before it among them, all of them)
  auto each_owned = [&](auto&& act) {
    __syncwarp();
    auto some = [&](bool here, int v, int i) {
      const unsigned all = __ballot_sync(0xFFFFFFFFu, here);
      if (here) {
        const unsigned peers = __match_any_sync(all, v);
        act(v, i, __popc(peers & before), peers, all);
      }
      __syncwarp();
    };
    if (listed <= kList) {
      for (int i = 0; i < listed; i += 32) {
        const unsigned e = i + lane < listed ? list[i + lane] : 0u;
        some(i + lane < listed, e & 1023u, begin + static_cast<int>(e >> 10));
      }
    } else {
      for (int base = begin; base < end; base += 32) {
        const int v = base + lane < end ? a.tokens[base + lane] : -1;
        if (__any_sync(0xFFFFFFFFu, own(v))) some(own(v), own(v) ? v - lo : 0, base + lane);
      }
    }
  };
  each_owned([&](int v, int, int rank, unsigned peers, unsigned) {
    if (rank == 0) mine[v] += __popc(peers);
  });
  less = warp_sum_int(less);
  if (lane == 0) below[warp] = less;
  __syncthreads();
  // token tid: its total, the prefix over the warps, then over the tokens
  int total = 0;
  if (tid < range) {
#pragma unroll 16
    for (int w = 0; w < kSortWarps; ++w) {
      const int n = count[w * range + tid];
      count[w * range + tid] = total;
      total += n;
    }
  }
  const int inc = warp_inclusive_scan(total);
  if (lane == 31) scan[warp] = inc;
  // which tokens occur: a bit each
  const unsigned occur = __ballot_sync(0xFFFFFFFFu, total > 0);
  if (a.present != nullptr && lane == 0 && 32 * warp < range) a.present[(lo >> 5) + warp] = occur;
  __syncthreads();
  const int at = warp_sum_int(below[lane] + (lane < warp ? scan[lane] : 0)) + inc - total;
  if (tid < range) start[tid] = at;
  if (tid == range - 1) start[range] = at + total;
  if (blockIdx.x == gridDim.x - 1 && tid == kSortThreads - 1) *a.n_valid = at + total;
  __syncthreads();
  each_owned([&](int v, int position, int rank, unsigned peers, unsigned all) {
    const int was = mine[v], slot = start[v] + was + rank;
    __syncwarp(all);
    if (rank == 0) mine[v] = was + __popc(peers);
    if (!TW_CHECKED(slot >= 0 && slot < a.T && position < a.T, a.status)) return;
    a.pos[slot] = position;
    a.key[slot] = lo + v;
    a.run[slot] = make_int2(start[v], start[v + 1]);
  });
}

// ------------------------------------------------------------------ backward: sums
// Each warp takes `chunk` sorted positions (16; short batches 4 or 8), whatever tokens they
// are, and 256 columns: frequent tokens cost no more than rare ones. A run of up to kWhole positions is the warp's that has its
// first, to its end; of a longer one over several chunks the part here is kept: at the chunk's
// head (a run that began before) or its tail (one that begins here and goes on).
//
// Bound by how fast rows in no order come (40009 of 1027 fp16, with the event's 4 us: 37 us for
// 82 MB and the 34 MB added to): two rows a group of copies, four groups a warp, 32 warps an SM.
// 24 warps 41, 40 or more 41 to 43, four rows a group 39, four groups of them 43; loads into
// registers behind an L2 prefetch 53, without it 80. The CTAs behind those zero the rows of
// absent tokens, eight each (16384 tokens of 131072 x 2048, all of it: 172 us; with CTAs of both
// kinds in turn, of 64 rows or of 128 threads 2 to 8 % more).
constexpr int kWhole = 16;  // (1: the join takes twice as long where runs are of 8; 32: sums of short batches 6 us longer)
TW_DEV bool in_parts(const int2& run, int chunk) { return run.y - run.x > kWhole && run.x / chunk != (run.y - 1) / chunk; }

// A warp's 256 columns of rows of dy on their way through shared memory, kBatch rows a group
// of asynchronous copies, kGroups groups. VEC: each lane copies the vectors that it will read.
// Else the aligned vectors that the columns lie in, and a column is read by the element.
template <int DT, bool VEC>
struct RowRing {
  using S = typename Elem<DT>::S;
  static constexpr int E = Elem<DT>::E, NV = kCols / E;         // a lane's vectors of a row
  static constexpr int kBatch = 2, kGroups = NV == 1 ? 4 : 2;
  static constexpr int kRowVecs = 32 * NV + 1;                    // places of a row
  static constexpr int kVecs = kBatch * kGroups * kRowVecs;       // of a warp
  const EmbedBwdArgs& a;
  const S* columns;  // of dy's first row
  uint4* mine;       // the warp's places
  int width, lane;
  TW_DEV uint4* place(int i) const { return mine + i % (kBatch * kGroups) * kRowVecs; }
  // elements from an aligned 16 bytes to row pos's columns
  TW_DEV int lead(int pos) const {
    return static_cast<int>(reinterpret_cast<uintptr_t>(columns) / sizeof(S) + static_cast<unsigned>(pos) * static_cast<unsigned>(a.lddy)) & (E - 1);
  }
  // row `pos` into the place of the block's i-th position
  TW_DEV void copy(int i, int pos) const {
    uint4* to = place(i) + lane;
    const S* from = columns + static_cast<size_t>(pos) * a.lddy;
    if constexpr (VEC) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (lane * kCols + k * E < width) cp_async16(to + k * 32, from + lane * kCols + k * E);
    } else {
      const int before = lead(pos), end = before + width;
      from += lane * E - before;
      const bool careful = pos == 0 || pos == a.T - 1 || a.lddy < 8;  // nothing of the row's neighbours may be read
      if (!careful) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if ((k * 32 + lane) * E < end) cp_async16(to + k * 32, from + k * 32 * E);
        if (lane == 0 && NV * 32 * E < end) cp_async16(to + NV * 32, from + NV * 32 * E);
        return;
      }
      for (int k = 0; (k * 32 + lane) * E < end; ++k)
        for (int q = 0; q < E; ++q) {
          const int c = (k * 32 + lane) * E + q;
          if (c >= before && c < end) reinterpret_cast<S*>(to + k * 32)[q] = from[k * 32 * E + q];
        }
    }
  }
  // (the sums of columns past the last are of whatever is there, and go nowhere)
  TW_DEV void add(int i, int pos, float (&acc)[kCols]) const {
    const uint4* from = place(i);
    if constexpr (VEC) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float u[E];
        Elem<DT>::unpack(from[k * 32 + lane], u);
#pragma unroll
        for (int q = 0; q < E; ++q) acc[k * E + q] += u[q];
      }
    } else {
      const S* e = reinterpret_cast<const S*>(from) + lead(pos) + lane;
#pragma unroll
      for (int k = 0; k < kCols; ++k) acc[k] += Elem<DT>::get(e[k * 32]);
    }
  }
};

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) embed_sum_kernel(const EmbedBwdArgs a, int fills, int parts) {
  extern __shared__ uint4 places[];
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31;
  const int sums = gridDim.x - fills;
  if (static_cast<int>(blockIdx.x) >= sums) {
    const int lo = (blockIdx.x - sums) * kFillRows, hi = min(lo + kFillRows, a.V);
    for (int v = lo; v < hi; ++v)
      if (!((a.present[v >> 5] >> (v & 31)) & 1u)) zero_row(a, v, tid, kThreads);
    return;
  }
  const int id = blockIdx.x * kWarps + (tid >> 5), chunk = id / parts;  // of all warps
  const int n_valid = *a.n_valid, begin = chunk * a.chunk, past = min(begin + a.chunk, n_valid);
  if (begin >= past) return;  // the whole warp
  if (!TW_CHECKED(n_valid <= a.T, a.status)) return;
  const int block = (id - chunk * parts) * kWarpCols, width = min(kWarpCols, a.d - block);
  using Ring = RowRing<DT, VEC>;
  constexpr int kBatch = Ring::kBatch;
  const Ring ring{a, static_cast<const typename Ring::S*>(a.dy) + block, places + (tid >> 5) * Ring::kVecs, width, lane};
  RowSum<DT, VEC> sum(a, block);
  const int2 first_run = a.run[begin], last_run = a.run[past - 1];
  if (!TW_CHECKED(first_run.x <= begin && begin < first_run.y && last_run.x < past && past <= last_run.y && last_run.y <= n_valid, a.status)) return;
  const bool skip = first_run.x < begin && !in_parts(first_run, a.chunk);  // (another warp's)
  const int lo = skip ? min(first_run.y, past) : begin;
  const bool goes_on = last_run.y > past && in_parts(last_run, a.chunk);
  const int n = (goes_on || (skip && first_run.y >= past) ? past : last_run.y) - lo;
  bool head = first_run.x < begin && !skip;
  float* part = a.part + static_cast<size_t>(chunk) * 2 * a.part_ld + block;
  for (int first = 0; first < n; first += 32) {  // 32 keys and positions, a lane each
    const int m = min(32, n - first), at = lo + first + lane;
    int key = lane < m ? a.key[at] : -1, pos = lane < m ? a.pos[at] : 0;
    if (!TW_CHECKED(lane >= m || (key >= 0 && key < a.V && pos >= 0 && pos < a.T), a.status)) key = pos = 0;
    auto fetch = [&](int i) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int p = __shfl_sync(0xFFFFFFFFu, pos, (i + k) & 31);
        if (i + k < m) ring.copy(i + k, p);
      }
      cp_commit();
    };
#pragma unroll
    for (int g = 0; g < Ring::kGroups; ++g) fetch(g * kBatch);
    // where a run ends, or the chunk
    const unsigned ends = __ballot_sync(0xFFFFFFFFu, lane < m && (first + lane + 1 == n || a.run[at].y == at + 1));
    // the rows that a run's sum will be added to, asked for in L2 now
    if (a.add && (ends >> lane & 1u)) prefetch_out(a, key, block);
    for (int i = 0; i < m; i += kBatch) {
      cp_wait<Ring::kGroups - 1>();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (i + k >= m) break;
        ring.add(i + k, __shfl_sync(0xFFFFFFFFu, pos, i + k), sum.acc);
        if (!((ends >> (i + k)) & 1u)) continue;
        const bool tail = first + i + k + 1 == n && goes_on;
        if (head || tail)
          sum.keep(part + (head ? 0 : a.part_ld));
        else
          sum.put(__shfl_sync(0xFFFFFFFFu, key, i + k));
        sum.clear();
        head = false;
      }
      __syncwarp();
      fetch(i + kBatch * Ring::kGroups);
    }
  }
}

// The runs in parts: the tail where the run begins, then the heads of the chunks after it, in
// order. A CTA takes 256 columns of the runs that begin in 32 chunks (a lane each looks for
// one), a warp each; a run of many heads is left to all warps, a stretch of the heads each,
// whose sums are joined in order. (The split goes by the heads' number alone.)
constexpr int kAlone = 16, kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps;

template <int DT, bool VEC>
__global__ void __launch_bounds__(kJoinThreads) embed_join_kernel(const EmbedBwdArgs a) {
  __shared__ float4 sums[kJoinWarps - 1][2][32];
  pdl_enter();
  const int n_valid = *a.n_valid, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, block = blockIdx.y * kWarpCols;
  auto part_of = [&](long chunk) { return a.part + static_cast<size_t>(chunk) * 2 * a.part_ld + block; };
  RowSum<DT, VEC> sum(a, block);
  const long first = static_cast<long>(blockIdx.x) * 32, next = (first + lane + 1) * a.chunk;
  int heads = 0, key = 0;  // chunks after the lane's that begin inside its run
  if (next < n_valid) {
    const int2 run = a.run[next - 1];
    if (run.x >= next - a.chunk && run.y > next && in_parts(run, a.chunk)) heads = static_cast<int>((run.y - next + a.chunk - 1) / a.chunk), key = a.key[next];
    if (!TW_CHECKED(run.y <= n_valid && n_valid <= a.T && key >= 0 && key < a.V, a.status)) heads = 0;
  }
  unsigned few = __ballot_sync(0xFFFFFFFFu, heads > 0 && heads <= kAlone), many = __ballot_sync(0xFFFFFFFFu, heads > kAlone);
  if (a.add && heads > 0 && warp == 0) prefetch_out(a, key, block);
  for (int i = 0; few != 0u; few &= few - 1u, ++i) {
    if (i % kJoinWarps != warp) continue;
    const int q = __ffs(few) - 1, n = __shfl_sync(0xFFFFFFFFu, heads, q), v = __shfl_sync(0xFFFFFFFFu, key, q);
    const float* part = part_of(first + q);
    sum.clear();
    sum.template join<1>(part + a.part_ld, 1, 0);
    sum.template join<4>(part + 2 * a.part_ld, n, 2 * static_cast<size_t>(a.part_ld));
    if (sum.c < a.d) sum.put(v);
  }
  for (; many != 0u; many &= many - 1u) {
    const int q = __ffs(many) - 1, n = __shfl_sync(0xFFFFFFFFu, heads, q), v = __shfl_sync(0xFFFFFFFFu, key, q);
    const int each = (n + kJoinWarps - 1) / kJoinWarps, from = min(n, warp * each), to = min(n, from + each);
    const float* part = part_of(first + q);
    sum.clear();
    if (warp == 0) sum.template join<1>(part + a.part_ld, 1, 0);
    sum.template join<8>(part + static_cast<size_t>(from + 1) * 2 * a.part_ld, to - from, 2 * static_cast<size_t>(a.part_ld));
    if (warp > 0) {
      sums[warp - 1][0][lane] = make_float4(sum.acc[0], sum.acc[1], sum.acc[2], sum.acc[3]);
      sums[warp - 1][1][lane] = make_float4(sum.acc[4], sum.acc[5], sum.acc[6], sum.acc[7]);
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int w = 0; w < kJoinWarps - 1; ++w) sum.join(sums[w][0][lane], sums[w][1][lane]);
      if (sum.c < a.d) sum.put(v);
    }
    __syncthreads();
  }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t size_of(int dtype) { return dtype == TW_F32 ? 4 : 2; }
bool rows16(const void* p, int64_t ld, int dtype) { return on16(p) && ld * static_cast<int64_t>(size_of(dtype)) % 16 == 0; }

template <int DT, int WT>
cudaError_t embed_fwd(const EmbedFwdArgs& a, bool vec, cudaStream_t s) {
  constexpr int per_cta = kFwdThreads * kFwdVecs;
  const int vecs = (a.d + Elem<DT>::E - 1) / Elem<DT>::E, per_row = vec ? vecs : (vecs + 31) / 32 * 32, rows = std::max(1, per_cta / per_row);
  const dim3 grid((a.T + rows - 1) / rows, (per_row + per_cta - 1) / per_cta);
  const cudaError_t e =
      launch(vec ? embed_fwd_kernel<DT, WT, true> : embed_fwd_kernel<DT, WT, false>, grid, dim3(kFwdThreads), 0, s, a, per_row, rows);
  trace_mark(s, "embed_fwd");
  return e;
}

template <int DT, bool VEC>
cudaError_t embed_bwd_as(EmbedBwdArgs a, cudaStream_t s) {
  const unsigned parts = (a.d + kWarpCols - 1) / kWarpCols;  // of a row, a warp each
  const int fill = a.add ? 0 : (a.V + kFillRows - 1) / kFillRows;  // CTAs that zero rows
  cudaError_t e;
  if (a.T <= kFewTokens) {
    e = launch(embed_bwd_few_kernel<DT, VEC>, dim3(a.T + fill, (parts + kWarps - 1) / kWarps), dim3(kThreads), 0, s, a);
    trace_mark(s, "embed_bwd_few");
    return e;
  }
  const int ctas = (a.V + a.range - 1) / a.range;
  const size_t smem = (static_cast<size_t>(kSortWarps + 1) * a.range + 1 + kSortWarps * kList) * sizeof(int);
  e = allow_smem(embed_sort_kernel, smem);
  if (e != cudaSuccess) return e;
  if (a.add) a.present = nullptr;
  e = launch(embed_sort_kernel, dim3(ctas), dim3(kSortThreads), smem, s, a);
  trace_mark(s, "embed_sort");
  if (e != cudaSuccess) return e;
  const int chunks = (a.T + a.chunk - 1) / a.chunk;
  const size_t places = sizeof(uint4) * kWarps * RowRing<DT, VEC>::kVecs;
  e = allow_smem(embed_sum_kernel<DT, VEC>, places);
  if (e != cudaSuccess) return e;
  e = launch(embed_sum_kernel<DT, VEC>, dim3((chunks * parts + kWarps - 1) / kWarps + fill), dim3(kThreads), places, s, a, fill, static_cast<int>(parts));
  trace_mark(s, "embed_sum");
  if (e != cudaSuccess || chunks < 2) return e;
  e = launch(embed_join_kernel<DT, VEC>, dim3((chunks + 31) / 32, parts), dim3(kJoinThreads), 0, s, a);
  trace_mark(s, "embed_join");
  return e;
}
template <int DT>
cudaError_t embed_bwd(const EmbedBwdArgs& a, cudaStream_t s) {
  return rows16(a.dy, a.lddy, DT) && a.d % Elem<DT>::E == 0 ? embed_bwd_as<DT, true>(a, s) : embed_bwd_as<DT, false>(a, s);
}

}  // namespace

constexpr int kMostChunks = 4096;  // whole ones
// Short batches go in chunks of 4 or 8 positions while those are no more warps than this, some
// 40 an SM: a warp's sums are added to their rows one after the other (added, 4096 positions of
// 1027 fp16 19.4 us, 28.5 in chunks of 16; 2000 of 2048 bf16 16.8, 28.3; at 3000 warps 21.8
// and 20.4, at 12000 the same).
constexpr int kFewWarps = 6000;

EmbedBwdPlan embed_bwd_plan(int T, int V, int d) {
  EmbedBwdPlan p{};
  if (T <= kFewTokens) return p;
  // tokens of a sorting CTA: whole words of the bits that say which occur
  p.range = std::min(kMostRange, ((V + 151) / 152 + 31) / 32 * 32);
  p.part_ld = (d + kWarpCols - 1) / kWarpCols * kWarpCols;
  const int parts = p.part_ld / kWarpCols;
  p.chunk = 4;
  while (p.chunk < 16 && T / p.chunk * parts > kFewWarps) p.chunk *= 2;
  while (T / p.chunk > kMostChunks) p.chunk *= 2;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at = (at + bytes + 255) / 256 * 256;
    return was;
  };
  p.key = take(sizeof(int) * static_cast<size_t>(T)), p.pos = take(sizeof(int) * static_cast<size_t>(T));
  p.run = take(sizeof(int2) * static_cast<size_t>(T));
  p.n_valid = take(sizeof(int));
  p.present = take((static_cast<size_t>(V) + kMostRange) / 8);
  // never less than for fewer tokens, whose smaller chunks may be more: whoever has room for T
  // has it for any number below
  p.part = take(sizeof(float) * 2 * static_cast<size_t>(p.part_ld) *
                std::min((T + 3) / 4, std::max(kFewWarps / parts + 2, std::min((T + 15) / 16, kMostChunks + 1))));
  p.bytes = at;
  return p;
}

cudaError_t launch_embed_fwd(const EmbedFwdArgs& a, cudaStream_t s) {
  const bool vec = a.d % 8 == 0 && rows16(a.w, a.ldw, a.wtype) && rows16(a.y, a.ldy, a.dtype);
  switch (a.dtype) {
    case TW_F32: return embed_fwd<TW_F32, TW_F32>(a, vec, s);
    case TW_BF16: return a.wtype == TW_F32 ? embed_fwd<TW_BF16, TW_F32>(a, vec, s) : embed_fwd<TW_BF16, TW_BF16>(a, vec, s);
    default: return a.wtype == TW_F32 ? embed_fwd<TW_F16, TW_F32>(a, vec, s) : embed_fwd<TW_F16, TW_F16>(a, vec, s);
  }
}

cudaError_t launch_embed_bwd(const EmbedBwdArgs& given, void* ws, cudaStream_t s) {
  EmbedBwdArgs a = given;
  const EmbedBwdPlan p = embed_bwd_plan(a.T, a.V, a.d);
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (p.bytes > 0) {
    a.key = reinterpret_cast<int*>(w + p.key), a.pos = reinterpret_cast<int*>(w + p.pos), a.run = reinterpret_cast<int2*>(w + p.run);
    a.n_valid = reinterpret_cast<int*>(w + p.n_valid), a.present = reinterpret_cast<unsigned*>(w + p.present);
    a.part = reinterpret_cast<float*>(w + p.part);
    a.range = p.range, a.chunk = p.chunk, a.part_ld = p.part_ld;
  }
  a.vec_out = a.d % 4 == 0 && rows16(a.dw, a.lddw, TW_F32);
  switch (a.dtype) {
    case TW_F32: return embed_bwd<TW_F32>(a, s);
    case TW_BF16: return embed_bwd<TW_BF16>(a, s);
    default: return embed_bwd<TW_F16>(a, s);
  }
}

}  // namespace tw
