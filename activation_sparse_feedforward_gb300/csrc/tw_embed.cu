// Token embedding, forward and backward (tw_embedding_fwd, tw_embedding_bwd).
//
//   y[t] = scale E[tok_t]                               (0 for a token of -1)
//   dE[v] = scale sum_{t: tok_t = v} dy[t]  (+ dE[v])   in the order of t, fp32
//
// The forward is a gather of rows, 16 bytes a lane. The backward adds no row to another by
// atomics: it sorts the positions by token, stably, and sums each token's rows in that
// order, so the same call gives the same bits. Both are bound by HBM; the gradient written
// whole is mostly the zeros of the tokens that do not occur.
#include <algorithm>

#include "tw_internal.h"
#include "tw_rows.cuh"

namespace tw {

namespace {

// ------------------------------------------------------------------ forward
constexpr int kFwdThreads = 128, kFwdVecs = 4;  // a CTA's vectors of 16 bytes of y: 512, of one row

// E elements of a table row from column c on, widened
template <int WT, int E, bool VEC>
TW_DEV void load_row(const typename Elem<WT>::S* row, int c, int d, bool careful, float (&v)[E]) {
  constexpr int EW = Elem<WT>::E;
#pragma unroll
  for (int k = 0; k < E / EW; ++k) {
    float u[EW];
    uint4 w = make_uint4(0, 0, 0, 0);
    const int at = c + k * EW;
    if (at < d) w = VEC ? __ldg(reinterpret_cast<const uint4*>(row + at)) : load_any<WT>(row + at, d - at, careful);
    Elem<WT>::unpack(w, u);
#pragma unroll
    for (int i = 0; i < EW; ++i) v[k * EW + i] = u[i];
  }
}

template <int DT, int WT, bool VEC>
__global__ void __launch_bounds__(kFwdThreads) embed_fwd_kernel(const EmbedFwdArgs a) {
  using S = typename Elem<DT>::S;
  constexpr int E = Elem<DT>::E;
  pdl_enter();
  const int t = blockIdx.x, first = blockIdx.y * kFwdThreads * kFwdVecs + threadIdx.x;
  const int tok = a.tokens[t];
  const bool valid = tok >= 0 && tok < a.V;
  if (threadIdx.x == 0 && blockIdx.y == 0 && !valid && tok != -1) raise_status(a.status, TW_EINVAL);
  const auto* row = static_cast<const typename Elem<WT>::S*>(a.w) + static_cast<size_t>(valid ? tok : 0) * a.ldw;
  const bool careful = tok == 0 || tok == a.V - 1 || a.ldw < 8;
  S* y = static_cast<S*>(a.y) + static_cast<size_t>(t) * a.ldy;
  float v[kFwdVecs][E];
#pragma unroll
  for (int k = 0; k < kFwdVecs; ++k) {
    const int c = (first + k * kFwdThreads) * E;
    if (valid && c < a.d) {
      load_row<WT, E, VEC>(row, c, a.d, careful, v[k]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[k][i] = 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < kFwdVecs; ++k) {
    const int c = (first + k * kFwdThreads) * E;
    float2 u[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) u[i] = make_float2(v[k][2 * i] * a.scale, v[k][2 * i + 1] * a.scale);
    const uint4 w = Elem<DT>::pack_pairs(u);
    if (VEC) {
      if (c < a.d) *reinterpret_cast<uint4*>(y + c) = w;
    } else {
      store_any<DT>(y + c, w, a.d - c, threadIdx.x & 31);
    }
  }
}

// ------------------------------------------------------------------ backward: rows into registers
// Columns [c, c + 8) of dy's rows, summed into acc in order; `n` rows at pos[0], pos[1], ...
constexpr int kCols = 8, kBatch = 8;

template <int DT, bool VEC>
struct RowSum {
  using S = typename Elem<DT>::S;
  static constexpr int E = Elem<DT>::E, NV = kCols / E;
  const EmbedBwdArgs& a;
  int c;
  float acc[kCols];
  TW_DEV RowSum(const EmbedBwdArgs& a_, int c_) : a(a_), c(c_) { clear(); }
  TW_DEV void clear() {
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
  }
  TW_DEV void load(int pos, uint4 (&w)[NV]) const {
    const S* row = static_cast<const S*>(a.dy) + static_cast<size_t>(pos) * a.lddy;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int at = c + k * E;
      w[k] = make_uint4(0, 0, 0, 0);
      if (at < a.d)
        w[k] = VEC ? __ldg(reinterpret_cast<const uint4*>(row + at))
                   : load_any<DT>(row + at, a.d - at, pos == 0 || pos == a.T - 1 || a.lddy < E);
    }
  }
  TW_DEV void add(const uint4 (&w)[NV]) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float u[E];
      Elem<DT>::unpack(w[k], u);
#pragma unroll
      for (int i = 0; i < E; ++i) acc[k * E + i] += u[i];
    }
  }
  // the finished sum of token v
  TW_DEV void put(int v) {
    float* out = a.dw + static_cast<size_t>(v) * a.lddw + c;
    if (a.vec_out) {
#pragma unroll
      for (int k = 0; k < kCols / 4; ++k) {
        if (c + 4 * k >= a.d) break;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.add) o = reinterpret_cast<const float4*>(out)[k];
        o.x = fmaf(a.scale, acc[4 * k], o.x), o.y = fmaf(a.scale, acc[4 * k + 1], o.y);
        o.z = fmaf(a.scale, acc[4 * k + 2], o.z), o.w = fmaf(a.scale, acc[4 * k + 3], o.w);
        reinterpret_cast<float4*>(out)[k] = o;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (c + i < a.d) out[i] = fmaf(a.scale, acc[i], a.add ? out[i] : 0.f);
    }
  }
};

// Zeros into row v's columns, by `threads` threads.
TW_DEV void zero_row(const EmbedBwdArgs& a, int v, int tid, int threads) {
  float* out = a.dw + static_cast<size_t>(v) * a.lddw;
  if (a.vec_out) {
    for (int c = tid * 4; c < a.d; c += threads * 4) __stcs(reinterpret_cast<float4*>(out + c), make_float4(0.f, 0.f, 0.f, 0.f));
  } else {
    for (int c = tid; c < a.d; c += threads) __stcs(out + c, 0.f);
  }
}

constexpr int kThreads = 256;                 // of the kernels below: 2048 columns
constexpr int kBlockCols = kThreads * kCols;

// ------------------------------------------------------------------ backward of few tokens
// One launch and no sort: the CTA of position i looks through the tokens; where its own
// occurs before i it has nothing to do, else it sums all rows of the token. The CTAs behind
// those zero the rows of the tokens that do not occur, kFillRows each.
constexpr int kFewTokens = 512, kFillRows = 64;

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) embed_bwd_few_kernel(const EmbedBwdArgs a) {
  __shared__ int tok[kFewTokens];
  __shared__ unsigned same[kFewTokens / 32];
  pdl_enter();
  const int tid = threadIdx.x;
  for (int i = tid; i < a.T; i += kThreads) tok[i] = a.tokens[i];
  if (tid < kFewTokens / 32) same[tid] = 0u;
  __syncthreads();
  const int words = (a.T + 31) / 32;
  if (static_cast<int>(blockIdx.x) >= a.T) {  // zeros
    if (blockIdx.y > 0) return;
    const int lo = (blockIdx.x - a.T) * kFillRows, rows = min(kFillRows, a.V - lo);
    for (int i = tid; i < a.T; i += kThreads) {
      const int r = tok[i] - lo;
      if (r >= 0 && r < rows) atomicOr(&same[r >> 5], 1u << (r & 31));
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
  RowSum<DT, VEC> sum(a, (blockIdx.y * kThreads + tid) * kCols);
  if (sum.c >= a.d) return;
  uint4 w[kBatch][RowSum<DT, VEC>::NV];
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
// Positions in the order of (token, position). Each CTA owns `range` tokens (at most
// kMostRange) and needs nothing from the others: it reads all tokens, counts those below
// its own (where its part of the result begins) and its own for each warp's stretch of the
// positions, and after a prefix sum over (token, warp) goes through them once more, each
// warp its stretch in order, and puts them down.
constexpr int kSortWarps = 16, kSortThreads = 32 * kSortWarps, kMostRange = 1024, kAhead = 8;

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const EmbedBwdArgs a) {
  extern __shared__ int count[];  // [kSortWarps][range]
  __shared__ int scan[kSortWarps], below[kSortWarps];
  pdl_enter();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, range = a.range;
  const int lo = blockIdx.x * range;
  for (int i = tid; i < kSortWarps * range; i += kSortThreads) count[i] = 0;
  __syncthreads();
  const int stretch = (a.T + kSortThreads - 1) / kSortThreads * 32;
  const int begin = min(a.T, warp * stretch), end = min(a.T, begin + stretch);
  int* mine = count + warp * range;
  int less = 0;
  bool bad = false;
  for (int i = begin + lane; i < end; i += 32 * kAhead) {
    int t[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) t[k] = i + 32 * k < end ? a.tokens[i + 32 * k] : -1;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      bad |= t[k] < -1 || t[k] >= a.V;
      less += t[k] >= 0 && t[k] < lo;
      if (static_cast<unsigned>(t[k] - lo) < static_cast<unsigned>(range) && t[k] < a.V) atomicAdd(mine + (t[k] - lo), 1);
    }
  }
  if (bad && blockIdx.x == 0) raise_status(a.status, TW_EINVAL);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) less += __shfl_xor_sync(0xFFFFFFFFu, less, o);
  if (lane == 0) below[warp] = less;
  __syncthreads();
  // tokens 2 tid and 2 tid + 1: totals, prefixes over the warps, then over the tokens
  int total[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = 2 * tid + k;
    if (r < range)
      for (int w = 0; w < kSortWarps; ++w) {
        const int n = count[w * range + r];
        count[w * range + r] = total[k];
        total[k] += n;
      }
  }
  const int both_ = total[0] + total[1], inc = warp_inclusive_scan(both_);
  if (lane == 31) scan[warp] = inc;
  // which tokens occur: a bit each
  if (a.present != nullptr) {
    const unsigned e = __ballot_sync(0xFFFFFFFFu, total[0] > 0), o = __ballot_sync(0xFFFFFFFFu, total[1] > 0);
    if (lane < 2) {  // lane 0: tokens 64 warp .. + 31, lane 1: the next 32
      const unsigned eh = lane ? e >> 16 : e & 0xFFFFu, oh = lane ? o >> 16 : o & 0xFFFFu;
      unsigned m = 0u;
#pragma unroll
      for (int b = 0; b < 16; ++b) m |= ((eh >> b) & 1u) << (2 * b) | ((oh >> b) & 1u) << (2 * b + 1);
      const int r = 64 * warp + 32 * lane;
      if (r < range) a.present[(lo + r) >> 5] = m;
    }
  }
  __syncthreads();
  int at = inc - both_;
  for (int w = 0; w < kSortWarps; ++w) at += (w < warp ? scan[w] : 0) + below[w];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = 2 * tid + k;
    if (r < range)
      for (int w = 0; w < kSortWarps; ++w) count[w * range + r] += at;
    at += total[k];
  }
  if (blockIdx.x == gridDim.x - 1 && tid == kSortThreads - 1) *a.n_valid = at;
  __syncthreads();
  for (int base = begin; base < end; base += 32 * kAhead) {
    int t[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) t[k] = base + 32 * k + lane < end ? a.tokens[base + 32 * k + lane] : -1;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool own = static_cast<unsigned>(t[k] - lo) < static_cast<unsigned>(range) && t[k] < a.V;
      const unsigned act = __ballot_sync(0xFFFFFFFFu, own);
      if (act == 0u) continue;
      if (own) {
        const unsigned peers = __match_any_sync(act, t[k]);
        int* n = mine + (t[k] - lo);
        const int slot = *n + __popc(peers & ((1u << lane) - 1u));
        __syncwarp(act);
        if (lane == __ffs(peers) - 1) *n += __popc(peers);
        a.pos[slot] = base + 32 * k + lane;
        a.key[slot] = t[k];
      }
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------ backward: sums
// A CTA takes `chunk` sorted positions, whatever tokens they are, so that frequent tokens
// cost no more than rare ones. Runs that begin and end in the chunk are finished; of the
// others the part here is kept: at the chunk's head (a run that began before) or its tail
// (one that begins here and goes on). The CTAs behind those zero the rows of absent tokens.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const EmbedBwdArgs a, int sum_ctas) {
  __shared__ int key[kEmbedMostChunk], pos[kEmbedMostChunk];
  pdl_enter();
  const int tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) >= sum_ctas) {
    if (blockIdx.y > 0) return;
    const int lo = (blockIdx.x - sum_ctas) * kFillRows, hi = min(lo + kFillRows, a.V);
    for (int v = lo; v < hi; ++v)
      if (!((a.present[v >> 5] >> (v & 31)) & 1u)) zero_row(a, v, tid, kThreads);
    return;
  }
  const int n_valid = *a.n_valid, lo = blockIdx.x * a.chunk, n = min(a.chunk, n_valid - lo);
  if (n <= 0) return;
  const bool from_before = lo > 0 && a.key[lo - 1] == a.key[lo];
  const bool goes_on = lo + n < n_valid && a.key[lo + n] == a.key[lo + n - 1];
  for (int i = tid; i < n; i += kThreads) key[i] = a.key[lo + i], pos[i] = a.pos[lo + i];
  __syncthreads();
  RowSum<DT, VEC> sum(a, (blockIdx.y * kThreads + tid) * kCols);
  if (sum.c >= a.d) return;
  bool head = from_before;
  for (int i = 0; i < n; i += kBatch) {
    uint4 w[kBatch][RowSum<DT, VEC>::NV];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i + k < n) sum.load(pos[i + k], w[k]);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int j = i + k;
      if (j >= n) break;
      sum.add(w[k]);
      const bool last = j + 1 == n;
      if (!last && key[j + 1] == key[j]) continue;
      if (head || (last && goes_on)) {
        float4* to = reinterpret_cast<float4*>(a.part + (static_cast<size_t>(blockIdx.x) * 2 + (head ? 0 : 1)) * a.part_ld + sum.c);
        to[0] = make_float4(sum.acc[0], sum.acc[1], sum.acc[2], sum.acc[3]);
        to[1] = make_float4(sum.acc[4], sum.acc[5], sum.acc[6], sum.acc[7]);
      } else {
        sum.put(key[j]);
      }
      sum.clear();
      head = false;
    }
  }
}

// The runs over several chunks: the tail where the run begins, then the heads of the chunks
// after it, in order.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const EmbedBwdArgs a) {
  pdl_enter();
  const int n_valid = *a.n_valid, tid = threadIdx.x, lane = tid & 31;
  const int lo = blockIdx.x * a.chunk, next = lo + a.chunk;
  if (next >= n_valid) return;
  const int v = a.key[next];
  // the run begins in this chunk and goes on in the next
  if (a.key[next - 1] != v || (lo > 0 && a.key[lo - 1] == v)) return;
  int heads = 0;  // chunks after this one that begin inside the run
  for (;; heads += 32) {
    const long i = next + static_cast<long>(heads + lane) * a.chunk;
    const unsigned m = __ballot_sync(0xFFFFFFFFu, i < n_valid && a.key[i] == v);
    if (m != 0xFFFFFFFFu) {
      heads += __ffs(~m) - 1;
      break;
    }
  }
  RowSum<DT, VEC> sum(a, (blockIdx.y * kThreads + tid) * kCols);
  if (sum.c >= a.d) return;
  auto add = [&](const float4& p, const float4& q) {
    sum.acc[0] += p.x, sum.acc[1] += p.y, sum.acc[2] += p.z, sum.acc[3] += p.w;
    sum.acc[4] += q.x, sum.acc[5] += q.y, sum.acc[6] += q.z, sum.acc[7] += q.w;
  };
  const float4* tail = reinterpret_cast<const float4*>(a.part + (static_cast<size_t>(blockIdx.x) * 2 + 1) * a.part_ld + sum.c);
  add(tail[0], tail[1]);
  const float* head = a.part + (static_cast<size_t>(blockIdx.x) + 1) * 2 * a.part_ld + sum.c;
#pragma unroll 8
  for (int h = 0; h < heads; ++h) {
    const float4* p = reinterpret_cast<const float4*>(head + static_cast<size_t>(h) * 2 * a.part_ld);
    add(p[0], p[1]);
  }
  sum.put(v);
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t size_of(int dtype) { return dtype == TW_F32 ? 4 : 2; }
bool rows16(const void* p, int64_t ld, int dtype) { return on16(p) && ld * static_cast<int64_t>(size_of(dtype)) % 16 == 0; }

template <int DT, int WT>
cudaError_t embed_fwd(const EmbedFwdArgs& a, bool vec, cudaStream_t s) {
  constexpr int per_cta = kFwdThreads * kFwdVecs * Elem<DT>::E;
  const dim3 grid(a.T, (a.d + per_cta - 1) / per_cta);
  const cudaError_t e = launch(vec ? embed_fwd_kernel<DT, WT, true> : embed_fwd_kernel<DT, WT, false>, grid, dim3(kFwdThreads), 0, s, a);
  trace_mark(s, "embed_fwd");
  return e;
}

template <int DT>
cudaError_t embed_bwd(EmbedBwdArgs a, cudaStream_t s) {
  const bool vec = rows16(a.dy, a.lddy, DT) && a.d % Elem<DT>::E == 0;
  const unsigned blocks = (a.d + kBlockCols - 1) / kBlockCols;
  const int fill = a.add ? 0 : (a.V + kFillRows - 1) / kFillRows;
  cudaError_t e;
  if (a.T <= kFewTokens) {
    // (the fill's CTAs past the first column block have nothing to do)
    e = launch(vec ? embed_bwd_few_kernel<DT, true> : embed_bwd_few_kernel<DT, false>, dim3(a.T + fill, blocks), dim3(kThreads), 0, s, a);
    trace_mark(s, "embed_bwd_few");
    return e;
  }
  const int ctas = (a.V + a.range - 1) / a.range;
  const size_t smem = static_cast<size_t>(kSortWarps) * a.range * sizeof(int);
  e = allow_smem(embed_sort_kernel, smem);
  if (e != cudaSuccess) return e;
  if (a.add) a.present = nullptr;
  e = launch(embed_sort_kernel, dim3(ctas), dim3(kSortThreads), smem, s, a);
  trace_mark(s, "embed_sort");
  if (e != cudaSuccess) return e;
  const int chunks = (a.T + a.chunk - 1) / a.chunk;
  e = launch(vec ? embed_sum_kernel<DT, true> : embed_sum_kernel<DT, false>, dim3(chunks + fill, blocks), dim3(kThreads), 0, s, a, chunks);
  trace_mark(s, "embed_sum");
  if (e != cudaSuccess || chunks < 2) return e;
  e = launch(vec ? embed_join_kernel<DT, true> : embed_join_kernel<DT, false>, dim3(chunks - 1, blocks), dim3(kThreads), 0, s, a);
  trace_mark(s, "embed_join");
  return e;
}

}  // namespace

EmbedBwdPlan embed_bwd_plan(int T, int V, int d) {
  EmbedBwdPlan p{};
  if (T <= kFewTokens) return p;
  // tokens of a sorting CTA: whole words of the bits that say which occur
  p.range = std::min(kMostRange, ((V + 151) / 152 + 31) / 32 * 32);
  p.chunk = 32;
  while (p.chunk < kEmbedMostChunk && T / p.chunk > 4096) p.chunk *= 2;
  p.part_ld = (d + kCols - 1) / kCols * kCols;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at = (at + bytes + 255) / 256 * 256;
    return was;
  };
  p.key = take(sizeof(int) * static_cast<size_t>(T)), p.pos = take(sizeof(int) * static_cast<size_t>(T));
  p.n_valid = take(sizeof(int));
  p.present = take((static_cast<size_t>(V) + kMostRange) / 8);
  p.part = take(sizeof(float) * 2 * static_cast<size_t>(p.part_ld) * ((T + p.chunk - 1) / p.chunk));
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
    a.key = reinterpret_cast<int*>(w + p.key), a.pos = reinterpret_cast<int*>(w + p.pos);
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
