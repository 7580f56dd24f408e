// The distillation loss and its gradient with one small CTA a row, for many short rows, and
// the loss alone for long ones (see tw_logits.cu for when). A row comes from HBM once, through a ring of asynchronous copies,
// for its statistics; for the gradient it is read again, from L2: the rows under way on
// the device, at most 52 KB times eight CTAs an SM, are still there (loads and stores of
// that sweep are marked as the last use).
#pragma once

#include <algorithm>

#include "tw_logits.cuh"

namespace tw {

namespace {

TW_DEV uint4 load_last(const uint4* p) { return __ldcs(p); }
TW_DEV void store_last(uint4* p, uint4 v) { __stcs(p, v); }

// w with -inf at the elements named by bits
template <int DT>
TW_DEV uint4 hide(const uint4& w, uint32_t bits) {
  const uint4 none = no_vector<DT>();
  auto pick = [&](uint32_t v, uint32_t inf, uint32_t b) {
    uint32_t m;
    if constexpr (Elem<DT>::E == 4)
      m = b & 1u ? ~0u : 0u;
    else
      m = (b & 1u ? 0xFFFFu : 0u) | (b & 2u ? 0xFFFF0000u : 0u);
    return (v & ~m) | (inf & m);
  };
  constexpr int kStep = Elem<DT>::E / 4;
  return make_uint4(pick(w.x, none.x, bits), pick(w.y, none.y, bits >> kStep), pick(w.z, none.z, bits >> 2 * kStep),
                    pick(w.w, none.w, bits >> 3 * kStep));
}

constexpr int kRowDepth = 3;  // batches a thread has on their way from HBM

// NT threads; 1024 / NT CTAs an SM. bit_bytes: a byte for each of the row's vectors, which
// says what elements of it are listed. ahead: how many rows later the targets are asked for.
template <int DT, int HARD, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) distill_rows_kernel(const DistillArgs a, int bit_bytes, int ahead) {
  using El = Elem<DT>;
  using S = typename El::S;
  using Ring = RowRing<DT, NT, kRowDepth>;
  constexpr int E = El::E, kWarps = NT / 32;
  extern __shared__ uint4 smem[];
  __shared__ SoftSum stats[kWarps], list;
  __shared__ float shares[kWarps];
  __shared__ Target target;
  __shared__ DistillStat row_stat;
  __shared__ int label_entry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = a.K;
  const size_t row = blockIdx.x;
  uint8_t* bits = reinterpret_cast<uint8_t*>(smem) + Ring::kBytes;
  const List l(bits + bit_bytes, K);
  const float c0 = kLog2e / a.temperature;
  if (K > 0)
    for (int i = tid; i < bit_bytes / 16; i += NT) reinterpret_cast<uint4*>(bits)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) label_entry = -1;
  pdl_enter();

  const S* z = static_cast<const S*>(a.z) + row * a.ldz;
  const Part<DT> p(z, a.V, 0, 1);
  const Ring ring(smem);
  int label = a.labels != nullptr ? a.labels[row] : -1;
  int i_first = -1;
  float t_first = 0.f;
  if (tid < K) i_first = a.t_idx[row * K + tid], t_first = teacher_logit(a, row * K + tid);
  ring.start(p);
  if (K > 0) __syncthreads();  // the marks' places are clear
  if (label < -1 || label >= a.V) {
    if (tid == 0) raise_status(a.status, TW_EINVAL);
    label = -1;
  }

  // Listed tokens leave the sums of the rest: an entry marks its token, and the first to do
  // so owns it; where tokens are listed twice, the lowest entry.
  bool dup = false;
  for (int k = tid; k < K; k += NT) {
    int i = k == tid ? i_first : a.t_idx[row * K + k];
    float t = k == tid ? t_first : teacher_logit(a, row * K + k);
    bool owner = false;
    if (i >= 0 && i < a.V) {
      const int c = i + p.lead, at = c / E;
      const uint32_t bit = 1u << (c % E + at % 4 * 8);
      owner = !(atomicOr(reinterpret_cast<uint32_t*>(bits) + at / 4, bit) & bit);
      l.z[k] = El::get(z[i]);
      if (!owner) dup = true;
    } else {
      if (i != -1) raise_status(a.status, TW_EINVAL);
      i = -1;
      t = neg_inf_f();
    }
    l.idx[k] = owner ? i : -2 - i;  // padding: -1
    l.lp[k] = t > neg_inf_f() ? fmaxf(t / a.temperature, -FLT_MAX) : t;  // a finite logit stays one
    if (owner && i == label) label_entry = k;
  }
  if (K > 0) dup = __syncthreads_or(dup);
  if (dup) lowest_own<NT>(l, K, label, &label_entry, [](int) { return true; });
  if (warp == kWarps - 1) {  // the teacher's distribution, read by the others after the sums
    teacher_distribution(l, K, a.t_rest != nullptr ? a.t_rest[row] : neg_inf_f(), &target);
    if (lane == 0) target.up = a.scale * (a.dloss != nullptr ? a.dloss[row] : 1.f), target.label = label;
    if (lane == 0) target.z_label = label >= 0 ? El::get(z[label]) : 0.f;  // before dz, which may be z
  }
  if (warp == 0 && row + ahead < static_cast<size_t>(a.N)) prefetch_target(a, row + ahead);

  {
    Sums<DT, HARD> sums(c0);
    auto add = [&](uint4 (&r)[kBatch], const int (&j)[kBatch]) {
      if (K > 0) {
        uint32_t m[kBatch], any = 0;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) any |= m[i] = j[i] < p.n ? bits[j[i]] : 0u;
        if (any != 0) {
#pragma unroll
          for (int i = 0; i < kBatch; ++i) r[i] = hide<DT>(r[i], m[i]);
        }
      }
      sums.add(r);
    };
    const bool first = p.template first_edge<NT>(), last = p.template last_edge<NT>();
    const uint4 e0 = first ? p.edge(0) : no_vector<DT>(), e1 = last ? p.edge(p.n - 1) : no_vector<DT>();
    ring.sweep(p, [&](uint4 (&r)[kBatch], int j) {
      const int at[kBatch] = {j, j + NT, j + 2 * NT, j + 3 * NT};
      add(r, at);
    });
    if (first || last) {
      uint4 r[kBatch] = {e0, e1, no_vector<DT>(), no_vector<DT>()};
      const int at[kBatch] = {first ? 0 : p.n, last ? p.n - 1 : p.n, p.n, p.n};
      add(r, at);
    }
    const SoftSum own = join<HARD>(sums.get(), c0);
    if (lane == 0) stats[warp] = own;
    if (warp == 0) {
      const SoftSum of_list = list_sums<HARD, 0>(l, K, c0);
      if (lane == 0) list = of_list;
    }
  }
  __syncthreads();
  {
    const SoftSum rest = join<HARD>(lane < kWarps ? stats[lane] : SoftSum::none(), c0);
    const DistillStat st = row_stat_of<HARD>(rest, list, c0);
    if (tid == 0) row_stat = st;  // for after the sweep, which wants the registers
    if (a.dz != nullptr) {
      S* dz = static_cast<S*>(a.dz) + row * a.lddz;
      Gradient<HARD>(a, st, c0, target).template with<DT>([&](auto f) {
        const uint4* src = reinterpret_cast<const uint4*>(p.at(0));
        auto singly = [&](const uint4& r, int j) {
          const uint4 v = f(r);
          const S* o = reinterpret_cast<const S*>(&v);
          const int c = p.col(j);
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (c + e >= 0 && c + e < a.V) dz[c + e] = o[e];
        };
        if (Part<DT>::lead_of(dz) == p.lead) {  // the same alignment as z's row
          uint4* out = reinterpret_cast<uint4*>(dz + p.col(0));
          in_batches<NT>(p.lo, p.hi, [&](int j, auto all) {
            uint4 r[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              if (all.value || j + i * NT < p.hi) r[i] = load_last(src + j + i * NT);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              if (all.value || j + i * NT < p.hi) store_last(out + j + i * NT, f(r[i]));
          });
        } else {
          store_shifted<DT, NT>(p, dz, p.lo, p.hi, [&](int j) { return src[j]; },
                                [&](int j, int shift) { return shifted<DT>(src[j], src[j + 1], shift); }, f);
        }
        if (p.template first_edge<NT>()) singly(p.edge(0), 0);
        if (p.template last_edge<NT>()) singly(p.edge(p.n - 1), p.n - 1);
      });
    }
  }
  __syncthreads();
  const DistillStat st = row_stat;
  const bool some = target.some;
  const float z_label = target.z_label;
  if (a.dz != nullptr) {  // the listed tokens and the label overwrite what the sweep stored
    S* dz = static_cast<S*>(a.dz) + row * a.lddz;
    const Gradient<HARD> g(a, st, c0, target);
    if (some && !g.zero) {
      for (int k = tid; k < K; k += NT)
        if (l.idx[k] >= 0) dz[l.idx[k]] = El::put(g.listed(st, l, K, k, label, dup));
    }
    if (tid == 0 && label >= 0 && (label_entry < 0 || !some) && !g.zero) dz[label] = El::put(g.at_label(z_label));
  }
  if (a.loss == nullptr) return;
  const float share = warp_sum(
      loss_share(a, st, l, target, NT, tid == 0, tid == 0 && label >= 0, z_label, [](int) { return true; }));
  if (lane == 0) shares[warp] = share;
  __syncthreads();
  if (warp != 0) return;
  const float loss = warp_sum(lane < kWarps ? shares[lane] : 0.f);
  if (lane == 0) a.loss[row] = !some && label < 0 ? 0.f : st.total == 0.f ? __int_as_float(0x7F800000) : loss;
}

template <int DT, int NT>
cudaError_t distill_rows(const DistillArgs& a, cudaStream_t s) {
  const int bit_bytes = a.K > 0 ? (row_vectors(a.V, DT) + 15) / 16 * 16 : 0;
  const size_t smem = RowRing<DT, NT, kRowDepth>::kBytes + bit_bytes + kListBytes * static_cast<size_t>(a.K);
  const int ahead = device_sm_count() * (1024 / NT);
  auto run = [&](auto kern) {
    cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    e = launch(kern, dim3(a.N), dim3(NT), smem, s, a, bit_bytes, ahead);
    trace_mark(s, "distill_rows");
    return e;
  };
  switch (hard_form(a)) {
    case kNoSum: return run(distill_rows_kernel<DT, kNoSum, NT>);
    case 2: return run(distill_rows_kernel<DT, 2, NT>);
    case 4: return run(distill_rows_kernel<DT, 4, NT>);
    default: return run(distill_rows_kernel<DT, kOwnSum, NT>);
  }
}

template <int NT>
cudaError_t distill_rows_any(const DistillArgs& a, cudaStream_t s) {
  return a.dtype == TW_F32    ? distill_rows<TW_F32, NT>(a, s)
         : a.dtype == TW_BF16 ? distill_rows<TW_BF16, NT>(a, s)
                              : distill_rows<TW_F16, NT>(a, s);
}

}  // namespace

}  // namespace tw
