// Orthogonalised updates of weight matrices: momentum, then Newton-Schulz products that
// bring every singular value of the update near 1 (tw_orthogonalize).
//
//   M' = mu M + G;  U = G + mu M' (or M');  X0 = U / |U|_F
//   X <- a X + X (b A + c A^2),  A = X^T X            (once per step)
//   out = beta out + scale X
//
// X is kept with its longer side as rows ([m, n], m >= n; a wide matrix is transposed on
// the way in and out), padded with zeros to 256 x 256 tiles, which the products keep zero.
// Three products a step on the tensor cores, each on CTA pairs (tcgen05.mma.cta_group::2,
// 256 x 256 units, TMEM double-buffered, TMA ring):
//
//   gram    E = X^T X - t I     the lower triangle's tiles, stored on both sides
//   square  B = q1 E + c E^2    the same
//   apply   X' = q0 X + X B
//
// with q0 = a + b t + c t^2, q1 = b + 2 c t: the step's polynomial written around t. Any t
// gives the same X'. With t = 1 once the singular values have come near 1 (from the fourth
// step on) the terms are small instead of cancelling (3.44 - 4.78 + 2.03 at 1), and so are
// their roundings.
//
// Operands of the products are fp16 (11 bits; bf16's 8 leave errors of 1e-2) scaled by
// powers of two into its range, sums fp32 in TMEM. X itself is kept as hi + lo, two fp16
// of 22 bits: the products read hi, the term q0 X reads both. Roundings of X would
// otherwise be amplified as the small singular values are (up to 3.44 a step), while in
// X B they meet B's small rows. Against the definition in 64 bits, in the 2-norm: 4e-4 to
// 1.3e-3 for spectra over up to four decades (hi alone: up to 2.4e-2).
#include <cuda.h>

#include <algorithm>
#include <cmath>

#include "tw_internal.h"
#include "tw_rows.cuh"

namespace tw {

namespace {

constexpr int kTile = 256;         // rows and columns of a unit; workspace matrices are whole tiles
constexpr int kBK = 64;            // K of a stage
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;       // two per TMEM lane quarter, 128 columns each
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kOperandBytes = 128 * kBK * 2;  // a CTA's 128 rows of A, or its half of B's
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kSmem = kStages * kStageBytes + 1024 + 256;
constexpr int kGramLog2 = 12;      // E is stored times 2^12: |E| <= 4
constexpr int kPolyLog2 = 10;      // B times 2^10: |B| <= 32

enum Kind { GRAM, SQUARE, APPLY };

// a word's worth of fp16
TW_DEV float2 half2_of(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

struct NsArgs {
  CUtensorMap a, b;
  int tiles_m, tiles_n;      // of one matrix of the result, in 256 x 256 tiles
  int count;                 // matrices
  int rows_a, rows_b;        // rows from one matrix to the next in the operands' maps
  int kb_total, ksplit;      // K blocks; slices of a tile's K loop
  int np, mp;                // padded sizes
  float* part;               // [tiles][ksplit][2][kEpiWarps][128][32] fp32 (ksplit > 1)
  int* arrived;              // [tiles][2][kEpiWarps], 0 between launches
  int32_t* status;
  // epilogues
  uint16_t* d;               // GRAM: E; SQUARE: B; APPLY: the next hi (null in the last step)
  const uint16_t* e;         // SQUARE: E; APPLY: hi
  uint16_t* lo;              // APPLY: lo, read and written in place
  float f0, f1;              // GRAM: acc * f0 - f1 on the diagonal; SQUARE: e * f0 + acc * f1;
                             // APPLY: x * f0 + acc * f1
  // the last step's APPLY: out [rows, cols] of type otype, row stride ldo, transposed or not
  void* out[TW_ORTHO_MOST];
  int64_t ldo;
  int rows, cols, otype, transposed;
  float scale, beta;
};

struct Unit {
  int tile;   // over all matrices
  int mat, i, j, slice, kb_lo, kb_hi;
};
template <int KIND>
TW_DEV Unit unit_of(const NsArgs& p, int u, int per_mat) {
  Unit r;
  r.tile = u / p.ksplit;
  r.slice = u - r.tile * p.ksplit;
  r.mat = r.tile / per_mat;
  const int t = r.tile - r.mat * per_mat;
  if (KIND == APPLY) {
    r.i = t / p.tiles_n;
    r.j = t - r.i * p.tiles_n;
  } else {  // the lower triangle, row by row
    int i = static_cast<int>((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    while (i * (i + 1) / 2 > t) --i;
    r.i = i;
    r.j = t - i * (i + 1) / 2;
  }
  const int chunk = (p.kb_total + p.ksplit - 1) / p.ksplit;
  r.kb_lo = r.slice * chunk;
  r.kb_hi = min(p.kb_total, r.kb_lo + chunk);
  return r;
}

// One output value of the last step.
template <int OT>
TW_DEV void put_out(const NsArgs& p, void* out, size_t at, float x) {
  using S = typename Elem<OT>::S;
  S* o = static_cast<S*>(out) + at;
  float v = p.scale * x;
  if (p.beta != 0.f) v = fmaf(p.beta, Elem<OT>::get(*o), v);
  *o = Elem<OT>::put(v);
}

// 32 columns from `col` on of the result's row `row` (both within the matrix).
template <int KIND>
TW_DEV void emit(const NsArgs& p, const Unit& u, int row, int col, float (&v)[32]) {
  const int ld = p.np;
  if constexpr (KIND == GRAM) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = v[i] * p.f0 - (row == col + i ? p.f1 : 0.f);
  } else {
    const size_t at = (static_cast<size_t>(u.mat) * (KIND == APPLY ? p.mp : p.np) + row) * ld + col;
    const uint4* e = reinterpret_cast<const uint4*>(p.e + at);
    const uint4* lo = reinterpret_cast<const uint4*>(p.lo + at);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 w = e[q];
      uint4 l = make_uint4(0, 0, 0, 0);
      if (KIND == APPLY) l = lo[q];
      const uint32_t h[4] = {w.x, w.y, w.z, w.w}, m[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float2 x = half2_of(h[k]);
        if (KIND == APPLY) x = add2(x, half2_of(m[k]));
        const int i = 8 * q + 2 * k;
        v[i] = fmaf(v[i], p.f1, x.x * p.f0);
        v[i + 1] = fmaf(v[i + 1], p.f1, x.y * p.f0);
      }
    }
  }
  if constexpr (KIND == APPLY) {
    if (p.d == nullptr) {
      void* out = p.out[u.mat];
      if (row >= p.rows) return;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (col + i >= p.cols) break;
        const size_t at = p.transposed ? static_cast<size_t>(col + i) * p.ldo + row
                                       : static_cast<size_t>(row) * p.ldo + col + i;
        if (p.otype == TW_F32) put_out<TW_F32>(p, out, at, v[i]);
        else if (p.otype == TW_BF16) put_out<TW_BF16>(p, out, at, v[i]);
        else put_out<TW_F16>(p, out, at, v[i]);
      }
      return;
    }
  }
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack_f16x2_rn(v[2 * i], v[2 * i + 1]);
  const size_t base = static_cast<size_t>(u.mat) * (KIND == APPLY ? p.mp : p.np);
  uint4* d = reinterpret_cast<uint4*>(p.d + (base + row) * ld + col);
#pragma unroll
  for (int q = 0; q < 4; ++q) d[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  if constexpr (KIND == APPLY) {
    uint4* lo = reinterpret_cast<uint4*>(p.lo + (base + row) * ld + col);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 h = half2_of(w[i]);
      w[i] = pack_f16x2_rn(v[2 * i] - h.x, v[2 * i + 1] - h.y);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) lo[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  } else if (u.i != u.j) {  // the other side of the diagonal: 32 rows' worth of a column at once
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      p.d[(base + col + 2 * i) * ld + row] = static_cast<uint16_t>(w[i]);
      p.d[(base + col + 2 * i + 1) * ld + row] = static_cast<uint16_t>(w[i] >> 16);
    }
  }
}

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1) ns_gemm_kernel(const __grid_constant__ NsArgs p) {
  constexpr bool kMN = KIND == GRAM;  // both operands stored [K, MN]
  constexpr uint32_t kIdesc = idesc_bf16_f32(kTile, kTile, kMN, kMN, true);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* tiles = smem_raw + pad;
  uint64_t* full = reinterpret_cast<uint64_t*>(tiles + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + b, 1);
      mbar_init(tempty + b, 2 * kEpiWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.a);
    tma_prefetch_desc(&p.b);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  pdl_enter();

  const int per_mat = KIND == APPLY ? p.tiles_m * p.tiles_n : p.tiles_n * (p.tiles_n + 1) / 2;
  const int units = per_mat * p.count * p.ksplit;
  const int pairs = gridDim.x >> 1, first = blockIdx.x >> 1;

  if (warp == 0) {
    if (lane == 0) {  // TMA producer
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      bool ok = true;
      for (int n = first; ok && n < units; n += pairs) {
        const Unit u = unit_of<KIND>(p, n, per_mat);
        const int m0 = u.i * kTile + static_cast<int>(rank) * 128, n0 = u.j * kTile + static_cast<int>(rank) * 128;
        for (int kb = u.kb_lo; kb < u.kb_hi; ++kb) {
          if (!mbar_wait(empty + stage, phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          uint8_t* sa = tiles + stage * kStageBytes;
          uint8_t* sb = sa + kOperandBytes;
          if (rank == 0) mbar_arrive_expect_tx(full + stage, 2 * kStageBytes);
          const uint32_t bar = peer_smem_addr(full + stage, 0);
          const int k0 = kb * kBK;
          if (kMN) {
            const int row = u.mat * p.rows_a + k0;
            tma_load_2d_pair(sa, &p.a, bar, m0, row);
            tma_load_2d_pair(sa + 8192, &p.a, bar, m0 + 64, row);
            tma_load_2d_pair(sb, &p.b, bar, n0, row);
            tma_load_2d_pair(sb + 8192, &p.b, bar, n0 + 64, row);
          } else {
            tma_load_2d_pair(sa, &p.a, bar, k0, u.mat * p.rows_a + m0);
            tma_load_2d_pair(sb, &p.b, bar, k0, u.mat * p.rows_b + n0);
          }
          ++issued;
          if (++stage == kStages) stage = 0, phase ^= 1u;
        }
      }
      if (!ok && rank == 0) {
        for (long i = 0; i < kStages && i < issued; ++i) {
          const long q = issued - 1 - i;
          mbar_wait_drain(full + (q % kStages), static_cast<uint32_t>((q / kStages) & 1));
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {  // MMA issuer, for both CTAs
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = true, issued_any = false;
      for (int n = first; ok && n < units; n += pairs, ++local) {
        const Unit u = unit_of<KIND>(p, n, per_mat);
        const int buf = local & 1;
        if (!mbar_wait(tempty + buf, ((local >> 1) & 1u) ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d0 = tmem_base + static_cast<uint32_t>(buf * kTile);
        for (int kb = u.kb_lo; kb < u.kb_hi; ++kb) {
          if (!mbar_wait(full + stage, phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sa = smem_addr(tiles + stage * kStageBytes), sb = sa + kOperandBytes;
#pragma unroll
          for (int k16 = 0; k16 < kBK / 16; ++k16) {
            const uint64_t ad = kMN ? smem_desc_sw128(sa + k16 * 2048, 8192, 1024) : smem_desc_sw128(sa + k16 * 32, 16, 1024);
            const uint64_t bd = kMN ? smem_desc_sw128(sb + k16 * 2048, 8192, 1024) : smem_desc_sw128(sb + k16 * 32, 16, 1024);
            tc_mma_bf16_pair(d0, ad, bd, kIdesc, kb > u.kb_lo || k16 > 0 ? 1u : 0u);
          }
          issued_any = true;
          tc_commit_pair(empty + stage);
          if (++stage == kStages) stage = 0, phase ^= 1u;
        }
        if (!ok) break;
        tc_commit_pair(tfull + buf);
      }
      if (!ok && issued_any) {
        tc_commit_pair(empty + stage);
        mbar_wait_drain(empty + stage, phase);
      }
    }
  } else {
    const int ew = warp - 2, quarter = warp & 3, half = ew >> 2;
    int local = 0;
    for (int n = first; n < units; n += pairs, ++local) {
      const Unit u = unit_of<KIND>(p, n, per_mat);
      const int buf = local & 1;
      int ok = 0;
      if (lane == 0) ok = mbar_wait(tfull + buf, (local >> 1) & 1u, abort_flag, p.status) ? 1 : 0;
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t t0 = tmem_base + static_cast<uint32_t>(buf * kTile + half * 128) + (static_cast<uint32_t>(quarter * 32) << 16);
      const int row = u.i * kTile + static_cast<int>(rank) * 128 + quarter * 32 + lane, col = u.j * kTile + half * 128;
      bool finish = true;
      // this warp's block of a slice's sums, a column's 32 rows side by side
      auto slot = [&](int slice) {
        return p.part + ((static_cast<size_t>(u.tile) * p.ksplit + slice) * 2 * kEpiWarps + rank * kEpiWarps + ew) * (128 * 32) + lane;
      };
      int* arrived = p.arrived + (static_cast<size_t>(u.tile) * 2 + rank) * kEpiWarps + ew;
      if (p.ksplit > 1) {
        // the warp that finds all other slices' sums here adds them, in the slices' order
        int seen = 0;
        if (lane == 0) seen = *static_cast<volatile int*>(arrived);
        seen = __shfl_sync(0xFFFFFFFFu, seen, 0);
        if (seen != p.ksplit - 1) {
          float* to = slot(u.slice);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(t0 + c * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) __stcg(to + (c * 32 + i) * 32, __uint_as_float(v[i]));
          }
          __threadfence();
          __syncwarp();
          if (lane == 0) seen = atomicAdd(arrived, 1);
          seen = __shfl_sync(0xFFFFFFFFu, seen, 0);
        }
        finish = seen == p.ksplit - 1;
        __threadfence();
      }
      if (finish) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t w[32];
          float v[32];
          tmem_ld32(t0 + c * 32, w);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(w[i]);
          if (p.ksplit > 1) {
            float s[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = 0.f;
            for (int q = 0; q < p.ksplit; ++q) {
              const float* from = slot(q) + c * 32 * 32;
              if (q == u.slice) {
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i] += v[i];
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i] += __ldcg(from + i * 32);
              }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = s[i];
          }
          emit<KIND>(p, u, row, col + c * 32, v);
        }
        if (p.ksplit > 1 && lane == 0) *arrived = 0;
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(peer_smem_addr(tempty + buf, 0));
    }
  }
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ------------------------------------------------------------------ the way in
// |U|_F without overflow or underflow of a square: each value's square goes to one of
// three sums, of values scaled by 2^90 (below 2^-50), 1 and 2^-80 (above 2^40).
struct NormSums {
  float small, mid, big;
};
TW_DEV void add_square(NormSums& s, float v) {
  const float a = fabsf(v);
  if (a > 0x1p40f) {
    const float w = v * 0x1p-80f;
    s.big = fmaf(w, w, s.big);
  } else if (a < 0x1p-50f) {
    const float w = v * 0x1p90f;
    s.small = fmaf(w, w, s.small);
  } else {
    s.mid = fmaf(v, v, s.mid);
  }
}

struct NsInArgs {
  const void* g[TW_ORTHO_MOST];
  float* m[TW_ORTHO_MOST];     // momentum buffers, or null
  int64_t ldg, ldm;
  int gtype, count, rows, cols;  // of g as given
  float mu;
  int nesterov;
  float* norms;                // [count][kNormBlocks][3]
  float2* factor;              // [count]: two factors whose product is 2^k / |U|_F
  int* arrived;                // counters to clear
  int n_arrived;
  uint16_t *hi, *lo;           // [count][mp][np]
  int mp, np, transposed, klog2;
};

constexpr int kNormBlocks = 304, kNormThreads = 512;

template <int GT>
TW_DEV float update_of(const NsInArgs& a, int mat, int r, int c, bool store) {
  using S = typename Elem<GT>::S;
  const float g = Elem<GT>::get(static_cast<const S*>(a.g[mat])[static_cast<size_t>(r) * a.ldg + c]);
  if (a.m[mat] == nullptr) return g;
  float* m = a.m[mat] + static_cast<size_t>(r) * a.ldm + c;
  float v = *m;
  if (store) *m = v = fmaf(a.mu, v, g);
  return a.nesterov ? fmaf(a.mu, v, g) : v;
}

// The momentum, and the squares' sums of U.
template <int GT>
__global__ void __launch_bounds__(kNormThreads) ns_norm_kernel(const NsInArgs a) {
  __shared__ NormSums red[kNormThreads / 32];
  pdl_enter();
  const int mat = blockIdx.y;
  NormSums s = {0.f, 0.f, 0.f};
  for (int r = blockIdx.x; r < a.rows; r += gridDim.x)
    for (int c = threadIdx.x; c < a.cols; c += kNormThreads) add_square(s, update_of<GT>(a, mat, r, c, true));
  s.small = warp_sum(s.small), s.mid = warp_sum(s.mid), s.big = warp_sum(s.big);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kNormThreads / 32; ++w)
      s.small += red[w].small, s.mid += red[w].mid, s.big += red[w].big;
    float* to = a.norms + (static_cast<size_t>(mat) * kNormBlocks + blockIdx.x) * 3;
    to[0] = s.small, to[1] = s.mid, to[2] = s.big;
  }
  if (mat == 0)
    for (int i = blockIdx.x * kNormThreads + threadIdx.x; i < a.n_arrived; i += gridDim.x * kNormThreads) a.arrived[i] = 0;
}

// X0 = U / |U|_F as hi + lo, times 2^klog2, on 64 x 64 tiles of the padded matrix.
template <int GT>
__global__ void __launch_bounds__(256) ns_start_kernel(const NsInArgs a, int norm_blocks) {
  __shared__ float t[64][65];
  __shared__ double sum[256];
  __shared__ float2 factor;
  pdl_enter();
  const int mat = blockIdx.z, tid = threadIdx.x;
  {  // the norm, by every CTA in the same order
    double s = 0.0;
    for (int i = tid; i < norm_blocks; i += 256) {
      const float* n = a.norms + (static_cast<size_t>(mat) * kNormBlocks + i) * 3;
      s += static_cast<double>(n[0]) * 0x1p-180 + static_cast<double>(n[1]) + static_cast<double>(n[2]) * 0x1p160;
    }
    sum[tid] = s;
    __syncthreads();
    if (tid < 32) {
      for (int i = tid + 32; i < 256; i += 32) s += sum[i];
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      if (tid == 0) {
        // 2^k / |U| as two factors, so that neither they nor a product by one overflows
        const double f = s > 0.0 ? ldexp(1.0 / sqrt(s), a.klog2) : (s == 0.0 ? 0.0 : s);
        int e = 0;
        if (f > 0.0 && f < 1e300) e = ilogb(f) / 2;
        factor = make_float2(static_cast<float>(ldexp(1.0, e)), static_cast<float>(ldexp(f, -e)));
      }
    }
    __syncthreads();
  }
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;  // in the padded matrix
  const int lane = tid & 63, first = tid >> 6;
  for (int i = first; i < 64; i += 4) {
    const int r = a.transposed ? c0 + i : r0 + i, c = a.transposed ? r0 + lane : c0 + lane;  // in g
    float v = 0.f;
    if (r < a.rows && c < a.cols) v = update_of<GT>(a, mat, r, c, false) * factor.x * factor.y;
    if (a.transposed)
      t[lane][i] = v;
    else
      t[i][lane] = v;
  }
  __syncthreads();
  for (int i = tid; i < 64 * 32; i += 256) {
    const int r = i >> 5, c = (i & 31) * 2;
    const float x = t[r][c], y = t[r][c + 1];
    const uint32_t h = pack_f16x2_rn(x, y);
    const float2 hv = half2_of(h);
    const size_t at = (static_cast<size_t>(mat) * a.mp + r0 + r) * a.np + c0 + c;
    *reinterpret_cast<uint32_t*>(a.hi + at) = h;
    *reinterpret_cast<uint32_t*>(a.lo + at) = pack_f16x2_rn(x - hv.x, y - hv.y);
  }
}

// ------------------------------------------------------------------ host
int up(int n) { return (n + kTile - 1) / kTile * kTile; }

struct Layout {
  int mp, np, tri, ksplit_most;
  size_t hi0, hi1, lo, e, b, part, arrived, norms, bytes;
};
// K slices of a symmetric product's tiles, so that its units about fill the pairs once.
int slices(int tiles, int kb, int pairs, int most) {
  int best = 1;
  long best_cost = -1;
  for (int s = 1; s <= std::min(kb, most); ++s) {
    const int chunk = (kb + s - 1) / s;
    if ((kb + chunk - 1) / chunk != s) continue;  // no empty slice
    const long rounds = (static_cast<long>(tiles) * s + pairs - 1) / pairs;
    const long cost = rounds * (chunk + 6) + (s > 1 ? 4 : 0);  // in K blocks; 6: a unit's fill and drain
    if (best_cost < 0 || cost < best_cost) best = s, best_cost = cost;
  }
  return best;
}
Layout layout(int m, int n, int count) {
  Layout l{};
  l.mp = up(std::max(m, n)), l.np = up(std::min(m, n));
  const int t = l.np / kTile;
  l.tri = t * (t + 1) / 2 * count;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at = (at + bytes + 1023) / 1024 * 1024;
    return was;
  };
  const size_t x = static_cast<size_t>(count) * l.mp * l.np * 2, s = static_cast<size_t>(count) * l.np * l.np * 2;
  l.hi0 = take(x), l.hi1 = take(x), l.lo = take(x), l.e = take(s), l.b = take(s);
  // at most 16 slices of a tile, and no more units than two rounds of 76 pairs unless the tiles are more
  l.ksplit_most = std::max(1, std::min(16, 160 / l.tri));
  l.part = take(l.ksplit_most > 1 ? static_cast<size_t>(l.tri) * l.ksplit_most * kTile * kTile * 4 : 0);
  l.arrived = take(static_cast<size_t>(l.tri) * 2 * kEpiWarps * 4);
  l.norms = take(static_cast<size_t>(count) * kNormBlocks * 3 * 4);
  l.bytes = at;
  return l;
}

template <int KIND>
cudaError_t run_gemm(NsArgs& p, cudaStream_t s, const char* label) {
  auto kern = ns_gemm_kernel<KIND>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int per_mat = KIND == APPLY ? p.tiles_m * p.tiles_n : p.tiles_n * (p.tiles_n + 1) / 2;
  const long units = static_cast<long>(per_mat) * p.count * p.ksplit;
  static int resident = -1;  // the query depends only on the kernel
  if (resident < 0) resident = max_active_clusters(kern, kThreads, kSmem, 2);
  const int pairs = static_cast<int>(std::min<long>(units, std::min(resident, device_sm_count() / 2)));
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  e = launch_clustered(kern, dim3(2 * pairs), dim3(kThreads), kSmem, 2, s, p);
  trace_mark(s, label);
  return e;
}

}  // namespace

size_t ortho_workspace(int m, int n, int count) { return layout(m, n, count).bytes; }

cudaError_t launch_ortho(const OrthoArgs& o, cudaStream_t s) {
  const Layout l = layout(o.m, o.n, o.count);
  uint8_t* ws = static_cast<uint8_t*>(o.ws);
  auto at16 = [&](size_t off) { return reinterpret_cast<uint16_t*>(ws + off); };
  const bool wide = o.m < o.n;
  const int k = std::min(14, std::max(0, static_cast<int>(std::lround(0.5 * std::log2(static_cast<double>(o.m) * o.n)))));

  NsInArgs in = {};
  for (int i = 0; i < o.count; ++i) in.g[i] = o.g[i], in.m[i] = o.buf != nullptr ? o.buf[i] : nullptr;
  in.ldg = o.ldg, in.ldm = o.ldbuf, in.gtype = o.gtype, in.count = o.count, in.rows = o.m, in.cols = o.n;
  in.mu = o.mu, in.nesterov = o.nesterov;
  in.norms = reinterpret_cast<float*>(ws + l.norms);
  in.arrived = reinterpret_cast<int*>(ws + l.arrived), in.n_arrived = l.tri * 2 * kEpiWarps;
  in.hi = at16(l.hi0), in.lo = at16(l.lo), in.mp = l.mp, in.np = l.np, in.transposed = wide, in.klog2 = k;
  const int norm_blocks = std::min(o.m, kNormBlocks);
  const dim3 start(l.np / 64, l.mp / 64, o.count);
  cudaError_t e;
  auto both_kernels = [&](auto norm, auto begin) {
    e = launch(norm, dim3(norm_blocks, o.count), dim3(kNormThreads), 0, s, in);
    trace_mark(s, "ortho_norm");
    if (e != cudaSuccess) return;
    e = launch(begin, start, dim3(256), 0, s, in, norm_blocks);
    trace_mark(s, "ortho_start");
  };
  if (o.gtype == TW_F32) both_kernels(ns_norm_kernel<TW_F32>, ns_start_kernel<TW_F32>);
  else if (o.gtype == TW_BF16) both_kernels(ns_norm_kernel<TW_BF16>, ns_start_kernel<TW_BF16>);
  else both_kernels(ns_norm_kernel<TW_F16>, ns_start_kernel<TW_F16>);
  if (e != cudaSuccess) return e;

  const uint64_t np2 = static_cast<uint64_t>(l.np) * 2;
  const uint64_t xrows = static_cast<uint64_t>(l.mp) * o.count, srows = static_cast<uint64_t>(l.np) * o.count;
  CUtensorMap x_k[2], x_mn[2], em, bm;
  for (int i = 0; i < 2; ++i) {
    const uint16_t* x = at16(i ? l.hi1 : l.hi0);
    if (!make_tmap_bf16(&x_k[i], x, l.np, xrows, np2, 64, 128, false) ||
        !make_tmap_bf16(&x_mn[i], x, l.np, xrows, np2, 64, 64, false))
      return cudaErrorInvalidValue;
  }
  if (!make_tmap_bf16(&em, at16(l.e), l.np, srows, np2, 64, 128, false) ||
      !make_tmap_bf16(&bm, at16(l.b), l.np, srows, np2, 64, 128, false))
    return cudaErrorInvalidValue;

  const int pairs = device_sm_count() / 2;
  NsArgs base = {};
  base.tiles_m = l.mp / kTile, base.tiles_n = l.np / kTile, base.count = o.count;
  base.np = l.np, base.mp = l.mp;
  base.part = reinterpret_cast<float*>(ws + l.part), base.arrived = in.arrived;
  base.status = o.status, base.ksplit = 1;
  for (int step = 0; step < o.steps; ++step) {
    const double a = o.coef[3 * step], b = o.coef[3 * step + 1], c = o.coef[3 * step + 2];
    const double t = step >= 3 ? 1.0 : 0.0, q0 = a + b * t + c * t * t, q1 = b + 2.0 * c * t;
    const int at = step & 1;
    NsArgs p = base;
    p.a = p.b = x_mn[at];
    p.rows_a = p.rows_b = l.mp, p.kb_total = l.mp / kBK;
    p.ksplit = slices(l.tri, p.kb_total, pairs, l.ksplit_most);
    p.d = at16(l.e);
    p.f0 = std::ldexp(1.f, kGramLog2 - 2 * k), p.f1 = static_cast<float>(std::ldexp(t, kGramLog2));
    e = run_gemm<GRAM>(p, s, "ortho_gram");
    if (e != cudaSuccess) return e;

    p.a = p.b = em;
    p.rows_a = p.rows_b = l.np, p.kb_total = l.np / kBK;
    p.ksplit = slices(l.tri, p.kb_total, pairs, l.ksplit_most);
    p.d = at16(l.b), p.e = at16(l.e);
    p.f0 = static_cast<float>(std::ldexp(q1, kPolyLog2 - kGramLog2));
    p.f1 = static_cast<float>(std::ldexp(c, kPolyLog2 - 2 * kGramLog2));
    e = run_gemm<SQUARE>(p, s, "ortho_square");
    if (e != cudaSuccess) return e;

    p = base;
    p.a = x_k[at], p.b = bm;
    p.rows_a = l.mp, p.rows_b = l.np, p.kb_total = l.np / kBK;
    const bool last = step + 1 == o.steps;
    p.d = last ? nullptr : at16(at ? l.hi0 : l.hi1);
    p.e = at16(at ? l.hi1 : l.hi0), p.lo = at16(l.lo);
    p.f0 = static_cast<float>(q0), p.f1 = std::ldexp(1.f, -kPolyLog2);
    if (last) {
      for (int i = 0; i < o.count; ++i) p.out[i] = o.out[i];
      p.ldo = o.ldo, p.rows = std::max(o.m, o.n), p.cols = std::min(o.m, o.n), p.otype = o.otype, p.transposed = wide;
      p.scale = static_cast<float>(std::ldexp(static_cast<double>(o.scale), -k)), p.beta = o.beta;
    }
    e = run_gemm<APPLY>(p, s, "ortho_apply");
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace tw
