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

#include <type_traits>

#include "tw_gemm.cuh"
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
constexpr int kChunkBytes = 32 * 32 * 2;       // an epilogue warp's 32 rows x 32 columns of fp16
constexpr int kStagingBytes = kEpiWarps * 2 * kChunkBytes;  // two blocks a warp
constexpr int kSmem = kStages * kStageBytes + kStagingBytes + 1024 + 512;
static_assert(kSmem <= 232448, "shared memory per CTA");
constexpr int kGramLog2 = 12;      // E is stored times 2^12: |E| <= 4
constexpr int kPolyLog2 = 10;      // B times 2^10: |B| <= 32

enum Kind { GRAM, SQUARE, APPLY };

// a word's worth of fp16
TW_DEV float2 half2_of(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

struct NsArgs {
  CUtensorMap a, b;          // operands
  const uint16_t *in0, *in1; // what the epilogue reads: SQUARE: E; APPLY: hi and lo
  CUtensorMap out0, out1;    // GRAM: E; SQUARE: B; APPLY: the next hi, and lo
  int tiles_m, tiles_n;      // of one matrix of the result, in 256 x 256 tiles
  int count;                 // matrices
  int rows_a, rows_b;        // rows from one matrix to the next in the operands' maps
  int kb_total;              // K blocks of a tile
  int tiles, whole, ksplit;  // tiles; how many of the first run as one unit, the others in ksplit slices
  int np, mp;                // padded sizes
  float* part;               // [tiles - whole][ksplit][2][kEpiWarps][128][32] fp32
  int* arrived;              // [tiles - whole][2][kEpiWarps], 0 between launches
  int32_t* status;
  float f0, f1;              // GRAM: acc * f0 - f1 on the diagonal; SQUARE: e * f0 + acc * f1;
                             // APPLY: x * f0 + acc * f1
  int last;                  // APPLY: the last step, into out
  // the last step's APPLY: out [rows, cols] of type otype, row stride ldo, transposed or not
  void* out[TW_ORTHO_MOST];
  int64_t ldo;
  int rows, cols, otype, transposed;
  float scale, beta;
};

struct Unit {
  int mat, i, j;             // matrix and tile
  int split, slice;          // the tile's number among those in slices, or -1
  int kb_lo, kb_hi;
};
template <int KIND>
TW_DEV Unit unit_of(const NsArgs& p, int u, int per_mat) {
  Unit r;
  int tile = u;
  r.split = -1, r.slice = 0, r.kb_lo = 0, r.kb_hi = p.kb_total;
  if (u >= p.whole) {
    r.split = (u - p.whole) / p.ksplit;
    r.slice = (u - p.whole) - r.split * p.ksplit;
    tile = p.whole + r.split;
    const int chunk = (p.kb_total + p.ksplit - 1) / p.ksplit;
    r.kb_lo = r.slice * chunk;
    r.kb_hi = min(p.kb_total, r.kb_lo + chunk);
  }
  r.mat = tile / per_mat;
  const int t = tile - r.mat * per_mat;
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
  return r;
}

// The last step's result: 32 x 32 of it, a row a lane, into out's own type and strides.
template <int OT>
TW_DEV void put_out(const NsArgs& p, void* base, int row, int col, const float (&v)[32], uint8_t* staging) {
  using S = typename Elem<OT>::S;
  S* out = static_cast<S*>(base);
  const int lane = threadIdx.x & 31;
  auto one = [&](size_t at, float x) {
    x *= p.scale;
    if (p.beta != 0.f) x = fmaf(p.beta, Elem<OT>::get(out[at]), x);
    out[at] = Elem<OT>::put(x);
  };
  if (p.transposed) {  // the lanes' rows are neighbours
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col + i < p.cols) one(static_cast<size_t>(col + i) * p.ldo + row, v[i]);
    }
    return;
  }
  // through shared memory, so that eight lanes write a row's 32 columns: rows of 128 bytes,
  // 16-byte pieces at piece ^ (row % 8)
  float4* st = reinterpret_cast<float4*>(staging);
#pragma unroll
  for (int q = 0; q < 8; ++q) st[lane * 8 + (q ^ (lane & 7))] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  __syncwarp();
  const int sub = lane >> 3, q = lane & 7, c = col + 4 * q, row0 = row - lane;
  const bool vec = p.ldo % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & (4 * sizeof(S) - 1)) == 0 && c + 4 <= p.cols;
#pragma unroll
  for (int r = sub; r < 32; r += 4) {
    if (row0 + r >= p.rows) break;
    float4 x = st[r * 8 + (q ^ (r & 7))];
    const size_t at = static_cast<size_t>(row0 + r) * p.ldo + c;
    if (vec) {
      x.x *= p.scale, x.y *= p.scale, x.z *= p.scale, x.w *= p.scale;
      using V = std::conditional_t<OT == TW_F32, uint4, uint2>;
      union {
        V w;
        S e[4];
      } u;
      if (p.beta != 0.f) {
        u.w = *reinterpret_cast<const V*>(out + at);
        x.x = fmaf(p.beta, Elem<OT>::get(u.e[0]), x.x), x.y = fmaf(p.beta, Elem<OT>::get(u.e[1]), x.y);
        x.z = fmaf(p.beta, Elem<OT>::get(u.e[2]), x.z), x.w = fmaf(p.beta, Elem<OT>::get(u.e[3]), x.w);
      }
      u.e[0] = Elem<OT>::put(x.x), u.e[1] = Elem<OT>::put(x.y), u.e[2] = Elem<OT>::put(x.z), u.e[3] = Elem<OT>::put(x.w);
      *reinterpret_cast<V*>(out + at) = u.w;
    } else {
      const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < p.cols) one(at + i, y[i]);
    }
  }
  __syncwarp();
}

// A warp's way out: 32 x 32 blocks of the result by TMA from shared memory, each
// block's 64-byte rows in 16-byte pieces at piece ^ ((row / 2) % 4) (the maps'
// 64-byte swizzle). Where the epilogue reads matrices (SQUARE: E, APPLY: hi and lo), a
// block's 16 bytes a lane, four lanes to a row, are asked for a chunk ahead into registers
// and handed to the lanes of their rows through the same buffer. (Row by row from
// registers, 32 rows to an instruction, the accesses alone outlasted the products; with the
// blocks read by TMA a chunk waited 1 us for its own.)
template <int KIND>
struct Blocks {
  static constexpr int kIn = KIND == GRAM ? 0 : KIND == SQUARE ? 1 : 2;
  const NsArgs& p;
  uint8_t* staging;     // this warp's two blocks
  int lane;
  uint4 ahead[kIn > 0 ? kIn * 4 : 1];
  // the chunk at (row0, col) of the stacked matrices
  TW_DEV void ask(int row0, int col) {
    const uint16_t* in[2] = {p.in0, p.in1};
#pragma unroll
    for (int m = 0; m < kIn; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        ahead[4 * m + q] = __ldcg(reinterpret_cast<const uint4*>(in[m] + static_cast<size_t>(row0 + 8 * q + (lane >> 2)) * p.np + col) + (lane & 3));
  }
  // the buffer is free for every lane, and holds what was asked for
  TW_DEV void take() {
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
    if constexpr (kIn > 0) {
#pragma unroll
      for (int m = 0; m < kIn; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q) *piece(staging + m * kChunkBytes, 8 * q + (lane >> 2), lane & 3) = ahead[4 * m + q];
      __syncwarp();
    }
  }
  TW_DEV uint4* piece(uint8_t* block, int row, int q) const {
    return reinterpret_cast<uint4*>(block + row * 64) + (q ^ ((row >> 1) & 3));
  }
  // v: the products' sums of row `row` of the matrix (this lane's), columns [col, col + 32);
  // base: the matrix's first row in the maps
  TW_DEV void put(const Unit& u, int base, int row, int col, float (&v)[32]) {
    uint8_t* b0 = staging;
    uint8_t* b1 = b0 + kChunkBytes;
    if constexpr (KIND == GRAM) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = v[i] * p.f0 - (row == col + i ? p.f1 : 0.f);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 w = *piece(b0, lane, q);
        uint4 l = make_uint4(0, 0, 0, 0);
        if (KIND == APPLY) l = *piece(b1, lane, q);
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
      if (p.last) {
        __syncwarp();  // every lane has read its rows
        void* out = p.out[u.mat];
        if (p.otype == TW_F32) put_out<TW_F32>(p, out, row, col, v, b0);
        else if (p.otype == TW_BF16) put_out<TW_BF16>(p, out, row, col, v, b0);
        else put_out<TW_F16>(p, out, row, col, v, b0);
        return;
      }
    }
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_f16x2_rn(v[2 * i], v[2 * i + 1]);
#pragma unroll
    for (int q = 0; q < 4; ++q) *piece(b0, lane, q) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    const bool mirror = KIND != APPLY && u.i != u.j;
    if constexpr (KIND == APPLY) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 h = half2_of(w[i]);
        w[i] = pack_f16x2_rn(v[2 * i] - h.x, v[2 * i + 1] - h.y);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) *piece(b1, lane, q) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    } else if (mirror) {  // the other side of the diagonal: columns as rows, 64 bytes a warp's store
#pragma unroll
      for (int i = 0; i < 32; ++i)
        reinterpret_cast<uint16_t*>(piece(b1, i, lane >> 3))[lane & 7] = static_cast<uint16_t>(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(&p.out0, b0, col, base + row);
      if (KIND == APPLY) tma_store_2d(&p.out1, b1, col, base + row);
      if (mirror) tma_store_2d(&p.out1, b1, row, base + col);
      bulk_commit();
    }
  }
};

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1) ns_gemm_kernel(const __grid_constant__ NsArgs p) {
  constexpr bool kMN = KIND == GRAM;  // both operands stored [K, MN]
  constexpr uint32_t kIdesc = idesc_bf16_f32(kTile, kTile, kMN, kMN, true);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* tiles = smem_raw + pad;
  uint8_t* staging = tiles + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kStagingBytes);
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
  const int units = p.whole + (p.tiles - p.whole) * p.ksplit;
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
    Blocks<KIND> blocks{p, staging + ew * 2 * kChunkBytes, lane};
    int local = 0;
    for (int n = first; n < units; n += pairs, ++local) {
      const Unit u = unit_of<KIND>(p, n, per_mat);
      const int buf = local & 1;
      const int base = u.mat * (KIND == APPLY ? p.mp : p.np);
      const int row = u.i * kTile + static_cast<int>(rank) * 128 + quarter * 32 + lane, col = u.j * kTile + half * 128;
      const bool split = u.split >= 0;
      // while the products run (a slice may have nothing to finish: its blocks come later)
      if (!split) blocks.ask(base + row - lane, col);
      int done = 0;
      if (lane == 0) done = mbar_wait(tfull + buf, (local >> 1) & 1u, abort_flag, p.status) ? 1 : 0;
      if (!__shfl_sync(0xFFFFFFFFu, done, 0)) break;
      tc_fence_after_sync();
      const uint32_t t0 = tmem_base + static_cast<uint32_t>(buf * kTile + half * 128) + (static_cast<uint32_t>(quarter * 32) << 16);
      bool finish = true;
      // this warp's block of a slice's sums, a column's 32 rows side by side
      auto slot = [&](int slice) {
        return p.part + ((static_cast<size_t>(u.split) * p.ksplit + slice) * 2 * kEpiWarps + rank * kEpiWarps + ew) * (128 * 32) + lane;
      };
      int* arrived = p.arrived + (static_cast<size_t>(u.split) * 2 + rank) * kEpiWarps + ew;
      if (split) {
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
        if (finish) blocks.ask(base + row - lane, col);
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
          if (split) {
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
          blocks.take();
          if (c + 1 < 4) blocks.ask(base + row - lane, col + (c + 1) * 32);
          blocks.put(u, base, row, col + c * 32, v);
        }
        if (split && lane == 0) *arrived = 0;
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(peer_smem_addr(tempty + buf, 0));
    }
    if (lane == 0) bulk_wait_all();
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
  int* arrived;                // counters to clear
  int n_arrived;
  uint16_t *hi, *lo;           // [count][mp][np]
  int mp, np, klog2;
  int first;                   // the launch's first matrix
  bool vec;                    // g's and m's rows are whole vectors of 8 elements on 16 bytes
};

constexpr int kNormBlocks = 304, kNormThreads = 512;

// U at element (r, c); store: writes the new momentum
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
// The same for the 8 elements from c on; vec: rows of whole vectors on 16 bytes. Elements
// past the row are 0.
template <int GT>
TW_DEV void update8(const NsInArgs& a, int mat, int r, int c, bool store, float (&u)[8]) {
  if (!a.vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = c + i < a.cols ? update_of<GT>(a, mat, r, c + i, store) : 0.f;
    return;
  }
  constexpr int E = Elem<GT>::E;
  const uint4* g = reinterpret_cast<const uint4*>(static_cast<const typename Elem<GT>::S*>(a.g[mat]) + static_cast<size_t>(r) * a.ldg + c);
#pragma unroll
  for (int k = 0; k < 8 / E; ++k) {
    float w[E];
    Elem<GT>::unpack(g[k], w);
#pragma unroll
    for (int i = 0; i < E; ++i) u[k * E + i] = w[i];
  }
  if (a.m[mat] == nullptr) return;
  float4* m = reinterpret_cast<float4*>(a.m[mat] + static_cast<size_t>(r) * a.ldm + c);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float4 v = m[k];
    float* x = u + 4 * k;
    if (store) {
      v = make_float4(fmaf(a.mu, v.x, x[0]), fmaf(a.mu, v.y, x[1]), fmaf(a.mu, v.z, x[2]), fmaf(a.mu, v.w, x[3]));
      m[k] = v;
    }
    if (a.nesterov)
      x[0] = fmaf(a.mu, v.x, x[0]), x[1] = fmaf(a.mu, v.y, x[1]), x[2] = fmaf(a.mu, v.z, x[2]), x[3] = fmaf(a.mu, v.w, x[3]);
    else
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
}

// The momentum, and the squares' sums of U.
template <int GT>
__global__ void __launch_bounds__(kNormThreads) ns_norm_kernel(const NsInArgs a) {
  __shared__ NormSums red[kNormThreads / 32];
  pdl_enter();
  const int mat = a.first + blockIdx.y;
  NormSums s = {0.f, 0.f, 0.f};
  const unsigned per_row = (a.cols + 7) / 8;
  const long total = static_cast<long>(a.rows) * per_row, step = static_cast<long>(gridDim.x) * kNormThreads;
  long i = static_cast<long>(blockIdx.x) * kNormThreads + threadIdx.x;
  int r = static_cast<int>(i / per_row), c = static_cast<int>(i - static_cast<long>(r) * per_row);
  const int dr = static_cast<int>(step / per_row), dc = static_cast<int>(step - static_cast<long>(dr) * per_row);
#pragma unroll 2
  for (; i < total; i += step) {
    float u[8];
    update8<GT>(a, mat, r, c * 8, true, u);
#pragma unroll
    for (int k = 0; k < 8; ++k) add_square(s, u[k]);
    r += dr, c += dc;
    if (c >= static_cast<int>(per_row)) c -= per_row, ++r;
  }
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
    for (int k = blockIdx.x * kNormThreads + threadIdx.x; k < a.n_arrived; k += gridDim.x * kNormThreads) a.arrived[k] = 0;
}

// 2^k / |U|_F from the sums, by every CTA (256 threads) in the same order; as two factors, so
// that neither they nor a product by one of them overflows.
TW_DEV float2 start_factor(const NsInArgs& a, int mat, int norm_blocks) {
  __shared__ double sum[256];
  __shared__ float2 factor;
  const int tid = threadIdx.x;
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
      const double f = s > 0.0 ? ldexp(1.0 / sqrt(s), a.klog2) : (s == 0.0 ? 0.0 : s);
      int e = 0;
      if (f > 0.0 && f < 1e300) e = ilogb(f) / 2;
      factor = make_float2(static_cast<float>(ldexp(1.0, e)), static_cast<float>(ldexp(f, -e)));
    }
  }
  __syncthreads();
  return factor;
}

// v as hi + lo, packed pairs
TW_DEV void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16x2_rn(x, y);
  const float2 h = half2_of(hi);
  lo = pack_f16x2_rn(x - h.x, y - h.y);
}

// X0 = U / |U|_F as hi + lo, times 2^klog2, into the padded matrix.
template <int GT>
__global__ void __launch_bounds__(256) ns_start_kernel(const NsInArgs a, int norm_blocks) {
  pdl_enter();
  const int mat = a.first + blockIdx.y;
  const float2 f = start_factor(a, mat, norm_blocks);
  const unsigned per_row = a.np / 8;
  const long total = static_cast<long>(a.mp) * per_row, step = static_cast<long>(gridDim.x) * 256;
  long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
  int r = static_cast<int>(i / per_row), c = static_cast<int>(i - static_cast<long>(r) * per_row);
  const int dr = static_cast<int>(step / per_row), dc = static_cast<int>(step - static_cast<long>(dr) * per_row);
#pragma unroll 2
  for (; i < total; i += step) {
    float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r < a.rows && c * 8 < a.cols) update8<GT>(a, mat, r, c * 8, false, u);
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) split_pair(u[2 * k] * f.x * f.y, u[2 * k + 1] * f.x * f.y, h[k], l[k]);
    const size_t at = (static_cast<size_t>(mat) * a.mp + r) * a.np + c * 8;
    *reinterpret_cast<uint4*>(a.hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(a.lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
    r += dr, c += dc;
    if (c >= static_cast<int>(per_row)) c -= per_row, ++r;
  }
}

// The same for a wide matrix, whose transpose is kept, on 64 x 64 tiles.
template <int GT>
__global__ void __launch_bounds__(256) ns_start_wide_kernel(const NsInArgs a, int norm_blocks) {
  __shared__ float t[64][65];
  pdl_enter();
  const int mat = a.first + blockIdx.z, tid = threadIdx.x;
  const float2 f = start_factor(a, mat, norm_blocks);
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;  // in the padded matrix
  const int lane = tid & 63, first = tid >> 6;
#pragma unroll 4
  for (int i = first; i < 64; i += 4) {
    const int r = c0 + i, c = r0 + lane;  // in g
    t[lane][i] = r < a.rows && c < a.cols ? update_of<GT>(a, mat, r, c, false) * f.x * f.y : 0.f;
  }
  __syncthreads();
  for (int i = tid; i < 64 * 32; i += 256) {
    const int r = i >> 5, c = (i & 31) * 2;
    uint32_t h, l;
    split_pair(t[r][c], t[r][c + 1], h, l);
    const size_t at = (static_cast<size_t>(mat) * a.mp + r0 + r) * a.np + c0 + c;
    *reinterpret_cast<uint32_t*>(a.hi + at) = h;
    *reinterpret_cast<uint32_t*>(a.lo + at) = l;
  }
}

// ------------------------------------------------------------------ host
int up(int n) { return (n + kTile - 1) / kTile * kTile; }

// The most units that run slices of tiles: two for each pair of SMs, or 8 for each tile.
constexpr int kMostSlices = 152;

struct Layout {
  int mp, np, tri, full, slices;
  size_t hi0, hi1, lo, e, b, part, arrived, norms, bytes;
};
Layout layout(int m, int n, int count) {
  Layout l{};
  l.mp = up(std::max(m, n)), l.np = up(std::min(m, n));
  const int t = l.np / kTile;
  l.tri = t * (t + 1) / 2 * count, l.full = l.mp / kTile * t * count;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at = (at + bytes + 1023) / 1024 * 1024;
    return was;
  };
  const size_t x = static_cast<size_t>(count) * l.mp * l.np * 2, s = static_cast<size_t>(count) * l.np * l.np * 2;
  l.hi0 = take(x), l.hi1 = take(x), l.lo = take(x), l.e = take(s), l.b = take(s);
  l.slices = std::min(kMostSlices, 8 * std::max(l.tri, l.full));
  l.part = take(static_cast<size_t>(l.slices) * kTile * kTile * 4);
  l.arrived = take(static_cast<size_t>(l.slices) * 2 * kEpiWarps * 4);
  l.norms = take(static_cast<size_t>(count) * kNormBlocks * 3 * 4);
  l.bytes = at;
  return l;
}

// Which of a product's tiles run whole, in full rounds over the pairs, and in how many
// slices of K the others do. Costs in K blocks (0.33 us): a unit's fill and drain that the
// next one does not hide, and what the last slice of a tile reads of the others.
void split_tiles(NsArgs& p, int pairs, int most) {
  p.whole = p.tiles, p.ksplit = 1;
  const int rounds = p.tiles / pairs;
  long best = static_cast<long>((p.tiles + pairs - 1) / pairs) * (p.kb_total + 1);
  for (int w = rounds; w >= std::max(0, rounds - 1); --w)
    for (int s = 2; s <= std::min(p.kb_total, 8); ++s) {
      const int rest = p.tiles - w * pairs, chunk = (p.kb_total + s - 1) / s;
      if (rest == 0 || rest * s > most || (p.kb_total + chunk - 1) / chunk != s) continue;  // no empty slice
      const long cost = static_cast<long>(w) * (p.kb_total + 1) + static_cast<long>((rest * s + pairs - 1) / pairs) * (chunk + 4) + 4 + 2 * s;
      if (cost < best) best = cost, p.whole = w * pairs, p.ksplit = s;
    }
}

template <int KIND>
cudaError_t run_gemm(NsArgs& p, int most_slices, cudaStream_t s, const char* label) {
  auto kern = ns_gemm_kernel<KIND>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  static int resident = -1;  // the query depends only on the kernel
  if (resident < 0) resident = max_active_clusters(kern, kThreads, kSmem, 2);
  const int most = std::min(resident, device_sm_count() / 2);
  if (most < 1) return cudaErrorInvalidConfiguration;
  p.tiles = (KIND == APPLY ? p.tiles_m * p.tiles_n : p.tiles_n * (p.tiles_n + 1) / 2) * p.count;
  split_tiles(p, most, most_slices);
  const int units = p.whole + (p.tiles - p.whole) * p.ksplit;
  e = launch_clustered(kern, dim3(2 * std::min(units, most)), dim3(kThreads), kSmem, 2, s, p);
  trace_mark(s, label);
  return e;
}

template <int GT>
cudaError_t way_in(NsInArgs& in, bool wide, cudaStream_t s) {
  // 8 rows or columns a thread and more; at most two CTAs an SM
  const long vecs = static_cast<long>(in.rows) * ((in.cols + 7) / 8);
  const int norm_blocks = static_cast<int>(std::min<long>(kNormBlocks, (vecs + kNormThreads - 1) / kNormThreads));
  // matrices that fit L2 together go together; larger ones one after the other, so that the
  // second kernel finds what the first has read and written
  const size_t bytes = static_cast<size_t>(in.rows) * in.cols * ((GT == TW_F32 ? 4 : 2) + (in.m[0] != nullptr ? 4 : 0));
  const int together = bytes * in.count <= (80u << 20) ? in.count : 1;
  for (in.first = 0; in.first < in.count; in.first += together) {
    cudaError_t e = launch(ns_norm_kernel<GT>, dim3(norm_blocks, together), dim3(kNormThreads), 0, s, in);
    trace_mark(s, "ortho_norm");
    if (e != cudaSuccess) return e;
    if (wide) {
      e = launch(ns_start_wide_kernel<GT>, dim3(in.np / 64, in.mp / 64, together), dim3(256), 0, s, in, norm_blocks);
    } else {
      const long n = static_cast<long>(in.mp) * (in.np / 8);
      e = launch(ns_start_kernel<GT>, dim3(static_cast<unsigned>(std::min<long>(152 * 6, (n + 255) / 256)), together), dim3(256), 0, s, in,
                 norm_blocks);
    }
    trace_mark(s, "ortho_start");
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
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
  bool vec = o.n % 8 == 0 && o.ldg * static_cast<int64_t>(o.gtype == TW_F32 ? 4 : 2) % 16 == 0 && o.ldbuf % 4 == 0;
  for (int i = 0; i < o.count; ++i) {
    in.g[i] = o.g[i], in.m[i] = o.buf != nullptr ? o.buf[i] : nullptr;
    vec = vec && ((reinterpret_cast<uintptr_t>(in.g[i]) | reinterpret_cast<uintptr_t>(in.m[i])) & 15u) == 0;
  }
  in.ldg = o.ldg, in.ldm = o.ldbuf, in.gtype = o.gtype, in.count = o.count, in.rows = o.m, in.cols = o.n;
  in.mu = o.mu, in.nesterov = o.nesterov, in.vec = vec;
  in.norms = reinterpret_cast<float*>(ws + l.norms);
  in.arrived = reinterpret_cast<int*>(ws + l.arrived), in.n_arrived = l.slices * 2 * kEpiWarps;
  in.hi = at16(l.hi0), in.lo = at16(l.lo), in.mp = l.mp, in.np = l.np, in.klog2 = k;
  cudaError_t e = o.gtype == TW_F32    ? way_in<TW_F32>(in, wide, s)
                  : o.gtype == TW_BF16 ? way_in<TW_BF16>(in, wide, s)
                                       : way_in<TW_F16>(in, wide, s);
  if (e != cudaSuccess) return e;

  // maps: operands in boxes of 64 x 128 (K-major) and 64 x 64 (MN-major), the epilogues' 32 x 32
  const uint64_t np2 = static_cast<uint64_t>(l.np) * 2;
  const uint64_t xrows = static_cast<uint64_t>(l.mp) * o.count, srows = static_cast<uint64_t>(l.np) * o.count;
  CUtensorMap x_k[2], x_mn[2], x_block[2], lo_block, e_k, b_k, e_block, b_block;
  bool ok = true;
  auto map = [&](CUtensorMap& m, size_t at, uint64_t rows, uint32_t box_cols, uint32_t box_rows) {
    ok = ok && make_tmap_bf16(&m, ws + at, l.np, rows, np2, box_cols, box_rows, box_cols == 32);
  };
  for (int i = 0; i < 2; ++i) {
    const size_t x = i ? l.hi1 : l.hi0;
    map(x_k[i], x, xrows, 64, 128), map(x_mn[i], x, xrows, 64, 64), map(x_block[i], x, xrows, 32, 32);
  }
  map(lo_block, l.lo, xrows, 32, 32);
  map(e_k, l.e, srows, 64, 128), map(b_k, l.b, srows, 64, 128), map(e_block, l.e, srows, 32, 32), map(b_block, l.b, srows, 32, 32);
  if (!ok) return cudaErrorInvalidValue;

  NsArgs p = {};
  p.tiles_m = l.mp / kTile, p.tiles_n = l.np / kTile, p.count = o.count, p.np = l.np, p.mp = l.mp;
  p.part = reinterpret_cast<float*>(ws + l.part), p.arrived = in.arrived, p.status = o.status;
  for (int i = 0; i < o.count; ++i) p.out[i] = o.out[i];
  p.ldo = o.ldo, p.rows = std::max(o.m, o.n), p.cols = std::min(o.m, o.n), p.otype = o.otype, p.transposed = wide;
  p.scale = static_cast<float>(std::ldexp(static_cast<double>(o.scale), -k)), p.beta = o.beta;
  for (int step = 0; step < o.steps; ++step) {
    const double a = o.coef[3 * step], b = o.coef[3 * step + 1], c = o.coef[3 * step + 2];
    const double t = step >= 3 ? 1.0 : 0.0, q0 = a + b * t + c * t * t, q1 = b + 2.0 * c * t;
    const int at = step & 1;
    p.a = p.b = x_mn[at], p.out0 = p.out1 = e_block;
    p.rows_a = p.rows_b = l.mp, p.kb_total = l.mp / kBK;
    p.f0 = std::ldexp(1.f, kGramLog2 - 2 * k), p.f1 = static_cast<float>(std::ldexp(t, kGramLog2));
    e = run_gemm<GRAM>(p, l.slices, s, "ortho_gram");
    if (e != cudaSuccess) return e;

    p.a = p.b = e_k, p.in0 = at16(l.e), p.out0 = p.out1 = b_block;
    p.rows_a = p.rows_b = l.np, p.kb_total = l.np / kBK;
    p.f0 = static_cast<float>(std::ldexp(q1, kPolyLog2 - kGramLog2));
    p.f1 = static_cast<float>(std::ldexp(c, kPolyLog2 - 2 * kGramLog2));
    e = run_gemm<SQUARE>(p, l.slices, s, "ortho_square");
    if (e != cudaSuccess) return e;

    p.a = x_k[at], p.b = b_k, p.in0 = at16(at ? l.hi1 : l.hi0), p.in1 = at16(l.lo), p.out0 = x_block[at ^ 1], p.out1 = lo_block;
    p.rows_a = l.mp;
    p.last = step + 1 == o.steps;
    p.f0 = static_cast<float>(q0), p.f1 = std::ldexp(1.f, -kPolyLog2);
    e = run_gemm<APPLY>(p, l.slices, s, "ortho_apply");
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace tw
