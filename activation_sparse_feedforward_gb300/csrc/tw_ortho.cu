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
// 256 x 256 units, TMEM double-buffered, TMA ring), all steps' in one launch: pairs draw
// units (a tile of a product of a matrix) from one list, and a unit's loads wait until the
// counter of what it reads says that it is there (15 launches had cost a tail each, in
// which most SMs had nothing to do):
//
//   gram    E = X^T X - t I     the lower triangle's tiles, stored on both sides
//   square  B = q1 E + c E^2    the same
//   apply   X' = q0 X + X B
//
// with q0 = a + b t + c t^2, q1 = b + 2 c t: the step's polynomial written around t. Any t
// gives the same X'. With t = 1 the terms are small where singular values are near 1, instead
// of cancelling (3.44 - 4.78 + 2.03), and so are their roundings; but where they are near 0 B is
// -b - c = 2.74, and the rounding of X's hi enters there, which each later step multiplies by
// a = 3.44. So t is 1 in a call's last step alone (from the fourth on), and else 0.
//
// Operands of the products are fp16 (11 bits; bf16's 8 leave errors of 1e-2) scaled by
// powers of two into its range, sums fp32 in TMEM. X itself is kept as hi + lo, two fp16
// of 22 bits: the products read hi, the term q0 X reads both. Roundings of X would
// otherwise be amplified as the small singular values are (up to 3.44 a step), while in
// X B they meet B's small rows. What B's diagonal, its largest elements, loses to fp16 is kept
// in fp32, and apply adds X's columns times that: else the most of the error where X is near
// orthogonal. Relative to the definition in 64 bits, in the Frobenius norm, after five steps
// (tests/test_ortho_roundings.py models these roundings): 0.5e-3 to 1.5e-3 from 64 rows and
// columns on, whatever the rank and for spectra over up to four decades (hi alone: up to 1e-2;
// t = 1 from the fourth step on: 2.6e-3 at rank 1 to 77, and 0.1 after eight). The diagonal costs
// 1 us a step of a small matrix (704 x 256, five steps: 105 us without, 110 with).
//
// Large matrices are bound by the tensor cores under the board's power: on one GB300 three of
// 5632 x 2048, fp32 gradients and momentum, five steps take 1.05 ms for 1.19e12 operations,
// 1130 TFLOP/s over all (0.65 of the sustained 1736): some 110 us are the way in (bytes), and of
// the products' the pairs spend 0.89 in MMAs, at 1340 W and 1.85 GHz. Small ones are bound by
// the latency of 15 products that wait for one another: 704 x 256 takes 110 us, two of
// 1027 x 2500 273 (products of bf16 operands by the library, which keep fewer bits, in a graph with
// the momentum and the norm: 1.40 ms, 72 and 1492 us).
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
constexpr int kStages = 5;
constexpr int kEpiWarps = 8;       // two per TMEM lane quarter, 128 columns each
constexpr int kThreads = 96 + 32 * kEpiWarps;
constexpr int kOperandBytes = 128 * kBK * 2;  // a CTA's 128 rows of A, or its half of B's
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kChunkBytes = 32 * 32 * 2;       // an epilogue warp's 32 rows x 32 columns of fp16
constexpr int kStagingBytes = kEpiWarps * 4 * kChunkBytes;  // two buffers of two blocks a warp
constexpr int kFactorBytes = kEpiWarps * 32 * 4;
constexpr int kSmem = kStages * kStageBytes + kStagingBytes + kFactorBytes + 1024 + 512;
static_assert(kSmem <= 232448, "shared memory per CTA");
constexpr int kGramLog2 = 12;      // E is stored times 2^12: |E| <= 4
constexpr int kPolyLog2 = 10;      // B times 2^10: |B| <= 32

enum Kind { GRAM, SQUARE, APPLY };

// a word's worth of fp16
TW_DEV float2 half2_of(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

constexpr int kMostSteps = 32;

struct NsArgs {
  // operands: X as K-major and MN-major boxes (X alternates between two buffers), E and B
  CUtensorMap x_k[2], x_mn[2], e_k;
  CUtensorMap e_n, b_n;      // as the right-hand operand: boxes of half a unit's columns (SQUARE, APPLY)
  // 32 x 32 blocks that the epilogues read and write: hi, lo, E, B
  CUtensorMap x_block[2], lo_block, e_block, b_block;
  int tiles_m, tiles_n;      // 256 x 256 tiles of X; tiles_n along a side of E and B
  int width[3];              // columns of a unit, by Kind: 256 or 128
  int count, steps;          // matrices, steps
  int np, mp;                // padded sizes
  int slices[3];             // slices of a tile's K loop, by Kind
  int slots;                 // part's and arrived's tiles x slices of one matrix
  float* part;               // [count][slots][2][kEpiWarps][128][32] fp32
  int* arrived;              // [count][slots][2][kEpiWarps], 0 between calls
  int* done;                 // [count][3]: blocks of warps finished, by Kind, over all steps; 0 at first
  int* next;                 // the next unit, 0 at first
  float* diag;               // [count][np]: B's diagonal less its fp16, times 2^kPolyLog2
  int withhold;              // (a test's) blocks that a square waits for and no one writes
  int32_t* status;
  // GRAM: acc * f0 - f1 on the diagonal; SQUARE: e * f0 + acc * f1; APPLY: x * f0 + acc * f1
  float f0[kMostSteps][3], f1[kMostSteps][3];
  // the last step's APPLY: out [rows, cols] of type otype, row stride ldo, transposed or not
  void* out[TW_ORTHO_MOST];
  int64_t ldo;
  int rows, cols, otype, transposed;
  float scale, beta;
};

// A unit: a tile of one product of one matrix in one step, or a slice of its K loop.
struct Unit {
  int step, kind, mat, tile, slice;
};
// tiles of one matrix's product: 256 rows by width columns
TW_DEV int tiles_of(const NsArgs& p, int kind) {
  return (kind == APPLY ? p.tiles_m * p.tiles_n : p.tiles_n * (p.tiles_n + 1) / 2) << (p.width[kind] == 128);
}
// The units in the order in which they are handed out. In a step: every matrix's gram, then
// a matrix's square always one matrix ahead of its apply, so that what a unit waits for was
// handed out well before it. A unit waits only for units before it in this order; whoever
// was given those is running, so the wait ends, however few of the CTAs are resident.
TW_DEV bool unit_at(const NsArgs& p, int n, Unit& u) {
  const int g = tiles_of(p, GRAM) * p.slices[GRAM], q = tiles_of(p, SQUARE) * p.slices[SQUARE], a = tiles_of(p, APPLY) * p.slices[APPLY];
  const int per_step = p.count * (g + q + a);
  u.step = n / per_step;
  if (u.step >= p.steps) return false;
  int r = n - u.step * per_step;
  auto is = [&](int kind, int mat) {
    u.kind = kind, u.mat = mat, u.tile = r / p.slices[kind], u.slice = r - u.tile * p.slices[kind];
  };
  if (r < p.count * g) {
    const int mat = r / g;
    r -= mat * g;
    is(GRAM, mat);
    return true;
  }
  r -= p.count * g;
  for (int i = -1; i < p.count; ++i) {
    if (i + 1 < p.count) {
      if (r < q) {
        is(SQUARE, i + 1);
        return true;
      }
      r -= q;
    }
    if (i >= 0) {
      if (r < a) {
        is(APPLY, i);
        return true;
      }
      r -= a;
    }
  }
  return false;
}
// tile row (of 256) and column (of width)
TW_DEV void tile_at(const NsArgs& p, const Unit& u, int& i, int& j) {
  const int narrow = p.width[u.kind] == 128;
  if (u.kind == APPLY) {
    const int per_row = p.tiles_n << narrow;
    i = u.tile / per_row;
    j = u.tile - i * per_row;
  } else {  // the lower triangle with the whole 256 x 256 blocks of the diagonal, row by row
    const int t = u.tile >> narrow;
    i = static_cast<int>((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    while (i * (i + 1) / 2 > t) --i;
    j = u.tile - (i * (i + 1) / 2 << narrow);
  }
}
TW_DEV void k_blocks(const NsArgs& p, const Unit& u, int& lo, int& hi) {
  const int total = (u.kind == GRAM ? p.mp : p.np) / kBK, chunk = (total + p.slices[u.kind] - 1) / p.slices[u.kind];
  lo = u.slice * chunk;
  hi = min(total, lo + chunk);
}

// `bytes` (a multiple of 16) of shared memory to p, both on 16 bytes, in the thread's bulk group.
TW_DEV void bulk_store(void* p, const void* smem, int bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(p), "r"(smem_addr(smem)), "r"(bytes) : "memory");
}

TW_DEV int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Orders what was written through the generic or async proxy and acquired here before this
// thread's later accesses through either.
TW_DEV void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// What a thread knows to be written: for each kind, 8 bits a matrix, the last step + 1 whose
// inputs it has waited for.
struct Known {
  uint64_t steps[3] = {0, 0, 0};
};
// Waits (one thread, bounded) until all that unit u reads has been written: the apply of the
// step before for a gram, the gram for a square, the square for an apply, of its matrix.
TW_DEV bool wait_inputs(const NsArgs& p, const Unit& u, Known& known, volatile int* abort_flag) {
  const uint64_t steps = u.kind == GRAM ? known.steps[GRAM] : u.kind == SQUARE ? known.steps[SQUARE] : known.steps[APPLY];
  const int at = 8 * u.mat;
  if (static_cast<int>(steps >> at & 255) == u.step + 1) return true;
  const int of = u.kind == GRAM ? APPLY : u.kind == SQUARE ? GRAM : SQUARE;
  const int need = (u.kind == GRAM ? u.step : u.step + 1) * tiles_of(p, of) * 2 * kEpiWarps + (u.kind == SQUARE ? p.withhold : 0);
  const int* done = p.done + u.mat * 3 + of;
  if (ld_acquire(done) < need) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t n = 1; ld_acquire(done) < need; ++n) {
      __nanosleep(40);
      if (*abort_flag) return false;
      if ((n & 31u) == 0 && global_timer_ns() - t0 > TW_WAIT_LIMIT_NS) {
        *abort_flag = 1;
        raise_status(p.status, TW_ETIMEOUT);
        return false;
      }
    }
  }
  fence_proxy_async_all();
  const uint64_t now = (steps & ~(255ull << at)) | static_cast<uint64_t>(u.step + 1) << at;
  if (u.kind == GRAM) known.steps[GRAM] = now;
  else if (u.kind == SQUARE) known.steps[SQUARE] = now;
  else known.steps[APPLY] = now;
  return true;
}

// A wait whose phase the other CTA of the pair completes, with data it wrote before.
TW_DEV bool mbar_try_wait_cluster(uint32_t addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(addr), "r"(parity)
      : "memory");
  return ok != 0;
}
TW_DEV bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  const uint32_t addr = smem_addr(bar);
  if (mbar_try_wait_cluster(addr, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait_cluster(addr, parity)) return true;
    if ((n & 31u) == 0) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > TW_WAIT_LIMIT_NS) {
        *abort_flag = 1;
        raise_status(status, TW_ETIMEOUT);
        return false;
      }
    }
  }
}

// An arrival on the barrier of a CTA of the pair that orders nothing but itself; `after`: a
// value that it waits for.
TW_DEV void mbar_arrive_cluster_relaxed(uint32_t cluster_addr, bool after) {
  asm volatile("{\n\t.reg .u32 t;\n\tand.b32 t, %1, 0;\n\tadd.u32 t, t, %0;\n\t"
               "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [t];\n\t}" ::"r"(cluster_addr),
               "r"(static_cast<uint32_t>(after))
               : "memory");
}

// The units of a pair: one thread of rank 0 draws them and puts each into a ring in both
// CTAs' shared memory; every role of both CTAs takes them from there in turn.
constexpr int kRing = 4;
constexpr int kDrawAhead = 18;  // K blocks before the end of a unit's loads
constexpr int kTakers = (2 + kEpiWarps) + (1 + kEpiWarps);  // rank 0's producer, issuer and warps; rank 1's
struct UnitRing {
  uint64_t full[kRing];    // one arrival
  uint64_t empty[kRing];   // rank 0's: kTakers arrivals
  uint64_t draw;           // rank 0's: its producer is near the end of a unit's loads
  uint2 unit[kRing];       // step | kind | mat | slice (8 bits each), tile; ~0: no more
};
struct Taker {
  UnitRing* ring;
  volatile int* abort_flag;
  int32_t* status;
  int n = 0;
  // whole warps (or one thread that stands for its warp): the next unit; false: no more, or given up
  TW_DEV bool take(Unit& u, bool one_thread) {
    const int slot = n & (kRing - 1);
    const bool ok = mbar_wait_cluster(ring->full + slot, (n / kRing) & 1u, abort_flag, status);
    if (!(one_thread ? ok : __all_sync(0xFFFFFFFFu, ok))) return false;
    const uint2 w = ring->unit[slot];
    ++n;
    u.step = w.x >> 24, u.kind = (w.x >> 16) & 255, u.mat = (w.x >> 8) & 255, u.slice = w.x & 255, u.tile = static_cast<int>(w.y);
    const bool more = w.x != ~0u;
    if (!one_thread) __syncwarp();
    // (relaxed: nothing was written that the place's next owner would have to see; a release
    // at the cluster's scope cost the producer 0.7 us a unit)
    if (one_thread || (threadIdx.x & 31) == 0) mbar_arrive_cluster_relaxed(peer_smem_addr(ring->empty + slot, 0), more);
    return more;
  }
};

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
  fence_proxy_async_smem();  // these accesses before the next block's arrival
  __syncwarp();
}

// A warp's way out: 32 x 32 blocks of the result by TMA, in two buffers of two blocks in
// turn, each block's 64-byte rows in 16-byte pieces at piece ^ ((row / 2) % 4) (the maps'
// 64-byte swizzle). Where the epilogue reads matrices (SQUARE: E, APPLY: hi and lo), their
// blocks arrive in the same places by TMA, the first two before the products are done.
// (Row by row from registers, 32 rows to an instruction, the accesses outlasted the
// products; loads into registers a chunk ahead are waited for by the fence before the
// stores: 2 us a chunk against 0.6.)
template <int KIND>
struct Blocks {
  static constexpr int kIn = KIND == GRAM ? 0 : KIND == SQUARE ? 1 : 2;
  const NsArgs& p;
  const Unit& u;
  uint8_t* staging;     // this warp's 8 KB
  float* factors;       // and 32 numbers: (APPLY) of the chunk's columns of X
  uint64_t* bar;        // [2]
  int turn;             // phases of each that are over: chunk c completes phase turn + c / 2 of its buffer's
  int lane, base;       // base: the matrix's first row in the maps
  bool mirror;          // off the diagonal's blocks: written on its other side too
  TW_DEV uint8_t* buffer(int c) const { return staging + (c & 1) * 2 * kChunkBytes; }
  // lane 0: chunk c's blocks, from row and column of the matrix
  TW_DEV void ask(int c, int row, int col) {
    if constexpr (kIn > 0) {
      uint8_t* b = buffer(c);
      mbar_arrive_expect_tx(bar + (c & 1), kIn * kChunkBytes);
      tma_load_2d(b, KIND == SQUARE ? &p.e_block : &p.x_block[u.step & 1], bar + (c & 1), col, base + row);
      if (KIND == APPLY) tma_load_2d(b + kChunkBytes, &p.lo_block, bar + (c & 1), col, base + row);
    }
  }
  // chunk c's buffer, for every lane: free, or filled with what was asked for
  TW_DEV bool here(int c, volatile int* abort_flag) {
    if constexpr (kIn > 0) return __all_sync(0xFFFFFFFFu, mbar_wait(bar + (c & 1), (turn + (c >> 1)) & 1u, abort_flag, p.status)) != 0;
    // one group a chunk: with the latest one excepted, this buffer's stores have been read
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
    return true;
  }
  TW_DEV uint4* piece(uint8_t* block, int row, int q) const {
    return reinterpret_cast<uint4*>(block + row * 64) + (q ^ ((row >> 1) & 3));
  }
  // v: the products' sums of row `row` of the matrix (this lane's), columns [col, col + 32)
  TW_DEV void put(int c, int row, int col, float (&v)[32]) {
    uint8_t* b0 = buffer(c);
    uint8_t* b1 = b0 + kChunkBytes;
    const float f0 = p.f0[u.step][KIND], f1 = p.f1[u.step][KIND];
    if constexpr (KIND == GRAM) {
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = v[k] * f0 - (row == col + k ? f1 : 0.f);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 w = *piece(b0, lane, q);
        uint4 l = make_uint4(0, 0, 0, 0);
        if (KIND == APPLY) l = *piece(b1, lane, q);
        const uint32_t h[4] = {w.x, w.y, w.z, w.w}, m[4] = {l.x, l.y, l.z, l.w};
        float f[8] = {f0, f0, f0, f0, f0, f0, f0, f0};
        if (KIND == APPLY) {
          const float4 a = reinterpret_cast<const float4*>(factors)[2 * q], b = reinterpret_cast<const float4*>(factors)[2 * q + 1];
          f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float2 x = half2_of(h[k]);
          if (KIND == APPLY) x = add2(x, half2_of(m[k]));
          const int at = 8 * q + 2 * k;
          v[at] = fmaf(v[at], f1, x.x * f[2 * k]);
          v[at + 1] = fmaf(v[at + 1], f1, x.y * f[2 * k + 1]);
        }
      }
    }
    if constexpr (KIND == APPLY) {
      if (u.step + 1 == p.steps) {
        __syncwarp();  // every lane has read its rows
        void* out = p.out[u.mat];
        if (p.otype == TW_F32) put_out<TW_F32>(p, out, row, col, v, b0);
        else if (p.otype == TW_BF16) put_out<TW_BF16>(p, out, row, col, v, b0);
        else put_out<TW_F16>(p, out, row, col, v, b0);
        if (lane == 0) bulk_commit();  // a group a chunk
        return;
      }
    }
    uint32_t w[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) w[k] = pack_f16x2_rn(v[2 * k], v[2 * k + 1]);
    if constexpr (KIND == SQUARE) {
      if (row - lane == col) {  // a block on the diagonal, whose element here is column col + lane
        float lost_here = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float2 h = half2_of(w[k / 2]);
          if (k == lane) lost_here = v[k] - (k % 2 ? h.y : h.x);
        }
        factors[lane] = lost_here;
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) *piece(b0, lane, q) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    if constexpr (KIND == APPLY) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float2 h = half2_of(w[k]);
        w[k] = pack_f16x2_rn(v[2 * k] - h.x, v[2 * k + 1] - h.y);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) *piece(b1, lane, q) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    } else if (mirror) {  // the other side of the diagonal: columns as rows, 64 bytes a warp's store
#pragma unroll
      for (int k = 0; k < 32; ++k)
        reinterpret_cast<uint16_t*>(piece(b1, k, lane >> 3))[lane & 7] = static_cast<uint16_t>(k & 1 ? w[k / 2] >> 16 : w[k / 2]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      const CUtensorMap* to = KIND == GRAM ? &p.e_block : KIND == SQUARE ? &p.b_block : &p.x_block[(u.step & 1) ^ 1];
      tma_store_2d(to, b0, col, base + row);
      if (KIND == APPLY) tma_store_2d(&p.lo_block, b1, col, base + row);
      if (mirror) tma_store_2d(to, b1, row, base + col);
      if (KIND == SQUARE && row == col) bulk_store(p.diag + static_cast<size_t>(u.mat) * p.np + row, factors, 32 * sizeof(float));
      bulk_commit();
    }
  }
};

// One warp's 32 rows of half a unit's columns; false where a bounded wait ran out.
template <int KIND>
TW_DEV bool epilogue(const NsArgs& p, const Unit& u, uint8_t* staging, float* factors, uint64_t* bar, int& turn, uint64_t* tfull,
                     uint32_t parity, uint32_t tmem, int rank, int ew, Known& known, volatile int* abort_flag) {
  const int lane = threadIdx.x & 31, quarter = (ew + 2) & 3, half = ew >> 2;
  const int width = p.width[KIND], chunks = width / 64, slices = p.slices[KIND];
  int ti, tj;
  tile_at(p, u, ti, tj);
  Blocks<KIND> blocks{p, u, staging, factors, bar, turn, lane, u.mat * (KIND == APPLY ? p.mp : p.np), KIND != APPLY && tj * width / kTile != ti};
  const int row = ti * kTile + rank * 128 + quarter * 32 + lane, col = tj * width + half * (width / 2);
  tmem += half * (width / 2) + (static_cast<uint32_t>(quarter * 32) << 16);
  int asked = 0, taken = 0;  // chunks
  auto ask = [&] {
    if (lane == 0) blocks.ask(asked, row, col + asked * 32);
    ++asked;
  };
  auto drained = [&] {  // given up: no copy of this warp's may be under way when its CTA leaves
    if (KIND != GRAM && lane == 0)
      for (; taken < asked; ++taken) mbar_wait_drain(bar + (taken & 1), (turn + (taken >> 1)) & 1u);
    __syncwarp();
    return false;
  };
  int ok = 1;
  if (KIND != GRAM) {
    if (lane == 0) ok = wait_inputs(p, u, known, abort_flag) ? 1 : 0;
    if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) return false;
    if (slices == 1) ask(), ask();  // while the products run (a slice may have nothing to finish)
  }
  // of X's columns, a lane each (read past L1: another SM wrote it, before what lane 0 has waited for)
  auto factor_at = [&](int c) {
    return fmaf(__ldcg(p.diag + static_cast<size_t>(u.mat) * p.np + col + c * 32 + lane), p.f1[u.step][APPLY], p.f0[u.step][APPLY]);
  };
  [[maybe_unused]] float factor = 0.f;
  if constexpr (KIND == APPLY) {
    __syncwarp();
    factor = factor_at(0);
  }
  if (lane == 0) ok = mbar_wait(tfull, parity, abort_flag, p.status) ? 1 : 0;
  if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) return drained();
  tc_fence_after_sync();
  // this warp's block of a slice's sums, a column's 32 rows side by side
  const size_t place = static_cast<size_t>(u.mat) * p.slots + static_cast<size_t>(u.tile) * slices;
  auto slot = [&](int slice) { return p.part + ((place + slice) * 2 * kEpiWarps + rank * kEpiWarps + ew) * (128 * 32) + lane; };
  int* arrived = p.arrived + (place * 2 + rank) * kEpiWarps + ew;
  if (slices > 1) {
    // the warp that finds all other slices' sums here adds them, in the slices' order
    int seen = 0;
    if (lane == 0) seen = ld_acquire(arrived);
    seen = __shfl_sync(0xFFFFFFFFu, seen, 0);
    if (seen != slices - 1) {
      float* to = slot(u.slice);
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        uint32_t v[32];
        tmem_ld32(tmem + c * 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) __stcg(to + (c * 32 + k) * 32, __uint_as_float(v[k]));
      }
      __threadfence();
      __syncwarp();
      if (lane == 0) seen = atomicAdd(arrived, 1);
      seen = __shfl_sync(0xFFFFFFFFu, seen, 0);
    }
    __threadfence();
    if (seen != slices - 1) return true;
    if (KIND != GRAM) ask(), ask();
  }
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    uint32_t w[32];
    float v[32];
    tmem_ld32(tmem + c * 32, w);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(w[k]);
    if (slices > 1) {
      float s[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) s[k] = 0.f;
      for (int q = 0; q < slices; ++q) {
        const float* from = slot(q) + c * 32 * 32;
        if (q == u.slice) {
#pragma unroll
          for (int k = 0; k < 32; ++k) s[k] += v[k];
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) s[k] += __ldcg(from + k * 32);
        }
      }
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = s[k];
    }
    if constexpr (KIND == APPLY) {
      factors[lane] = factor;
      __syncwarp();
      if (c + 1 < chunks) factor = factor_at(c + 1);
    }
    if (!blocks.here(c, abort_flag)) return drained();
    taken = c + 1;
    blocks.put(c, row, col + c * 32, v);
    if (KIND != GRAM && c > 0 && asked < chunks) {  // the buffer of the chunk before: its stores have been read by now
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      ask();
    }
  }
  if (KIND != GRAM) turn += chunks / 2;
  // the tile's writes are there for whoever is told so; the next step reads them
  if (lane == 0) {
    if (slices > 1) *arrived = 0;
    bulk_wait_all();
    asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p.done + u.mat * 3 + KIND) : "memory");
  }
  __syncwarp();
  return true;
}

// All steps' products in one launch. Warp 0: TMA producer; warp 1: MMA issuer (rank 0 of the
// pair, for both CTAs); warps 2 to 9: epilogues, while the next unit's MMAs fill the other
// TMEM buffer; warp 10: draws the pair's units (rank 0).
__global__ void __launch_bounds__(kThreads, 1) ns_kernel(const __grid_constant__ NsArgs p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* tiles = smem_raw + pad;
  uint8_t* staging = tiles + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kStagingBytes + kFactorBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* block_bars = tempty + 2;  // [kEpiWarps][2]
  UnitRing* ring = reinterpret_cast<UnitRing*>(block_bars + 2 * kEpiWarps);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ring + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + b, 1);
      mbar_init(tempty + b, 2 * kEpiWarps);
    }
    for (int b = 0; b < 2 * kEpiWarps; ++b) mbar_init(block_bars + b, 1);
    for (int b = 0; b < kRing; ++b) {
      mbar_init(ring->full + b, 1);
      mbar_init(ring->empty + b, kTakers);
    }
    mbar_init(&ring->draw, 1);
    *abort_flag = 0;
    fence_barrier_init();
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

  Taker units{ring, abort_flag, p.status};
  Known known;
  Unit u;
  if (warp == 0) {
    if (lane == 0) {  // TMA producer
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      bool ok = true;
      while (ok && units.take(u, true)) {
        int i, j, lo, hi;
        tile_at(p, u, i, j);
        k_blocks(p, u, lo, hi);
        if (!wait_inputs(p, u, known, abort_flag)) {
          ok = false;
          break;
        }
        const int half = p.width[u.kind] / 2;  // columns of the unit in each CTA
        const int m0 = i * kTile + rank * 128, n0 = j * 2 * half + rank * half, x = u.step & 1;
        const int xrow = u.mat * p.mp, srow = u.mat * p.np;
        const int draw_at = max(lo, hi - kDrawAhead);
        for (int kb = lo; kb < hi; ++kb) {
          if (rank == 0 && kb == draw_at) mbar_arrive(&ring->draw);
          if (!mbar_wait(empty + stage, phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          uint8_t* sa = tiles + stage * kStageBytes;
          uint8_t* sb = sa + kOperandBytes;
          if (rank == 0) mbar_arrive_expect_tx(full + stage, 2 * (kOperandBytes + half * kBK * 2));
          const uint32_t bar = peer_smem_addr(full + stage, 0);
          const int k0 = kb * kBK;
          if (u.kind == GRAM) {  // both operands stored [K, MN]
            tma_load_2d_pair(sa, &p.x_mn[x], bar, m0, xrow + k0);
            tma_load_2d_pair(sa + 8192, &p.x_mn[x], bar, m0 + 64, xrow + k0);
            tma_load_2d_pair(sb, &p.x_mn[x], bar, n0, xrow + k0);
            if (half == 128) tma_load_2d_pair(sb + 8192, &p.x_mn[x], bar, n0 + 64, xrow + k0);
          } else if (u.kind == SQUARE) {
            tma_load_2d_pair(sa, &p.e_k, bar, k0, srow + m0);
            tma_load_2d_pair(sb, &p.e_n, bar, k0, srow + n0);
          } else {
            tma_load_2d_pair(sa, &p.x_k[x], bar, k0, xrow + m0);
            tma_load_2d_pair(sb, &p.b_n, bar, k0, srow + n0);
          }
          ++issued;
          if (++stage == kStages) stage = 0, phase ^= 1u;
        }
      }
      if (*abort_flag && rank == 0) {
        // let the loads already issued land (rank 1's complete on rank 0's barriers)
        for (long n = 0; n < kStages && n < issued; ++n) {
          const long q = issued - 1 - n;
          mbar_wait_drain(full + (q % kStages), static_cast<uint32_t>((q / kStages) & 1));
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {  // MMA issuer, for both CTAs
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = true, issued_any = false;
      for (; ok && units.take(u, true); ++local) {
        int lo, hi;
        k_blocks(p, u, lo, hi);
        const int buf = local & 1;
        if (!mbar_wait(tempty + buf, ((local >> 1) & 1u) ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d0 = tmem_base + static_cast<uint32_t>(buf * kTile);
        const bool mn = u.kind == GRAM;
        const uint32_t idesc = p.width[u.kind] == 256
                                   ? (mn ? idesc_bf16_f32(kTile, 256, true, true, true) : idesc_bf16_f32(kTile, 256, false, false, true))
                                   : (mn ? idesc_bf16_f32(kTile, 128, true, true, true) : idesc_bf16_f32(kTile, 128, false, false, true));
        for (int kb = lo; kb < hi; ++kb) {
          if (!mbar_wait(full + stage, phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sa = smem_addr(tiles + stage * kStageBytes), sb = sa + kOperandBytes;
          const uint32_t step = mn ? 2048 : 32, lbo = mn ? 8192 : 16;
#pragma unroll
          for (int k16 = 0; k16 < kBK / 16; ++k16)
            tc_mma_bf16_pair(d0, smem_desc_sw128(sa + k16 * step, lbo, 1024), smem_desc_sw128(sb + k16 * step, lbo, 1024), idesc,
                             kb > lo || k16 > 0 ? 1u : 0u);
          issued_any = true;
          tc_commit_pair(empty + stage);
          if (++stage == kStages) stage = 0, phase ^= 1u;
        }
        if (!ok) break;
        tc_commit_pair(tfull + buf);
      }
      if (*abort_flag && issued_any) {
        tc_commit_pair(empty + stage);
        mbar_wait_drain(empty + stage, phase);
      }
    }
  } else if (warp < 2 + kEpiWarps) {
    const int ew = warp - 2;
    int turn = 0;
    bool ok = true;
    for (int local = 0; ok && units.take(u, false); ++local) {
      const int buf = local & 1;
      const uint32_t t0 = tmem_base + static_cast<uint32_t>(buf * kTile);
      uint8_t* st = staging + ew * 4 * kChunkBytes;
      float* factors = reinterpret_cast<float*>(staging + kStagingBytes) + ew * 32;
      uint64_t* bar = block_bars + 2 * ew;
      const uint32_t parity = (local >> 1) & 1u;
      if (u.kind == GRAM) ok = epilogue<GRAM>(p, u, st, factors, bar, turn, tfull + buf, parity, t0, rank, ew, known, abort_flag);
      else if (u.kind == SQUARE) ok = epilogue<SQUARE>(p, u, st, factors, bar, turn, tfull + buf, parity, t0, rank, ew, known, abort_flag);
      else ok = epilogue<APPLY>(p, u, st, factors, bar, turn, tfull + buf, parity, t0, rank, ew, known, abort_flag);
      if (!ok) break;
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(peer_smem_addr(tempty + buf, 0));
    }
    if (lane == 0) bulk_wait_all();
  } else if (rank == 0 && lane == 0) {
    // every unit drawn is given to both CTAs, the end too; one ahead of the loads, no more: a
    // unit held by a pair that is busy keeps those that wait for it waiting
    for (int n = 0;; ++n) {
      if (n > 0 && !mbar_wait(&ring->draw, (n - 1) & 1u, abort_flag, p.status)) break;
      const int slot = n & (kRing - 1);
      if (!mbar_wait_cluster(ring->empty + slot, ((n / kRing) & 1u) ^ 1u, abort_flag, p.status)) break;
      uint2 w = make_uint2(~0u, 0u);
      bool more = unit_at(p, atomicAdd(p.next, 1), u);
      if (more && !TW_CHECKED(u.mat >= 0 && u.mat < p.count && u.tile >= 0 && u.tile < tiles_of(p, u.kind) && u.slice >= 0 &&
                              u.slice < p.slices[u.kind], p.status))
        more = false;
      if (more) w = make_uint2(static_cast<uint32_t>(u.step << 24 | u.kind << 16 | u.mat << 8 | u.slice), static_cast<uint32_t>(u.tile));
#pragma unroll
      for (uint32_t r = 0; r < 2; ++r) {
        asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(peer_smem_addr(ring->unit + slot, r)), "r"(w.x), "r"(w.y) : "memory");
        mbar_arrive_cluster(peer_smem_addr(ring->full + slot, r));
      }
      if (!more) break;
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
  int count, rows, cols;       // of g as given
  float mu;
  int nesterov;
  double* norms;               // [count][kNormBlocks]
  int* arrived;                // counters to clear
  int n_arrived;
  uint16_t *hi, *lo;           // [count][mp][np]
  int mp, np, klog2;
  int first;                   // the launch's first matrix
  bool vec;                    // g's and m's rows are whole vectors of 8 elements on 16 bytes
  bool flat;                   // g's and m's rows follow each other: the sums take them as one, on 16 bytes
};

constexpr int kNormBlocks = 304, kNormThreads = 512;

// U at element (r, c); store: writes the new momentum
template <int GT>
TW_DEV float update_of(const NsInArgs& a, int mat, int r, long c, bool store) {
  using S = typename Elem<GT>::S;
  const float g = Elem<GT>::get(static_cast<const S*>(a.g[mat])[static_cast<size_t>(r) * a.ldg + c]);
  if (a.m[mat] == nullptr) return g;
  float* m = a.m[mat] + static_cast<size_t>(r) * a.ldm + c;
  float v = *m;
  if (store) *m = v = fmaf(a.mu, v, g);
  return a.nesterov ? fmaf(a.mu, v, g) : v;
}
// The same for the 8 elements from c on, on 16 bytes (or, where rows are not of whole vectors
// there and nothing is stored, anywhere; elements past the row are then 0).
template <int GT>
TW_DEV void update8(const NsInArgs& a, int mat, int r, long c, bool store, float (&u)[8]) {
  if (!a.vec && !store) {
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
  const long step = static_cast<long>(gridDim.x) * kNormThreads, first = static_cast<long>(blockIdx.x) * kNormThreads + threadIdx.x;
  if (a.flat) {
    const long all = static_cast<long>(a.rows) * a.cols;
#pragma unroll 2
    for (long i = first; i < all / 8; i += step) {
      float u[8];
      update8<GT>(a, mat, 0, i * 8, true, u);
#pragma unroll
      for (int k = 0; k < 8; ++k) add_square(s, u[k]);
    }
    if (first < all % 8) add_square(s, update_of<GT>(a, mat, 0, all / 8 * 8 + first, true));
  } else {
    const int one = a.vec ? 8 : 1;  // elements of a row at once
    const unsigned per_row = a.cols / one;
    const long total = static_cast<long>(a.rows) * per_row;
    long i = first;
    int r = static_cast<int>(i / per_row), c = static_cast<int>(i - static_cast<long>(r) * per_row);
    const int dr = static_cast<int>(step / per_row), dc = static_cast<int>(step - static_cast<long>(dr) * per_row);
    auto next = [&] {
      i += step, r += dr, c += dc;
      if (c >= static_cast<int>(per_row)) c -= per_row, ++r;
    };
    if (a.vec) {
#pragma unroll 2
      for (; i < total; next()) {
        float u[8];
        update8<GT>(a, mat, r, c * 8, true, u);
#pragma unroll
        for (int k = 0; k < 8; ++k) add_square(s, u[k]);
      }
    } else {
#pragma unroll 8
      for (; i < total; next()) add_square(s, update_of<GT>(a, mat, r, c, true));
    }
  }
  s.small = warp_sum(s.small), s.mid = warp_sum(s.mid), s.big = warp_sum(s.big);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kNormThreads / 32; ++w)
      s.small += red[w].small, s.mid += red[w].mid, s.big += red[w].big;
    a.norms[static_cast<size_t>(mat) * kNormBlocks + blockIdx.x] =
        static_cast<double>(s.small) * 0x1p-180 + static_cast<double>(s.mid) + static_cast<double>(s.big) * 0x1p160;
  }
  if (mat == 0)
    for (long k = first; k < a.n_arrived; k += step) a.arrived[k] = 0;
}

// 2^k / |U|_F from the sums, by one warp of every CTA in the same order (the SM adds two
// doubles a clock: all eight warps together took 7 us); as two factors, so that neither they
// nor a product by one of them overflows. The root of the sum's mantissa is fp32's: 2^-22 of
// a matrix's every value.
TW_DEV float2 start_factor(const NsInArgs& a, int mat, int norm_blocks) {
  __shared__ float2 factor;
  if (threadIdx.x < 32) {
    double s = 0.0;
    for (int i = threadIdx.x; i < norm_blocks; i += 32) s += a.norms[static_cast<size_t>(mat) * kNormBlocks + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    float2 f = make_float2(1.f, s == 0.0 || s > 0.0 ? 0.f : __int_as_float(0x7FC00000));
    if (s > 0.0 && s < 0x1p1000) {
      // s = m 4^e, 1 <= m < 4
      const int bits = __double2hiint(s), e = ((bits >> 20) - 1023) >> 1;
      const float m = static_cast<float>(__hiloint2double(bits - (e << 21), __double2loint(s)));
      const int power = a.klog2 - e, half = power >> 1;
      auto pow2 = [](int n) { return __int_as_float((n + 127) << 23); };
      f = make_float2(pow2(half), rsqrtf(m) * pow2(power - half));
    }
    if (threadIdx.x == 0) factor = f;
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
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int i = first + 4 * k;
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

// How a product of `tiles` 256 x 256 tiles (of all matrices) with kb K blocks runs: whole
// tiles where there is one for every pair of SMs (a matrix's products overlap the others');
// with fewer, units of 256 or 128 columns, and slices of their K loop. 76 pairs of SMs (a constant, so that the
// workspace does not depend on the device). Costs in K blocks of a 256-wide unit, 0.33 us: a
// narrow unit's takes 0.7 (its operands are three quarters of the bytes for half the work);
// after the last K block a unit's epilogue takes 23 (7.6 us), a narrow one's 14; slices hand
// on their sums and add them.
constexpr int kPairs = 76, kMostSlices = 8;
void form_of(int tiles, int kb, int& width, int& slices) {
  width = 256, slices = 1;
  if (tiles >= kPairs) return;
  float best = 0.f;
  for (int w = 256; w >= 128; w /= 2)
    for (int s = 1; s <= std::min(kMostSlices, kb); ++s) {
      const int units = tiles * (256 / w) * s, chunk = (kb + s - 1) / s;
      if ((kb + chunk - 1) / chunk != s || (s > 1 && units > kPairs)) continue;  // no empty slice
      const float cost = static_cast<float>((units + kPairs - 1) / kPairs) * chunk * (w == 256 ? 1.f : 0.7f) + (w == 256 ? 23.f : 14.f) +
                         (s > 1 ? (w == 256 ? 30.f : 18.f) + 3.f * s : 0.f);
      if (best == 0.f || cost < best) best = cost, width = w, slices = s;
    }
}

struct Layout {
  int mp, np, width[3], slices[3], slots;
  size_t hi0, hi1, lo, e, b, diag, part, arrived, counters, norms, bytes;
  int words() const { return static_cast<int>((norms - arrived) / 4); }  // arrived and the counters after it
};
Layout layout(int m, int n, int count) {
  Layout l{};
  l.mp = up(std::max(m, n)), l.np = up(std::min(m, n));
  const int t = l.np / kTile, tri = t * (t + 1) / 2, all = l.mp / kTile * t;
  const int tiles[3] = {tri, tri, all};
  for (int k = 0; k < 3; ++k) {
    form_of(tiles[k] * count, (k == GRAM ? l.mp : l.np) / kBK, l.width[k], l.slices[k]);
    if (l.slices[k] > 1) l.slots = std::max(l.slots, tiles[k] * (256 / l.width[k]) * l.slices[k]);
  }
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at = (at + bytes + 1023) / 1024 * 1024;
    return was;
  };
  const size_t x = static_cast<size_t>(count) * l.mp * l.np * 2, s = static_cast<size_t>(count) * l.np * l.np * 2;
  l.hi0 = take(x), l.hi1 = take(x), l.lo = take(x), l.e = take(s), l.b = take(s);
  l.diag = take(static_cast<size_t>(count) * l.np * 4);
  l.part = take(static_cast<size_t>(count) * l.slots * kTile * kTile * 4);
  l.arrived = take(static_cast<size_t>(count) * l.slots * 2 * kEpiWarps * 4);
  l.counters = take(static_cast<size_t>(3 * count + 1) * 4);
  l.norms = take(static_cast<size_t>(count) * kNormBlocks * sizeof(double));
  l.bytes = at;
  return l;
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
  bool on16 = true;
  for (int i = 0; i < o.count; ++i) {
    in.g[i] = o.g[i], in.m[i] = o.buf != nullptr ? o.buf[i] : nullptr;
    on16 = on16 && ((reinterpret_cast<uintptr_t>(in.g[i]) | reinterpret_cast<uintptr_t>(in.m[i])) & 15u) == 0;
  }
  in.ldg = o.ldg, in.ldm = o.ldbuf, in.count = o.count, in.rows = o.m, in.cols = o.n;
  in.mu = o.mu, in.nesterov = o.nesterov;
  in.vec = on16 && o.n % 8 == 0 && o.ldg * static_cast<int64_t>(o.gtype == TW_F32 ? 4 : 2) % 16 == 0 && o.ldbuf % 4 == 0;
  in.flat = on16 && (o.m == 1 || (o.ldg == o.n && (o.buf == nullptr || o.ldbuf == o.n)));
  in.norms = reinterpret_cast<double*>(ws + l.norms);
  in.arrived = reinterpret_cast<int*>(ws + l.arrived), in.n_arrived = l.words();
  in.hi = at16(l.hi0), in.lo = at16(l.lo), in.mp = l.mp, in.np = l.np, in.klog2 = k;
  cudaError_t e = o.gtype == TW_F32    ? way_in<TW_F32>(in, wide, s)
                  : o.gtype == TW_BF16 ? way_in<TW_BF16>(in, wide, s)
                                       : way_in<TW_F16>(in, wide, s);
  if (e != cudaSuccess) return e;

  // maps: operands in boxes of 64 x 128 (K-major) and 64 x 64 (MN-major), the epilogues' 32 x 32
  NsArgs p = {};
  const uint64_t np2 = static_cast<uint64_t>(l.np) * 2;
  const uint64_t xrows = static_cast<uint64_t>(l.mp) * o.count, srows = static_cast<uint64_t>(l.np) * o.count;
  bool ok = true;
  auto map = [&](CUtensorMap& m, size_t at, uint64_t rows, uint32_t box_cols, uint32_t box_rows) {
    ok = ok && make_tmap_bf16(&m, ws + at, l.np, rows, np2, box_cols, box_rows, box_cols == 32);
  };
  for (int i = 0; i < 2; ++i) {
    const size_t x = i ? l.hi1 : l.hi0;
    map(p.x_k[i], x, xrows, 64, 128), map(p.x_mn[i], x, xrows, 64, 64), map(p.x_block[i], x, xrows, 32, 32);
  }
  map(p.lo_block, l.lo, xrows, 32, 32), map(p.e_block, l.e, srows, 32, 32), map(p.b_block, l.b, srows, 32, 32);
  map(p.e_k, l.e, srows, 64, 128), map(p.e_n, l.e, srows, 64, l.width[SQUARE] / 2), map(p.b_n, l.b, srows, 64, l.width[APPLY] / 2);
  if (!ok) return cudaErrorInvalidValue;

  p.tiles_m = l.mp / kTile, p.tiles_n = l.np / kTile, p.count = o.count, p.steps = o.steps, p.np = l.np, p.mp = l.mp;
  for (int i = 0; i < 3; ++i) p.width[i] = l.width[i], p.slices[i] = l.slices[i];
  p.slots = l.slots, p.part = reinterpret_cast<float*>(ws + l.part), p.arrived = in.arrived;
  p.done = reinterpret_cast<int*>(ws + l.counters), p.next = p.done + 3 * o.count, p.status = o.status, p.withhold = o.withhold;
  p.diag = reinterpret_cast<float*>(ws + l.diag);
  for (int i = 0; i < o.count; ++i) p.out[i] = o.out[i];
  p.ldo = o.ldo, p.rows = std::max(o.m, o.n), p.cols = std::min(o.m, o.n), p.otype = o.otype, p.transposed = wide;
  p.scale = static_cast<float>(std::ldexp(static_cast<double>(o.scale), -k)), p.beta = o.beta;
  for (int step = 0; step < o.steps; ++step) {
    const double a = o.coef[3 * step], b = o.coef[3 * step + 1], c = o.coef[3 * step + 2];
    const double t = step >= 3 && step + 1 == o.steps ? 1.0 : 0.0, q0 = a + b * t + c * t * t, q1 = b + 2.0 * c * t;
    p.f0[step][GRAM] = std::ldexp(1.f, kGramLog2 - 2 * k), p.f1[step][GRAM] = static_cast<float>(std::ldexp(t, kGramLog2));
    p.f0[step][SQUARE] = static_cast<float>(std::ldexp(q1, kPolyLog2 - kGramLog2));
    p.f1[step][SQUARE] = static_cast<float>(std::ldexp(c, kPolyLog2 - 2 * kGramLog2));
    p.f0[step][APPLY] = static_cast<float>(q0), p.f1[step][APPLY] = std::ldexp(1.f, -kPolyLog2);
  }
  e = cudaFuncSetAttribute(ns_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  static KnownClusters known;
  const int resident = resident_clusters(known, ns_kernel, kThreads, kSmem, 2);
  // no more pairs than a product of all matrices has units
  long most = 0;
  for (int i = 0; i < 3; ++i) {
    const long tiles = i == APPLY ? static_cast<long>(p.tiles_m) * p.tiles_n : static_cast<long>(p.tiles_n) * (p.tiles_n + 1) / 2;
    most = std::max(most, o.count * tiles * (256 / l.width[i]) * l.slices[i]);
  }
  const int pairs = static_cast<int>(std::min<long>(most, std::min(resident, device_sm_count() / 2)));
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  e = launch_clustered(ns_kernel, dim3(2 * pairs), dim3(kThreads), kSmem, 2, s, p);
  trace_mark(s, "ortho_products");
  return e;
}

}  // namespace tw
