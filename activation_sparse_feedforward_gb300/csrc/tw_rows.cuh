// Device helpers of the row operators (tw_norm_rows.cuh, tw_logits.cuh, tw_embed.cu): the three element
// types, 16-byte vectors of them, asynchronous 16-byte copies into shared memory,
// sums over teams of warps, and reads of another CTA's shared memory in a cluster.
#pragma once

#include "tw_common.cuh"

namespace tw {

// ------------------------------------------------------------------ element types
// Elem<TW_*>: storage S, E elements per 16 bytes, widening to fp32 (exact; pairs: as
// packed pairs) and narrowing (round to nearest even).
template <int DT>
struct Elem;

// *p = v, and what was there, for 16 bits of shared memory
TW_DEV uint16_t exchange16(uint16_t* p, uint16_t v) {
  uint16_t was = *p, seen;
  while ((seen = atomicCAS(p, was, v)) != was) was = seen;
  return was;
}

template <>
struct Elem<TW_F32> {
  using S = float;
  static constexpr int E = 4;
  static TW_DEV float get(S v) { return v; }
  static TW_DEV S put(float v) { return v; }
  static TW_DEV S neg_inf() { return __int_as_float(0xFF800000); }
  static TW_DEV S exchange(S* p, S v) { return atomicExch(p, v); }  // shared memory
  static TW_DEV void pairs(const uint4& w, float2 (&v)[2]) {
    v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    v[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
  static TW_DEV void unpack(const uint4& w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
  }
  static TW_DEV float2 rounded(float2 v) { return v; }  // to the type and back
  static TW_DEV uint4 pack_pairs(const float2 (&v)[2]) {
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
  }
  // running maximum of vectors (a NaN loses to a number)
  struct Max {
    float m = -__builtin_huge_valf();
    TW_DEV void add(const uint4& w) { m = fmaxf(m, max16(w)); }
    TW_DEV float get() const { return m; }
  };
  // the largest of the four
  static TW_DEV float max16(const uint4& w) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
};

template <>
struct Elem<TW_BF16> {
  using S = uint16_t;
  static constexpr int E = 8;
  static TW_DEV float get(S v) { return bf16_to_f32(v); }
  static TW_DEV S put(float v) { return f32_to_bf16(v); }
  static TW_DEV S neg_inf() { return 0xFF80; }
  static TW_DEV S exchange(S* p, S v) { return exchange16(p, v); }
  static TW_DEV void pairs(const uint4& w, float2 (&v)[4]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(bf16_lo(r[i]), bf16_hi(r[i]));
  }
  static TW_DEV void unpack(const uint4& w, float (&v)[8]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(r[i]), v[2 * i + 1] = bf16_hi(r[i]);
  }
  static TW_DEV float2 rounded(float2 v) {
    const uint32_t r = pack_bf16x2_rn(v.x, v.y);
    return make_float2(bf16_lo(r), bf16_hi(r));
  }
  static TW_DEV uint4 pack_pairs(const float2 (&v)[4]) {
    return make_uint4(pack_bf16x2_rn(v[0].x, v[0].y), pack_bf16x2_rn(v[1].x, v[1].y), pack_bf16x2_rn(v[2].x, v[2].y),
                      pack_bf16x2_rn(v[3].x, v[3].y));
  }
  struct Max {
    uint32_t m = 0xFF80FF80u;
    TW_DEV void add(const uint4& w) {
      const __nv_bfloat162 r = __hmax2(__hmax2(h2(w.x), h2(w.y)), __hmax2(h2(w.z), h2(w.w)));
      const __nv_bfloat162 n = __hmax2(h2(m), r);
      m = *reinterpret_cast<const uint32_t*>(&n);
    }
    TW_DEV float get() const {
      const float2 f = __bfloat1622float2(h2(m));
      return fmaxf(f.x, f.y);
    }
    static TW_DEV __nv_bfloat162 h2(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); }
  };
  static TW_DEV float max16(const uint4& w) {
    Max m;
    m.add(w);
    return m.get();
  }
};

template <>
struct Elem<TW_F16> {
  using S = uint16_t;
  static constexpr int E = 8;
  static TW_DEV float get(S v) { return f16_to_f32(v); }
  static TW_DEV S put(float v) { return f32_to_f16(v); }
  static TW_DEV S neg_inf() { return 0xFC00; }
  static TW_DEV S exchange(S* p, S v) { return exchange16(p, v); }
  static TW_DEV void pairs(const uint4& w, float2 (&v)[4]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
  }
  static TW_DEV void unpack(const uint4& w, float (&v)[8]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
  static TW_DEV float2 rounded(float2 v) { return __half22float2(__floats2half2_rn(v.x, v.y)); }
  static TW_DEV uint4 pack_pairs(const float2 (&v)[4]) {
    return make_uint4(pack_f16x2_rn(v[0].x, v[0].y), pack_f16x2_rn(v[1].x, v[1].y), pack_f16x2_rn(v[2].x, v[2].y),
                      pack_f16x2_rn(v[3].x, v[3].y));
  }
  struct Max {
    uint32_t m = 0xFC00FC00u;
    TW_DEV void add(const uint4& w) {
      const __half2 r = __hmax2(__hmax2(h2(w.x), h2(w.y)), __hmax2(h2(w.z), h2(w.w)));
      const __half2 n = __hmax2(h2(m), r);
      m = *reinterpret_cast<const uint32_t*>(&n);
    }
    TW_DEV float get() const {
      const float2 f = __half22float2(h2(m));
      return fmaxf(f.x, f.y);
    }
    static TW_DEV __half2 h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
  };
  static TW_DEV float max16(const uint4& w) {
    Max m;
    m.add(w);
    return m.get();
  }
};

// Two fp32 lanes an instruction, one rounding per lane. (float2 and the intrinsics, not
// 64-bit registers: the compiler then places the halves without moves.)
TW_DEV float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
TW_DEV float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
TW_DEV float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
TW_DEV float2 both(float v) { return make_float2(v, v); }

// ------------------------------------------------------------------ asynchronous copies
// One 16-byte copy, global to shared, past L1; the copying thread sees its own copies
// after cp_wait (no wait loop: the hardware counts them).
TW_DEV void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
TW_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
TW_DEV void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Asks for the line of p in L2, without waiting or a place.
TW_DEV void prefetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ------------------------------------------------------------------ rows off 16 bytes
// The 16 bytes that begin `shift` elements (0 to E - 1) into a and b.
template <int DT>
TW_DEV uint4 shifted(const uint4& a, const uint4& b, int shift) {
  constexpr int kHalf = Elem<DT>::E / 4 - 1;  // elements of 16 bits: a last step of half a word
  const bool two = (shift >> kHalf) & 2, one = (shift >> kHalf) & 1;
  const uint32_t w[6] = {two ? a.z : a.x, two ? a.w : a.y, two ? b.x : a.z, two ? b.y : a.w, two ? b.z : b.x, two ? b.w : b.y};
  uint32_t v[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = one ? w[i + 1] : w[i];
  if constexpr (kHalf > 0) {
    const uint32_t half = shift & 1 ? 0x5432u : 0x3210u;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __byte_perm(v[i], v[i + 1], half);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// The same from two adjacent vectors in shared memory, from the 8 bytes on that hold the
// first element: fewer words to choose from.
template <int DT>
TW_DEV uint4 shifted_from(const uint4* from, int shift) {
  const uint32_t bytes = shift * sizeof(typename Elem<DT>::S);
  const uint2* at = reinterpret_cast<const uint2*>(from) + (bytes >> 3);
  const uint2 a = at[0], b = at[1], c = at[2];
  const uint32_t w[6] = {a.x, a.y, b.x, b.y, c.x, c.y};
  uint32_t v[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = bytes & 4 ? w[i + 1] : w[i];
  if constexpr (Elem<DT>::E == 8) {
    const uint32_t half = bytes & 2 ? 0x5432u : 0x3210u;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __byte_perm(v[i], v[i + 1], half);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// The first n (1 or more) elements of v, then 0.
template <int DT>
TW_DEV uint4 first_of(const uint4& v, int n) {
  constexpr int E = Elem<DT>::E;
  if (n >= E) return v;
  union {
    uint4 w;
    typename Elem<DT>::S e[E];
  } u;
  u.w = v;
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (i >= n) u.e[i] = Elem<DT>::put(0.f);
  return u.w;
}

// The vector of the E elements from p on, of which n (1 or more) are the row's: the others
// read 0. p may lie anywhere; read are whole 16 bytes that hold an element of the row, or,
// where careful, the row's elements alone.
template <int DT>
TW_DEV uint4 load_any(const typename Elem<DT>::S* p, int n, bool careful) {
  using S = typename Elem<DT>::S;
  constexpr int E = Elem<DT>::E;
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(S)), left = min(n, E);
  union {
    S e[E];
    uint4 w;
  } u;
  if (careful) {
#pragma unroll
    for (int i = 0; i < E; ++i) u.e[i] = i < left ? p[i] : Elem<DT>::put(0.f);
    return u.w;
  }
  const uint4* at = reinterpret_cast<const uint4*>(p - shift);
  const uint4 a = at[0], b = shift + left > E ? at[1] : make_uint4(0, 0, 0, 0);
  return first_of<DT>(shifted<DT>(a, b, shift), left);
}

// Stores v at p, of which n elements are the row's (0 or fewer: none). All lanes of a warp,
// whose vectors follow each other in one row: an aligned 16 bytes are written by the lane
// that holds their end, with the lane before's elements. What is left at a full warp's two
// ends makes one vector's elements: a lane each. Where the row ends, by the element.
template <int DT>
TW_DEV void store_any(typename Elem<DT>::S* p, const uint4& v, int n, int lane) {
  using S = typename Elem<DT>::S;
  constexpr int E = Elem<DT>::E;
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(S)), head = E - shift;
  const uint4 before = make_uint4(__shfl_up_sync(0xFFFFFFFFu, v.x, 1), __shfl_up_sync(0xFFFFFFFFu, v.y, 1),
                                  __shfl_up_sync(0xFFFFFFFFu, v.z, 1), __shfl_up_sync(0xFFFFFFFFu, v.w, 1));
  const bool whole = (lane > 0 || shift == 0) && n >= head;
  if (whole) *reinterpret_cast<uint4*>(p - shift) = shift == 0 ? v : shifted<DT>(before, v, head);
  if (n - (31 - lane) * E >= E) {  // every lane's vector is whole
    if (shift == 0) return;
    const int from = lane < head ? 0 : 31;
    const uint32_t w[4] = {__shfl_sync(0xFFFFFFFFu, v.x, from), __shfl_sync(0xFFFFFFFFu, v.y, from),
                           __shfl_sync(0xFFFFFFFFu, v.z, from), __shfl_sync(0xFFFFFFFFu, v.w, from)};
    if (lane < E) {
      const int word = lane / (E / 4);
      const uint32_t a = word & 2 ? w[2] : w[0], b = word & 2 ? w[3] : w[1], c = word & 1 ? b : a;
      S* q = p + (from - lane) * E + lane;
      if constexpr (E == 8)
        *reinterpret_cast<uint16_t*>(q) = static_cast<uint16_t>(lane & 1 ? c >> 16 : c);
      else
        *reinterpret_cast<uint32_t*>(q) = c;
    }
    return;
  }
  const bool next = shift > 0 && lane < 31 && n - E >= head;  // the next lane takes this one's end
  const int from = whole ? head : 0, to = next ? head : min(n, E);
  if (from < to) {
    union {
      uint4 w;
      S e[E];
    } u;
    u.w = v;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i >= from && i < to) p[i] = u.e[i];
  }
}

// ------------------------------------------------------------------ reductions
TW_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// Barrier `id` among `n` threads (a multiple of 32): the warps of one team of a CTA.
TW_DEV void team_barrier(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// ------------------------------------------------------------------ clusters
TW_DEV void st_cluster_f32(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}
TW_DEV void st_cluster_v4(uint32_t cluster_addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "f"(v.x), "f"(v.y), "f"(v.z),
               "f"(v.w)
               : "memory");
}
TW_DEV float ld_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}
TW_DEV unsigned long long ld_cluster_u64(uint32_t cluster_addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// A cluster barrier in two halves: what a thread did before arriving is done for every
// thread that has waited. (The warp converges first: the halves are warp-wide.)
TW_DEV void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
// Arriving with nothing to show: only that this CTA has started.
TW_DEV void cluster_arrive_relaxed() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
TW_DEV void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
TW_DEV void cluster_barrier() {
  cluster_arrive();
  cluster_wait();
}

// 2^x (hardware approximation, about 2 ulp; subnormal results flush to zero)
TW_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace tw
