// Device pieces shared by the attention kernels: the swizzled tile address, the
// packed FP4 / FP8 -> fp16 conversions, volatile read-only loads, rotate-half,
// in-warp reductions, head-group barriers and TMEM block loads and stores.
#pragma once

#include "csa_device.cuh"

namespace csa {

__device__ __forceinline__ uint32_t swz128(int row, int chunk) {
  return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
}

// Four FP4 pairs (the bytes of w, low byte first) -> four f16x2; in each the
// low nibble (even dimension) lands in the low half.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// Two E4M3 pairs (the 16-bit halves of w) -> two f16x2, low byte -> low half.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t (&o)[2]) {
  asm("{\n\t.reg .b16 h0, h1;\n\t"
      "mov.b32 {h0, h1}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, h0;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h1;\n\t}"
      : "=r"(o[0]), "=r"(o[1])
      : "r"(w));
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t x, __half2 s) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&x), s);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// In-warp reduction of NV values per lane (NV = 4, 8, 16 or 32) across the 32
// lanes: recursive halving, then a butterfly over the remaining lane bits.
// Lane l ends with the reduction of value index (l >> (5 - log2 NV)).
template <int NV>
struct RedShift {
  static constexpr int v = NV == 32 ? 0 : (NV == 16 ? 1 : (NV == 8 ? 2 : 3));
};
template <int NV, bool kMax>
__device__ __forceinline__ float warp_reduce_many(float (&v)[NV], int lane) {
  int cnt = NV;
#pragma unroll
  for (int o = 16; o >= 1 && cnt > 1; o >>= 1) {
    const int half = cnt >> 1;
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) {
      if (i < half) {
        const float send = upper ? v[i] : v[i + half];
        const float keep = upper ? v[i + half] : v[i];
        const float recv = __shfl_xor_sync(0xFFFFFFFFu, send, o);
        v[i] = kMax ? fmaxf(keep, recv) : keep + recv;
      }
    }
    cnt = half;
  }
  float x = v[0];
  constexpr int kShift = RedShift<NV>::v;
#pragma unroll
  for (int o = 1; o < (1 << kShift); o <<= 1) {
    const float y = __shfl_xor_sync(0xFFFFFFFFu, x, o);
    x = kMax ? fmaxf(x, y) : x + y;
  }
  return x;
}

// Loads written as volatile asm stay where the program issues them, so the
// prefetch of the next tile is in flight while this one is processed.
__device__ __forceinline__ uint4 ldg_nc_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint16_t ldg_nc_u16(const void* p) {
  uint16_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float ldg_nc_f32(const void* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint16_t v) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(v));
  return d;
}

// Rotate-half on the pair (a, b) = (dim 448 + j, dim 480 + j) of the last 64
// dims: a' = a*c - b*s, b' = b*c + a*s, each product and the sum rounded once
// (no fused multiply-add).  `mine` holds this thread's 16 values, `other` the
// partner's (the other half of the pairs); lower: this thread holds the a's.
__device__ __forceinline__ void rotate16(float (&mine)[16], const float (&other)[16], bool lower,
                                         const float* cs, const float* sn) {
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    const float c = __ldg(cs + t), s = __ldg(sn + t);
    mine[t] = lower ? __fsub_rn(__fmul_rn(mine[t], c), __fmul_rn(other[t], s))
                    : __fadd_rn(__fmul_rn(mine[t], c), __fmul_rn(other[t], s));
  }
}

// Barrier over the four warps that share one head group (ids 1..8).
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}
// The same barrier, also OR-ing a flag over the four warps: every thread of
// the head group gets the same answer, so all take the same branch after it.
__device__ __forceinline__ bool group_sync_or(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, %2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}

template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, float (&v)[N]) {
  if constexpr (N % 16 == 0) {
#pragma unroll
    for (int c = 0; c < N; c += 16) {
      uint32_t u[16];
      tmem_ld16(taddr + c, u);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) v[c + i] = __uint_as_float(u[i]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      uint32_t u[4];
      tmem_ld4(taddr + c, u);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c + i] = __uint_as_float(u[i]);
    }
  }
}

template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t taddr, const float (&v)[N]) {
  if constexpr (N % 16 == 0) {
#pragma unroll
    for (int c = 0; c < N; c += 16) {
      uint32_t u[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(v[c + i]);
      tmem_st16(taddr + c, u);
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(v[c + i]);
      tmem_st4(taddr + c, u);
    }
  }
}

}  // namespace csa
