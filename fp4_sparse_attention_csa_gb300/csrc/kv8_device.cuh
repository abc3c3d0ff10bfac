// Device pieces of the 8-bit cache of keys and values (include/csa.h, csa_kv8_t): the
// records' layout, which rows are valid, and rotation of 8 dims at a time.
#pragma once

#include "attn_device.cuh"
#include "csa_internal.h"

namespace csa {

constexpr int kKv8Tail = CSA_KV8_TAIL;
constexpr int kKv8MaxPos = INT32_MAX - 1024;     // positions stay within 32 bits
constexpr float kKv8Least = 7.888609052210118e-31f;   // 2^-100: what is smaller throughout is stored as zeros

// Pages of that many positions; the sum passes 32 bits.
__host__ __device__ constexpr int64_t kv8_pages(int64_t positions) { return (positions + PAGE - 1) / PAGE; }
// Record of page `page`, key head h.
template <int D>
__device__ __forceinline__ size_t kv8_record(int page, int heads, int h) {
  return ((size_t)page * heads + h) * CSA_KV8_RECORD_BYTES(D);
}
// A row is valid when its request exists and its position lies inside the request's
// pages, the rotary tables and the call's bound.
__device__ __forceinline__ int kv8_pos_limit(const Kv8Rows& r) {
  const int pages = (int)min((int64_t)r.max_pages * PAGE, (int64_t)kKv8MaxPos);
  return min(min(r.max_entries, pages), r.rope.cos == nullptr ? kKv8MaxPos : r.rope.rows);
}
__device__ __forceinline__ bool kv8_row_valid(const Kv8Rows& r, int b, int pos) {
  return b >= 0 && b < r.num_requests && pos >= 0 && pos < kv8_pos_limit(r);
}

// Eight bf16 to fp32, low half first.
__device__ __forceinline__ void bf16x8_to_f32(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rotation: a' = a*c - b*s, b' = b*c + a*s, each step rounded once, the result to bf16.  A
// pair's halves lie dims / 2 apart, a multiple of 8, so both are whole pieces of 8 dims.
// Place of the piece from dim i on: the other half's first dim, this one's table column and
// whether it is the lower half.  false: not rotated.
struct Kv8Turn {
  int other, column;
  bool lower;
};
__device__ __forceinline__ bool turn_of(const Kv8Rope& rope, int i, Kv8Turn& t) {
  const int half = rope.dims >> 1, at = i - rope.first;
  if (rope.cos == nullptr || at < 0 || at >= rope.dims) return false;
  t.lower = at < half;
  t.other = t.lower ? i + half : i - half;
  t.column = t.lower ? at : at - half;
  return true;
}
__device__ __forceinline__ uint4 turn8(uint4 mine, uint4 other, const Kv8Rope& rope, const Kv8Turn& t, int pos) {
  const size_t at = (size_t)pos * (rope.dims >> 1) + t.column;
  float x[8], y[8];
  // the lower half's b*s is subtracted: the same rounding as adding the negated product
  const uint32_t sign = t.lower ? 0x80008000u : 0u;
  bf16x8_to_f32(mine, x);
  bf16x8_to_f32(make_uint4(other.x ^ sign, other.y ^ sign, other.z ^ sign, other.w ^ sign), y);
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(rope.cos + at + k));
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(rope.sin + at + k));
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[k + j] = __fadd_rn(__fmul_rn(x[k + j], c[j]), __fmul_rn(y[k + j], s[j]));
  }
  return f32_to_bf16x8(x);
}
// Another lane's piece.
__device__ __forceinline__ uint4 of_lane(uint4 v, int from) {
  return make_uint4(__shfl_sync(0xFFFFFFFFu, v.x, from), __shfl_sync(0xFFFFFFFFu, v.y, from),
                    __shfl_sync(0xFFFFFFFFu, v.z, from), __shfl_sync(0xFFFFFFFFu, v.w, from));
}
// Dims i .. i + 7 (i a multiple of 8) of the head vector at vec, rotated at position pos.
__device__ __forceinline__ uint4 rotated8(const uint16_t* vec, int i, const Kv8Rope& rope, int pos) {
  const uint4 raw = __ldg(reinterpret_cast<const uint4*>(vec + i));
  Kv8Turn t;
  if (!turn_of(rope, i, t)) return raw;
  return turn8(raw, __ldg(reinterpret_cast<const uint4*>(vec + t.other)), rope, t, pos);
}

// Two fp32 to two E4M3 codes (round to nearest even, saturating; NaN stays NaN), a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_of(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_values(uint32_t codes) {
  const uint32_t h = e4m3x2_to_f16((uint16_t)codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The largest magnitude of eight bf16, in both halves; NaN if there is one.
__device__ __forceinline__ __nv_bfloat162 bf16x8_top(uint4 v) {
  auto two = [](uint32_t w) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)); };
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(two(v.x), two(v.y)), __hmax2_nan(two(v.z), two(v.w)));
  return __hmax2_nan(m, __lowhigh2highlow(m));
}
// That of a column, 8 each in LANES neighbouring lanes.
template <int LANES>
__device__ __forceinline__ float column_top(uint4 v) {
  __nv_bfloat162 m = bf16x8_top(v);
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    const uint32_t w = __shfl_xor_sync(0xFFFFFFFFu, *reinterpret_cast<const uint32_t*>(&m), o);
    m = __hmax2_nan(m, *reinterpret_cast<const __nv_bfloat162*>(&w));
  }
  return __low2float(m);
}

}  // namespace csa
