// csa_kv8_select: for each row and key head, the pages that a cheap score puts first.
//
// Mathematics.  score(j) = (max_g dot(qi_g, mi_j) * sq_g) * ss_j over the head's G queries,
// qi and mi int8.  A dot of int8 vectors is a whole number below 2^22, each product is
// rounded once and a maximum not at all, so the score has one value whatever the order of
// the work, and the selection is exact.
//
// k_kv8_score: whole numbers up to 2^11 are exact in fp16 and their products' sums below 2^24 in
// fp32, so the dots are tensor-core products (M = 16 pages, N = 8 queries, K = 16) of the codes as
// fp16.  A sum has no order, so a lane takes 32 consecutive dims of a page, two loads, as its places
// in all 8 steps, and the queries lie in shared memory to match.  A CTA has one head's 128 pages and
// the queries of up to kScoreCols columns; rows of one request follow one another, so a summary is
// read and converted once for them.  Where a key head has 1, 2, 4 or 8 queries their maximum is within
// a lane and its neighbours, and a warp goes on by itself; else products go through shared memory,
// where a thread has a page and takes the maximum over each row's queries.
// k_kv8_rank: one group of T threads per row and head, K consecutive pages a thread, their
// scores as ordered 32-bit keys in registers.  The need-th largest key is found bit by bit
// from the first in which ranked keys differ (the group counts the keys at or above the candidate; a
// count that is exactly `need` ends it); equal keys are taken from the lowest page on, and a prefix sum over the
// threads gives each selected page its place in ascending order.
//
// What bounds them.  One token over 128k tokens' 2048 pages takes 8.4 us, two launches and a chain of
// loads in each; 2048 rows of 32 heads over 8, each over 130 to 258 pages, 51 us: 36 of it the scores,
// a warp's chain of products and maxima with four warps a scheduler, and 17 the ranking.  Maxima through
// shared memory for these took 57; half as many pages a CTA 67 then, as each quantises its rows' queries
// anew; 32 columns a CTA 55, 96 columns 59, five CTAs a SM, at 102 registers a thread, 62.  A ranking
// that first drops the keys below the lanes' need-th largest took as long as this.
#include <algorithm>

#include "kv8_device.cuh"

namespace csa {

namespace {

constexpr int kScoreThreads = 128, kScoreCols = 64, kChunk = 32;   // columns of a CTA, at a time

// Four int8 to fp16, in order: 0x6400 | (c + 128) is 1152 + c.
__device__ __forceinline__ void int8x4_to_f16(uint32_t w, uint32_t (&o)[2]) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 bias = __float2half2_rn(-1152.0f);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t h = __byte_perm(u, 0x64646464u, k == 0 ? 0x4140 : 0x4342);
    const __half2 v = __hadd2(*reinterpret_cast<const __half2*>(&h), bias);
    o[k] = *reinterpret_cast<const uint32_t*>(&v);
  }
}
// Numbers as they are, zeros for the others.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}
constexpr float kWhole = 12582912.0f;            // 1.5 * 2^23: a sum with it is a whole number, ties to even
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t* a, uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}

// GR: queries of a key head where a lane's products and its neighbours' hold them (1, 2, 4, 8); 0: any number.
template <int D, int GR>
__global__ void __launch_bounds__(kScoreThreads, 4) k_kv8_score(Kv8SelectArgs a, int rows_per_cta, int chunks) {
  constexpr int kSteps = D / 16, kLane = D / 4;  // K steps; dims of a lane
  constexpr int kStride = D * 2 + 8;             // of a column's fp16 codes: lanes' banks differ
  __shared__ __align__(16) uint8_t s_q[kScoreCols + kChunk][kStride];
  __shared__ float s_scale[kScoreCols + kChunk];
  __shared__ float s_dot[GR ? 1 : kChunk][kScoreThreads + 4];
  __shared__ int s_req[kScoreCols], s_pos[kScoreCols], s_end[kScoreCols];
  const int tid = threadIdx.x, lane = lane_id(), warp = warp_id(), h = blockIdx.y, G = a.G, H = a.heads;
  const int r0 = blockIdx.x * rows_per_cta, rows = min(rows_per_cta, a.rows.num_rows - r0);
  pdl_trigger();                                 // the ranking waits for all of this before it reads scores
  // ---- the rows: request, and the end of the pages that they rank (0: none)
  constexpr int kPieces = D / 8, kAtOnce = kScoreThreads / kPieces;
  int end_of = 0;
  if (tid < rows) {
    const int b = __ldg(a.rows.row_req + r0 + tid), pos = __ldg(a.rows.row_pos + r0 + tid);
    if (kv8_row_valid(a.rows, b, pos)) end_of = (pos >> 6) + 1 - a.n_last;
    s_req[tid] = b;
    s_pos[tid] = pos;
    s_end[tid] = end_of;
  }
  if (!__syncthreads_or(end_of > max((int)blockIdx.z * kScoreThreads, a.n_first))) return;
  // ---- their queries, D / 8 lanes a column, four columns asked for at once
  const int i0 = 8 * (tid % kPieces);
  const Kv8Rope& rope = a.rows.rope;
  Kv8Turn turn{i0, 0, false};
  const bool turns = turn_of(rope, i0, turn);
  for (int c0 = tid / kPieces; c0 < rows * G + tid / kPieces; c0 += 4 * kAtOnce) {     // all lanes: they exchange
    uint4 raw[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u * kAtOnce, i = c / G;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (c < rows * G && s_end[i] > 0)
        raw[u] = __ldg(reinterpret_cast<const uint4*>(a.q + ((size_t)(r0 + i) * H * G + h * G + (c - i * G)) * D + i0));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u * kAtOnce;
      if (c - tid / kPieces >= rows * G) break;
      if (rope.cos != nullptr) {                 // a pair's other half is another lane's of the same column
        const int from = lane + (turn.other - i0) / 8;
        const uint4 other = of_lane(raw[u], from);
        if (turns && c < rows * G && s_end[c / G] > 0) raw[u] = turn8(raw[u], other, rope, turn, s_pos[c / G]);
      }
      float top = column_top<kPieces>(raw[u]);
      if (__any_sync(0xFFFFFFFFu, !(top <= 3.4028234663852886e38f))) {         // what is no number counts as 0
        raw[u] = make_uint4(finite_bf16x2(raw[u].x), finite_bf16x2(raw[u].y), finite_bf16x2(raw[u].z), finite_bf16x2(raw[u].w));
        top = column_top<kPieces>(raw[u]);
      }
      const bool some = top >= kKv8Least;
      const float inv = some ? __fdiv_rn(127.0f, top) : 0.0f;
      float x[8];
      bf16x8_to_f32(raw[u], x);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {           // |x| inv <= 127 (1 + 2^-23): the nearest whole number is at most 127
        const float2 y = make_float2(__fmul_rn(x[i], inv), __fmul_rn(x[i + 1], inv));    // never one step with the sum
        const float2 z = add2(add2(y, make_float2(kWhole, kWhole)), make_float2(-kWhole, -kWhole));
        const __half2 v = __floats2half2_rn(z.x, z.y);
        w[i / 2] = *reinterpret_cast<const uint32_t*>(&v);
      }
      if (c < rows * G) {                        // dims 4 s .. 4 s + 3 of a lane's share lie together: 8 bytes
        *reinterpret_cast<uint2*>(&s_q[c][2 * i0]) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(&s_q[c][2 * i0 + 8]) = make_uint2(w[2], w[3]);
        if (i0 == 0) s_scale[c] = some ? top : 0.0f;
      }
    }
  }
  __syncthreads();                               // queries are in place
  if (tid < rows * G) s_scale[tid] = __fdiv_rn(s_scale[tid], 127.0f);
  __syncthreads();
  const int t = lane & 3, p = lane >> 2;         // a lane's share of the dims, its page of 8
  [[maybe_unused]] const int together = G <= kChunk ? kChunk / G : 1;   // rows at a time
  for (int i = 0; i < rows;) {
    // ---- rows of one request
    const int b = s_req[i];
    int end = i + 1, most = s_end[i];
    for (; end < rows && s_req[end] == b; ++end) most = max(most, s_end[end]);
    for (int chunk = blockIdx.z; chunk < chunks && chunk * kScoreThreads < most; chunk += gridDim.z) {
      // its pages: a warp has two sixteens, a lane rows p and p + 8 of each
      const int j0 = chunk * kScoreThreads;
      if (GR && j0 + 32 * warp >= most) break;   // no pages for this warp, and none after
      uint32_t m[2][kSteps][4];
      [[maybe_unused]] float ssm[2][2];          // its pages' scales; NaN's payload would not do for a page that is not there
      uint32_t there = 0;
      const int32_t* table = a.page_table + (size_t)b * a.rows.max_pages;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = j0 + 32 * warp + 16 * s + p + 8 * k;
          const int page = j < most ? __ldg(table + j) : -1;
          const bool in = (uint32_t)page < (uint32_t)a.num_pages;
          there |= (uint32_t)in << (2 * s + k);
          if constexpr (GR > 0) ssm[s][k] = in ? __ldg(a.sum_scale + (size_t)page * H + h) : 0.0f;
          uint4 v[kLane / 16];
#pragma unroll
          for (int e = 0; e < kLane / 16; ++e) {
            v[e] = make_uint4(0u, 0u, 0u, 0u);
            if (in)
              v[e] = __ldg(reinterpret_cast<const uint4*>(a.sum_codes + ((size_t)page * H + h) * D + kLane * t) + e);
          }
#pragma unroll
          for (int e = 0; e < kSteps; ++e) {
            const uint32_t word[4] = {v[e / 4].x, v[e / 4].y, v[e / 4].z, v[e / 4].w};
            uint32_t o[2];
            int8x4_to_f16(word[e & 3], o);
            m[s][e][k] = o[0];
            m[s][e][2 + k] = o[1];
          }
        }
      if constexpr (GR > 0) {
        // ---- eight columns, 8 / GR rows, at a time
#pragma unroll 1
        for (int c0 = i * GR; c0 < end * GR; c0 += 8) {
          float d[2][4] = {};
#pragma unroll
          for (int e = 0; e < kSteps; ++e) {
            const uint2 q = *reinterpret_cast<const uint2*>(&s_q[c0 + p][2 * kLane * t + 8 * e]);
            mma_16x8x16(d[0], m[0][e], q);
            mma_16x8x16(d[1], m[1][e], q);
          }
          const float sq[2] = {s_scale[c0 + 2 * t], s_scale[c0 + 2 * t + 1]};
#pragma unroll
          for (int u = 0; u < (GR == 1 ? 2 : 1); ++u) {
            const int r = (c0 + 2 * t + u) / GR, n = r < end ? s_end[r] : 0;
            float* dst = a.scores + ((size_t)(r0 + r) * H + h) * a.ld;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float best = __fmul_rn(d[s][2 * k + u], sq[u]);
                if (GR > 1) best = fmaxf(best, __fmul_rn(d[s][2 * k + 1], sq[1]));
#pragma unroll
                for (int o = 1; 2 * o < GR; o <<= 1) best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
                // one of a row's lanes has the number; pages at either end take part without a score
                const int j = j0 + 32 * warp + 16 * s + p + 8 * k;
                if ((GR <= 2 || (t & (GR / 2 - 1)) == ((2 * s + k) & (GR / 2 - 1))) && j >= a.n_first && j < n) {
                  const bool in = (there >> (2 * s + k)) & 1u;
                  if (!in) raise_flag(a.status, CSA_FLAG_PAGE_OOB);
                  dst[j] = in ? __fmul_rn(best, ssm[s][k]) : -INFINITY;
                }
              }
          }
        }
        continue;
      }
      // the thread's own page, for the maxima
      const int j = j0 + tid;
      const int page = j < most ? __ldg(table + j) : -1;
      const bool in_pool = (uint32_t)page < (uint32_t)a.num_pages;
      const float ss = in_pool ? __ldg(a.sum_scale + (size_t)page * H + h) : 0.0f;
      for (int r = i; r < end; r += together) {
        const int n_rows = min(together, end - r);
        float best = -INFINITY;
        for (int g0 = 0; g0 < G; g0 += kChunk) { // more than once for more than kChunk queries a row
          const int c0 = r * G + g0, cols = G <= kChunk ? n_rows * G : min(kChunk, G - g0);
          __syncthreads();                       // the products before have been read
#pragma unroll
          for (int n = 0; n < kChunk; n += 8) {
            if (n >= cols) break;
            float d[2][4] = {};
#pragma unroll
            for (int e = 0; e < kSteps; ++e) {
              const uint2 q = *reinterpret_cast<const uint2*>(&s_q[c0 + n + p][2 * kLane * t + 8 * e]);
              mma_16x8x16(d[0], m[0][e], q);
              mma_16x8x16(d[1], m[1][e], q);
            }
            const float sq[2] = {s_scale[c0 + n + 2 * t], s_scale[c0 + n + 2 * t + 1]};
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                s_dot[n + 2 * t + (k & 1)][32 * warp + 16 * s + p + 8 * (k >> 1)] = __fmul_rn(d[s][k], sq[k & 1]);
          }
          __syncthreads();
          const int each = G <= kChunk ? G : cols;
          for (int k = 0; k < n_rows; ++k) {
            if (G <= kChunk) best = -INFINITY;
#pragma unroll 4
            for (int c = 0; c < each; ++c) best = fmaxf(best, s_dot[k * each + c][tid]);
            // pages at either end take part without a score
            if (g0 + kChunk >= G && j >= a.n_first && j < s_end[r + k]) {
              if (!in_pool) raise_flag(a.status, CSA_FLAG_PAGE_OOB);
              a.scores[((size_t)(r0 + r + k) * H + h) * a.ld + j] = in_pool ? __fmul_rn(best, ss) : -INFINITY;
            }
          }
        }
      }
    }
    i = end;
  }
}

// fp32 as an unsigned number of the same order; +0 and -0 alike, what is no number as -inf.
__device__ __forceinline__ uint32_t ordered(float v) {
  if (v != v) v = -INFINITY;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int T>
struct RankSmem {
  int part[2][T / 32];
};
// Sum over the group; `turn` alternates between calls.
template <int T>
__device__ __forceinline__ int group_sum(int v, RankSmem<T>& sm, int turn) {
  v = __reduce_add_sync(0xFFFFFFFFu, v);
  if constexpr (T > 32) {
    if (lane_id() == 0) sm.part[turn & 1][warp_id()] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) v += sm.part[turn & 1][w];
  }
  return v;
}
// Sum over the threads before this one.
template <int T>
__device__ __forceinline__ int group_before(int v, RankSmem<T>& sm, int turn) {
  int sum = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane_id() >= o) sum += y;
  }
  if constexpr (T > 32) {
    if (lane_id() == 31) sm.part[turn & 1][warp_id()] = sum;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / 32; ++w)
      if (w < warp_id()) sum += sm.part[turn & 1][w];
  }
  return sum - v;
}

template <int T>
__device__ __forceinline__ uint32_t group_max(uint32_t v, RankSmem<T>& sm, int turn) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  if constexpr (T > 32) {
    if (lane_id() == 0) sm.part[turn & 1][warp_id()] = (int)v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / 32; ++w) v = max(v, (uint32_t)sm.part[turn & 1][w]);
  }
  return v;
}

template <int T, int K, int GROUPS>
__global__ void __launch_bounds__(T * GROUPS) k_kv8_rank(Kv8SelectArgs a) {
  __shared__ RankSmem<T> s_group[GROUPS];
  pdl_wait();
  const int which = T == 32 ? warp_id() : 0, tid = T == 32 ? lane_id() : threadIdx.x;
  const int64_t at = (int64_t)blockIdx.x * GROUPS + which;
  if (at >= (int64_t)a.rows.num_rows * a.heads) return;
  RankSmem<T>& sm = s_group[which];
  const int r = (int)(at / a.heads), M = a.n_blocks;
  const int b = __ldg(a.rows.row_req + r), pos = __ldg(a.rows.row_pos + r);
  int32_t* out = a.blocks + at * M;
  if (!kv8_row_valid(a.rows, b, pos)) {
    if (tid == 0) raise_flag(a.status, CSA_FLAG_ROW_INVALID);
    for (int i = tid; i < M; i += T) out[i] = -1;
    return;
  }
  const int n = (pos >> 6) + 1, need = min(M, n);
  // ---- keys: 0 past the row's pages, all ones for those that take part without a score
  uint32_t key[K];
  const float* src = a.scores + at * a.ld;
#pragma unroll
  for (int k = 0; k < K; k += 4) {
    const int j = tid * K + k;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (j < n) v = __ldcg(reinterpret_cast<const float4*>(src + j));   // ld is a multiple of 4
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool always = j + i < a.n_first || j + i >= n - a.n_last;
      key[k + i] = j + i >= n ? 0u : (always ? 0xFFFFFFFFu : ordered(f[i]));
    }
  }
  uint32_t cut = 0;
  int turn = 0, ties = need;
  bool exact = need == n;
  if (!exact) {
    // what all ranked keys have in common needs no counting
    uint32_t most = 0, least = 0xFFFFFFFFu;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool ranked = key[k] != 0u && key[k] != 0xFFFFFFFFu;
      most = max(most, ranked ? key[k] : 0u);
      least = min(least, ranked ? key[k] : 0xFFFFFFFFu);
    }
    most = group_max<T>(most, sm, turn++);
    least = ~group_max<T>(~least, sm, turn++);
    const int top = 31 - __clz(most ^ least);     // -1: one value, or none is ranked
    cut = top < 0 ? most : most & ~((2u << top) - 1u);
#pragma unroll 1
    for (int bit = top; bit >= 0; --bit) {
      const uint32_t t = cut | (1u << bit);
      int c = 0;
#pragma unroll
      for (int k = 0; k < K; ++k) c += key[k] >= t;
      c = group_sum<T>(c, sm, turn++);
      if (c >= need) cut = t;
      if (c == need) {
        exact = true;
        break;
      }
    }
    if (!exact) {                                // more keys equal the cut than are needed
      int c = 0;
#pragma unroll
      for (int k = 0; k < K; ++k) c += key[k] > cut;
      ties = need - group_sum<T>(c, sm, turn++);
    }
  } else {
    cut = 1u;                                    // every page of the row
  }
  // ---- which of the thread's pages, and where they go
  uint64_t chosen = 0;
  if (exact) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (key[k] >= cut) chosen |= 1ull << k;
  } else {
    int c = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) c += key[k] == cut;
    int before = group_before<T>(c, sm, turn++);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (key[k] > cut || (key[k] == cut && before < ties)) chosen |= 1ull << k;
      before += key[k] == cut;
    }
  }
  int place = group_before<T>(__popcll(chosen), sm, turn++);
  while (chosen) {
    const int k = __ffsll((long long)chosen) - 1;
    chosen &= chosen - 1;
    if (place < M) out[place] = tid * K + k;
    ++place;
  }
  for (int i = need + tid; i < M; i += T) out[i] = -1;
}

template <int T, int K, int GROUPS>
cudaError_t launch_rank(const Kv8SelectArgs& a, cudaStream_t stream) {
  const int64_t groups = (int64_t)a.rows.num_rows * a.heads;
  return launch_kernel(Order::kChained, k_kv8_rank<T, K, GROUPS>, dim3((unsigned)((groups + GROUPS - 1) / GROUPS)),
                       dim3(T * GROUPS), 0, stream, a);
}

template <int D>
cudaError_t launch_score(const Kv8SelectArgs& a, dim3 grid, int per, int chunks, cudaStream_t stream) {
  auto launch = [&](auto kernel) {
    return launch_kernel(Order::kStream, kernel, grid, dim3(kScoreThreads), 0, stream, a, per, chunks);
  };
  switch (a.G) {
    case 1: return launch(k_kv8_score<D, 1>);
    case 2: return launch(k_kv8_score<D, 2>);
    case 4: return launch(k_kv8_score<D, 4>);
    case 8: return launch(k_kv8_score<D, 8>);
    default: return launch(k_kv8_score<D, 0>);
  }
}

int32_t score_ld(int32_t max_entries) { return (int32_t)((kv8_pages(max_entries) + 31) / 32 * 32); }

}  // namespace

size_t kv8_select_ws_bytes(int32_t num_rows, int32_t max_entries, int32_t heads) {
  return sizeof(float) * (size_t)num_rows * heads * score_ld(max_entries);
}

cudaError_t launch_kv8_select(Kv8SelectArgs a, void* ws, cudaStream_t stream) {
  a.scores = static_cast<float*>(ws);
  a.ld = score_ld(a.rows.max_entries);
  const int pages = (int)kv8_pages(a.rows.max_entries);
  const int per = std::max(1, std::min(kScoreCols / a.G, a.rows.max_rows_per_req));
  // a CTA takes several chunks of pages where there are rows enough to fill the GPU (above)
  const int tiles = (a.rows.num_rows + per - 1) / per, chunks = (pages + kScoreThreads - 1) / kScoreThreads;
  const int split = (int)std::max<int64_t>(1, std::min<int64_t>(chunks, 1024 / ((int64_t)tiles * a.heads)));
  const dim3 grid((unsigned)tiles, (unsigned)a.heads, (unsigned)split);
  const cudaError_t e = a.dim == 64 ? launch_score<64>(a, grid, per, chunks, stream) : launch_score<128>(a, grid, per, chunks, stream);
  if (e != cudaSuccess) return e;
  // a warp a group as long as its keys stay in few registers: 16 a thread from there on
  if (pages <= 128) return launch_rank<32, 4, 4>(a, stream);
  if (pages <= 256) return launch_rank<32, 8, 4>(a, stream);
  if (pages <= 384) return launch_rank<32, 12, 4>(a, stream);
  if (pages <= 512) return launch_rank<32, 16, 4>(a, stream);
  if (pages <= 2048) return launch_rank<128, 16, 1>(a, stream);
  if (pages <= 8192) return launch_rank<512, 16, 1>(a, stream);
  return launch_rank<512, 32, 1>(a, stream);
}

}  // namespace csa
