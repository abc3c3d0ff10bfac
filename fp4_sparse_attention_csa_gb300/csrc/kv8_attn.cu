// csa_kv8_attn, csa_kv8_block_attn: softmax attention of grouped query heads over the 8-bit
// paged cache, all positions up to the row's own or those of listed pages.
//
// Mathematics.  A segment is one key head and up to COLS / G rows of one request at
// consecutive positions (one row where pages are listed); its columns, G queries a row,
// share keys.  Tiles are two pages, 128 keys.  Per tile S^T = K Q^T (M = 128 keys),
// p = 2^(s - m), O^T += V^T P^T (M = dims), both products in E4M3 with fp32 sums on
// operands as they lie in the pages: nothing is converted but Q and P.
//   Q: a bf16 number has 8 bits and E4M3 holds 4, so a query scaled to [128, 256) is
// hi + lo / 16 with E4M3 parts, exact but for elements below 2^-13 of the largest.  The
// parts are columns c and COLS + c of one product, S = S_hi + S_lo / 16.
//   P: the page's value scale sv goes into the exponent, y = 2^(s + log2 sv - m) with m the
// running maximum of s + log2 sv: what y is small against is then what its contribution to O
// is small against.  y = hi + mid / 16 + lo / 512 in E4M3 parts, to 2^-12 of itself and 2^-18
// where the column's largest is at least 64: fp16's range, so that a long context's many small
// probabilities are not lost beside a large one.  Each part has columns of its own in O.
// The softmax's sum is l = sum of y / sv, in units of a power of two near 1 / sv.  That holds while a
// segment's value scales lie within kKv8Near of its first tile's; from the first page on that does not, or
// has no values at all (a scale of 0), the sum is formed with a maximum and powers of two of its own,
// l = sum of 2^(s - ms): y may have none of a key that the sum is made of, and the other way round.  What y
// is taken against is then held relative to ms.
// The key scale, the query's power of two and the softmax scale are the logit's factor.
//
// Work: the tiles of all segments, in row and head order, are one list; CTA i takes the i-th
// equal share.  A segment inside one share is written out directly; the parts of a cut one
// leave O / l and (m, l) in the workspace (at most two a CTA) and k_kv8_merge joins them in
// CTA order.
//
// Pipeline: 4 softmax warps, one key a thread, which also convert queries and write out; one
// warp that copies pages (one bulk copy a side), one that issues the products.  Several CTAs
// per SM overlap one another's chains, so inside a CTA only the copies run ahead.
//
// What bounds it.  With few columns HBM: 64 rows of 64 heads over 8 key heads of 128 at 4k to 64k
// tokens take 435 us for the 2.91 GB that they have to read, 6.68 TB/s of 6.68 measured for a copy.
// Lists of 16 pages for each of 2048 rows read 4.3 GB from L2 in 486 us, 8.9 TB/s: the chain of a
// tile (2200 clocks: S, probabilities, their product) and of a step between segments (another 5600:
// output, queries, first maximum), each overlapped by the two other CTAs of the SM; queries asked for
// ahead of the output before them left the time as it was.  One token after
// 4096 takes 11.3 us, one step after another: the parts more than half of it, some 1 until the join
// begins, the rest in it.  From 16 columns on the softmax's instructions count, each column's three parts above
// all: 32 requests at 4k to 6k tokens, 4 key heads of 64, take 27 us with 7 columns a group, 35 with
// 14 and 57 with 28.  Segments whose value scales are far apart read each tile's logits three times.
#include <algorithm>

#include "kv8_list.cuh"

namespace csa {

namespace {

constexpr int kThreads = 192, kSoftmaxThreads = 128, kCopyWarp = 4, kMmaWarp = 5;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// y is 2^kTop at the running maximum, which moves when it is exceeded by kSlack: y <= 446,
// inside E4M3's 448, what hi leaves is at most 16 and what mid leaves 1/2.
constexpr float kTop = 6.0f, kSlack = 2.8f;
constexpr float kMid = 16.0f, kLo = 512.0f;
constexpr float kNoMax = -3e38f;                 // running maximum of a column that has seen nothing
// ---- shared memory ---------------------------------------------------------------------
template <int COLS, int D>
struct Shape {
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kScoreBufs = 2;                        // S of this many tiles in tensor memory
  static constexpr int kParts = (3 * COLS + 15) / 16 * 16;    // columns of P and O: hi, mid and lo, in whole sixteens
  static constexpr uint32_t kOut = kScoreBufs * 2 * COLS;     // tensor memory columns: S, then O's three parts
  static constexpr uint32_t kNeed = kOut + kParts;
  static constexpr uint32_t kTmem = kNeed <= 64 ? 64 : (kNeed <= 128 ? 128 : 256);
  static constexpr int kValueSlot = 64 * D + 16;              // a page's values and its scales
  static constexpr int kStage = 128 * D + 2 * kValueSlot;
  static constexpr int kProbChunk = 128, kProbRows = 8 * kProbChunk;   // 16 keys, 8 columns of P
};
template <int COLS, int D>
struct Smem {
  using X = Shape<COLS, D>;
  uint8_t stage[X::kStages][X::kStage];          // keys of two pages, then each one's values and scales
  uint8_t q[2 * COLS * D];
  uint8_t p[X::kParts / 8 * X::kProbRows];      // columns' hi, mid and lo
  // the values' product reads 128 dims: with 64, another 4096 bytes behind a page's, in the last place's case these
  static constexpr int kBehind = 2 * COLS * D + X::kParts / 8 * X::kProbRows;
  uint8_t pad[D == 64 && kBehind < 4096 ? 4096 - kBehind : 16];
  int first_pos[X::kStages][2];                  // position of a page's first slot; INT_MAX: no page
  float factor[COLS];                            // of a column's logits (log2 units)
  float neg_m[COLS];                             // kTop minus the running maximum; once scales are far apart, beside neg_l
  float neg_l[COLS];                             // minus the sums' own maximum by then
  int far, large;                                // a page's scale is, in this tile; a column's maximum is (kKv8Large)
  float red[4][COLS];                            // per warp: maxima of a tile, sums of p
  float corr[COLS];                              // correction of a column whose maximum moved; at the end 1 / l
  int out_row[COLS];                             // a column's row of the output
  uint64_t full[X::kStages], free[X::kStages];
  uint64_t s_full[2], p_full, p_free, q_full, o_full, drain;
  uint32_t tmem_base;
  volatile int abort;                            // a wait ran out: every role leaves
  ShareScratch<kThreads> share;
};


// ---- pages ---------------------------------------------------------------------------------
template <int COLS, int D>
__device__ __forceinline__ void copy_pages(const Kv8AttnArgs& a, Smem<COLS, D>& sm, const Share& sh, int RG) {
  using X = Shape<COLS, D>;
  const int lane = lane_id();
  Walk w;
  uint32_t i = 0;
  bool ok = true;
  for (bool more = w.first(a, RG, sh); more && ok; more = w.next_segment(a, RG)) {
    if (w.t >= w.t_end) continue;
    int above = -1;
    bool ended = false;
    int chunk = -1;
    Pages x{INT_MAX, -1};
    if (a.blocks) {
      while (chunk + 1 < w.t >> 4) x = pages_of<true>(a, w.gr, w.h, ++chunk, above, ended);
    } else {
      chunk = (w.t >> 4) - 1;
    }
    Pages next = pages_of<true>(a, w.gr, w.h, chunk + 1, above, ended);
    for (; w.t < w.t_end; ++w.t, ++i) {
      if (w.t >> 4 != chunk) {
        chunk = w.t >> 4;
        x = next;
        if (32 * (chunk + 1) < 2 * w.t_end) next = pages_of<true>(a, w.gr, w.h, chunk + 1, above, ended);
      }
      const uint32_t st = i % X::kStages;
      ok = __all_sync(0xFFFFFFFFu, wait_or_abort(&sm.free[st], ((i / X::kStages) & 1) ^ 1, a.wait_budget, &sm.abort));
      if (!ok) break;
      int j[2], page[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        j[k] = __shfl_sync(0xFFFFFFFFu, x.j, (2 * w.t + k) & 31);
        page[k] = __shfl_sync(0xFFFFFFFFu, x.page, (2 * w.t + k) & 31);
      }
      if (lane == 0) {
        uint32_t bytes = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          sm.first_pos[st][k] = j[k] == INT_MAX ? INT_MAX : j[k] * PAGE;
          if (j[k] != INT_MAX) bytes += 64 * D + X::kValueSlot;
        }
        mbar_expect_tx(&sm.full[st], bytes);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (j[k] == INT_MAX) continue;
          const uint8_t* rec = a.pool + kv8_record<D>(page[k], a.heads, w.h);
          bulk_load(sm.stage[st] + k * 64 * D, rec, 64 * D, &sm.full[st]);
          bulk_load(sm.stage[st] + 128 * D + k * X::kValueSlot, rec + 64 * D, X::kValueSlot, &sm.full[st]);
        }
      }
      __syncwarp();
    }
    if (w.t_end == w.gr.tiles) end_of_list(a, w.gr, w.h, ended);
  }
  // after a wait that ran out: what is still being copied must land before the CTA ends
  if (lane == 0)
    for (uint32_t k = i > X::kStages ? i - X::kStages : 0; k < i; ++k) (void)mbar_wait(&sm.full[k % X::kStages], (k / X::kStages) & 1);
}

// ---- products --------------------------------------------------------------------------------
template <int COLS, int D>
struct Products {
  using X = Shape<COLS, D>;
  const Kv8AttnArgs& a;
  Smem<COLS, D>& sm;
  uint32_t tmem;
  bool started;                                  // O of the segment holds something

  // Asleep, but for a segment's queries: polling took issue slots from the softmax warps beside it (a list for
  // each of 4 x 512 rows: 493 us instead of 482).
  template <bool kPoll = false>
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, wait_or_abort<kPoll>(bar, parity, a.wait_budget, &sm.abort));
  }
  // The whole warp walks and waits, operands' addresses are uniform, and one elected lane issues.
  __device__ __forceinline__ void scores(uint32_t i) {
    const uint64_t k = smem_desc(smem_u32(sm.stage[0]), 128, 8 * D, kSwizzleNone) + (i % X::kStages) * (X::kStage / 16);
    const uint64_t q = smem_desc(smem_u32(sm.q), 128, 8 * D, kSwizzleNone);
    const uint32_t d = tmem + (i % X::kScoreBufs) * 2 * COLS;
    if (elect_one()) {
#pragma unroll
      for (int s = 0; s < D / 32; ++s) mma_f8(d, k + 16 * s, q + 16 * s, idesc_e4m3(128, 2 * COLS), s > 0);
      tc_commit(&sm.s_full[i % X::kScoreBufs]);
    }
    __syncwarp();
  }
  // O^T += V^T P^T of tile i; pages that are not there are left out, what their place holds may be NaN
  __device__ __forceinline__ bool values(uint32_t i, bool first, bool last) {
    if (!wait(&sm.p_full, i & 1)) return false;
    tc_fence_after();
    if (first) started = false;
    const uint32_t st = i % X::kStages;
    const bool there[2] = {sm.first_pos[st][0] != INT_MAX, sm.first_pos[st][1] != INT_MAX};
    const uint64_t v = smem_desc(smem_u32(sm.stage[0]) + 128 * D, 128, 512, kSwizzleNone) + st * (X::kStage / 16);
    const uint64_t p = smem_desc(smem_u32(sm.p), X::kProbChunk, X::kProbRows, kSwizzleNone);
    if (elect_one()) {
      bool acc = started;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!there[k]) continue;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          mma_f8(tmem + X::kOut, v + k * (X::kValueSlot / 16) + 16 * s, p + (4 * k + 2 * s) * (X::kProbChunk / 16),
                 idesc_e4m3(128, X::kParts), acc);
          acc = true;
        }
      }
      tc_commit(&sm.free[st]);
      tc_commit(&sm.p_free);
      if (last) tc_commit(&sm.o_full);
    }
    started = started || there[0] || there[1];
    __syncwarp();
    return true;
  }
  __device__ __forceinline__ void run(const Share& sh, int RG) {
    Walk w;
    uint32_t i = 0, seg = 0;
    bool before = false, before_first = false, before_last = false, ok = true;   // the tile before: its P is not used yet
    for (bool more = w.first(a, RG, sh); more && w.settle(a, RG); ++i, ++w.t) {
      const bool first = w.t == w.t0, last = w.t + 1 == w.t_end;
      if (before && first) {
        if (!(ok = values(i - 1, before_first, before_last))) break;
        before = false;
      }
      if (first && !(ok = wait<true>(&sm.q_full, seg++ & 1))) break;
      if (!(ok = wait(&sm.full[i % X::kStages], (i / X::kStages) & 1))) break;
      tc_fence_after();
      scores(i);
      if (before && !(ok = values(i - 1, before_first, before_last))) break;
      before = true;
      before_first = first;
      before_last = last;
    }
    if (ok && before) (void)values(i - 1, before_first, before_last);
    // everything issued is complete before the tensor memory is given back
    if (lane_id() == 0) {
      tc_commit(&sm.drain);
      (void)mbar_wait(&sm.drain, 0);
    }
    __syncwarp();
  }
};

// ---- queries -----------------------------------------------------------------------------------
// Columns to E4M3 parts, D / 8 lanes a column, and each one's factor and output row.
template <int COLS, int D>
__device__ __forceinline__ void convert_queries(const Kv8AttnArgs& a, Smem<COLS, D>& sm, const Group& gr, int h) {
  constexpr int kPieces = D / 8, kAtOnce = kSoftmaxThreads / kPieces;
  const int tid = threadIdx.x, i0 = 8 * (tid % kPieces), G = a.G;
#pragma unroll 1
  for (int c = tid / kPieces; c < COLS; c += kAtOnce) {
    const int i = c / G, row = (gr.r0 + i) * a.heads * G + h * G + (c - i * G);
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (i < gr.g) raw = rotated8(a.q + (size_t)row * D, i0, a.rows.rope, gr.p0 + i);
    const float big = column_top<kPieces>(raw);
    float x[8];
    bf16x8_to_f32(raw, x);
    // 2^-e puts the largest magnitude in [128, 256); e >= -126 keeps it in fp32's range, and a
    // query of such small elements has no logit to speak of
    const int ex = (int)(__float_as_uint(big) >> 23);
    const int e = (ex > 0 && ex < 255) ? max(ex - 127 - 7, -126) : 0;
    const float f = pow2(-e);
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float y0 = x[k] * f, y1 = x[k + 1] * f;
      const uint32_t code = e4m3x2_of(y0, y1);
      const uint32_t h2 = e4m3x2_to_f16((uint16_t)code);
      const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      const uint32_t rest = e4m3x2_of((y0 - back.x) * 16.0f, (y1 - back.y) * 16.0f);
      hi[k >> 2] = (k & 2) ? hi[k >> 2] | (code << 16) : code;
      lo[k >> 2] = (k & 2) ? lo[k >> 2] | (rest << 16) : rest;
    }
    uint8_t* dst = sm.q + (c >> 3) * 8 * D + (i0 >> 4) * 128 + (c & 7) * 16 + (i0 & 15);
    *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2*>(dst + COLS * D) = make_uint2(lo[0], lo[1]);
    if (i0 == 0) {
      // NaN where an element is infinite or not a number
      sm.factor[c] = fmaf(big, 0.0f, a.softmax_scale * kLog2e * pow2(e));
      sm.neg_m[c] = -kNoMax;
      sm.out_row[c] = row;
    }
  }
}

// ---- softmax -------------------------------------------------------------------------------------
template <int COLS, int D>
struct Logits {
  static constexpr int CH = COLS < 16 ? COLS : 16;   // columns at a time
  Smem<COLS, D>& sm;
  uint32_t tmem;                                 // with the warp's lanes
  int tid, warp, lane;

  // S_hi + S_lo / 16 of columns c0 .. c0 + CH - 1
  __device__ __forceinline__ void load_scores(uint32_t at, int c0, float (&v)[CH]) {
    uint32_t t[16], u[16];
    tmem_ld16(tmem + at + c0, t);
    if constexpr (COLS >= 16) tmem_ld16(tmem + at + COLS + c0, u);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      asm volatile("" : "+r"(t[k]));
      if constexpr (COLS >= 16) asm volatile("" : "+r"(u[k]));
    }
#pragma unroll
    for (int k = 0; k < CH; ++k)
      v[k] = fmaf(__uint_as_float(COLS >= 16 ? u[k] : t[8 + k % 8]), 0.0625f, __uint_as_float(t[k]));
  }
  // logits (log2 units) plus lsv and `add` of each column; -inf where the column does not see the key
  __device__ __forceinline__ void logits(uint32_t at, int c0, float sk, float lsv, int clo, bool masked, const float* add,
                                         float* x) {
    float v[CH];
    load_scores(at, c0, v);
#pragma unroll
    for (int k = 0; k < CH; k += 4) {
      const float4 f = *reinterpret_cast<const float4*>(sm.factor + c0 + k);
      const float4 m = add ? *reinterpret_cast<const float4*>(add + c0 + k) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      x[k] = fmaf(v[k], sk * f.x, m.x + lsv);
      x[k + 1] = fmaf(v[k + 1], sk * f.y, m.y + lsv);
      x[k + 2] = fmaf(v[k + 2], sk * f.z, m.z + lsv);
      x[k + 3] = fmaf(v[k + 3], sk * f.w, m.w + lsv);
    }
    if (masked) {
#pragma unroll
      for (int k = 0; k < CH; ++k)
        if (c0 + k < clo) x[k] = -INFINITY;
    }
  }

  // The tile's largest s + lsv of each column, the warps' to red; then a column's over all warps.
  __device__ __forceinline__ void tile_tops(uint32_t at, float sk, float lsv, int clo, bool masked) {
#pragma unroll 1
    for (int c0 = 0; c0 < COLS; c0 += CH) {
      float y[CH];
      logits(at, c0, sk, lsv, clo, masked, nullptr, y);
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const float t = warp_top(y[k]);
        if (lane == 0) sm.red[warp][c0 + k] = t;
      }
    }
    group_sync(1);
  }
  __device__ __forceinline__ float tile_top() {
    return fmaxf(fmaxf(sm.red[0][tid], sm.red[1][tid]), fmaxf(sm.red[2][tid], sm.red[3][tid]));
  }
};

// A tile where sums have a maximum of their own: l, O's corrections and the logits from its maxima.  l counts from neg_l,
// minus the largest s, and O from neg_l + neg_m: a difference of two large numbers would say nothing of value scales.
// units: of l in the first such tile, where it and O count from neg_m; -inf in later ones.  All threads of the four warps.
// Seldom called, and kept out of the loop that calls it.
template <int COLS, int D>
__device__ __noinline__ void far_tile(Smem<COLS, D>& sm, uint32_t tmem, uint32_t at, float sk, float lsv, int clo, float units,
                                      float* l, float* x) {
  Logits<COLS, D> s{sm, tmem, (int)threadIdx.x, warp_id(), lane_id()};
  constexpr int CH = Logits<COLS, D>::CH;
  float rel = 0.0f, shift = 0.0f;
  s.tile_tops(at, sk, 0.0f, clo, true);
  if (s.tid < COLS) {
    const float n = sm.neg_m[s.tid], before = units == -INFINITY ? sm.neg_l[s.tid] : n + units;
    const float now = fminf(before, -s.tile_top());
    rel = units == -INFINITY || !(n < -kNoMax) ? n : -units;          // that of a column that has seen nothing stays so
    shift = now - before;
    sm.corr[s.tid] = ex2(shift);
    sm.neg_l[s.tid] = now;
  }
  group_sync(1);
#pragma unroll 1
  for (int c0 = 0; c0 < COLS; c0 += CH) {
    s.logits(at, c0, sk, 0.0f, clo, true, nullptr, x + c0);
#pragma unroll 1
    for (int c = c0; c < c0 + CH; ++c) {
      x[c] += sm.neg_l[c];
      l[c] = fmaf(l[c], sm.corr[c], ex2(x[c]));
      x[c] += lsv;
      const float t = warp_top(x[c]);
      if (s.lane == 0) sm.red[s.warp][c] = t;
    }
  }
  group_sync(1);
  if (s.tid < COLS) {
    const float next = fminf(rel < -kNoMax ? rel - shift : rel, kTop - s.tile_top());
    sm.corr[s.tid] = ex2(shift + (next - rel));
    sm.neg_m[s.tid] = next;
  }
  group_sync(1);
#pragma unroll 1
  for (int c = 0; c < COLS; ++c) x[c] += sm.neg_m[c];
}
// A tile's differences to its maxima where these are large (kKv8Large).
template <int COLS, int D>
__device__ __noinline__ void large_logits(Smem<COLS, D>& sm, uint32_t tmem, uint32_t at, float sk, float lsv, int clo, float* x) {
  Logits<COLS, D> s{sm, tmem, (int)threadIdx.x, warp_id(), lane_id()};
#pragma unroll 1
  for (int c0 = 0; c0 < COLS; c0 += Logits<COLS, D>::CH) {
    s.logits(at, c0, sk, lsv, clo, true, nullptr, x + c0);
#pragma unroll 1
    for (int k = 0; k < Logits<COLS, D>::CH; ++k) x[c0 + k] += sm.neg_m[c0 + k];
  }
}

// O times neg_l, a factor by then.
template <int COLS, int D>
__device__ __noinline__ void scale_out(Smem<COLS, D>& sm, uint32_t tmem) {
  using X = Shape<COLS, D>;
#pragma unroll 1
  for (int c0 = 0; c0 < X::kParts; c0 += 16) {
    uint32_t u[16];
    tmem_ld16(tmem + X::kOut + c0, u);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      asm volatile("" : "+r"(u[k]));             // not before the wait
      u[k] = __float_as_uint(__uint_as_float(u[k]) * sm.neg_l[(c0 + k) % COLS]);
    }
    tmem_st16(tmem + X::kOut + c0, u);
  }
  tmem_st_wait();
}

template <int COLS, int D>
struct Softmax : Logits<COLS, D> {
  using X = Shape<COLS, D>;
  using L = Logits<COLS, D>;
  using L::CH, L::sm, L::tmem, L::tid, L::warp, L::lane, L::logits, L::tile_tops, L::tile_top;
  const Kv8AttnArgs& a;

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    return wait_or_abort(bar, parity, a.wait_budget, &sm.abort);
  }
  // tensor memory columns at + c0 .. (all lanes of the warp)
  __device__ __forceinline__ void load_raw(uint32_t at, float (&v)[CH]) {
    uint32_t t[16];
    tmem_ld16(tmem + at, t);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      asm volatile("" : "+r"(t[k]));             // not before the wait
      v[k] = __uint_as_float(t[k]);
    }
  }

  // false: a wait ran out
  __device__ __forceinline__ bool run(const Share& sh, int RG, int4& rec) {
    Walk w;
    uint32_t i = 0, outs = 0;
    bool ok = true;
    for (bool more = w.first(a, RG, sh); more; more = w.next_segment(a, RG)) {
      const Group& gr = w.gr;
      const bool whole = w.whole();
      if (gr.tiles > 0 && !whole && w.t0 == 0)
        rec = make_int4(gr.r0, gr.g | (w.h << 16), blockIdx.x,
                        (int)min((long long)gridDim.x - 1, blockIdx.x + quotient(gr.tiles - w.left + sh.per - 1, sh.per)));
      if (w.t >= w.t_end) {
        if (gr.tiles > 0) continue;              // the share begins behind the segment's last tile
        if (tid == 0) raise_flag(a.status, CSA_FLAG_ROW_INVALID);
        const int heads = a.heads * a.G;
        uint4* dst = reinterpret_cast<uint4*>(a.out + (size_t)gr.r0 * heads * D);
        for (int k = tid; k < heads * (D / 8); k += kSoftmaxThreads) dst[k] = make_uint4(0u, 0u, 0u, 0u);
        for (int k = tid; k < heads && a.lse; k += kSoftmaxThreads) a.lse[(size_t)gr.r0 * heads + k] = -INFINITY;
        continue;
      }
      const int cols = gr.g * a.G;
      group_sync(1);                             // the segment before has used factors and rows
      convert_queries<COLS, D>(a, sm, gr, w.h);
      fence_proxy_async_smem();
      warp_arrive(&sm.q_full, lane);
      group_sync(1);                             // factors, maxima and rows visible
      float l[COLS];
#pragma unroll
      for (int c = 0; c < COLS; ++c) l[c] = 0.0f;
      float lref = 0.0f;                         // about log2 of the first tile's value scales, a whole number: l is in its units
#pragma unroll 1
      for (; w.t < w.t_end; ++w.t, ++i) {
        const uint32_t st = i % X::kStages, at = (i % X::kScoreBufs) * 2 * COLS;
        ok = wait(&sm.full[st], (i / X::kStages) & 1) && ok;          // complete already: the scales are visible
        // the key, who sees it, and the pages' scales, while S is on its way
        const int page = tid >> 6, base = sm.first_pos[st][page];
        auto scales = [&](int k) {
          return *reinterpret_cast<const float2*>(sm.stage[st] + 128 * D + k * X::kValueSlot + 64 * D);
        };
        if (w.t == w.t0) {
          const float sv[2] = {sm.first_pos[st][0] != INT_MAX ? scales(0).y : 0.0f, sm.first_pos[st][1] != INT_MAX ? scales(1).y : 0.0f};
          lref = sv[1] > 0.0f ? rintf(log2f(sv[1])) : (sv[0] > 0.0f ? rintf(log2f(sv[0])) : 0.0f);
        }
        int clo = COLS;
        float sk = 0.0f, lsv = lref;
        if (base != INT_MAX) {
          const float2 s = scales(page);
          sk = s.x;
          lsv = log2f(s.y);                      // -inf where there are no values: to the sum they count as others do
          clo = max(0, base + (tid & 63) - gr.p0) * a.G;
        }
        // far from the first tile's: infinite, so that y is nothing to the sum and what any column sees moves the maximum
        if (!(fabsf(lsv - lref) <= kKv8Near)) lsv = INFINITY;
        float isv = ex2(lref - lsv);
        const bool masked = __any_sync(0xFFFFFFFFu, clo > 0);
        ok = wait(&sm.s_full[i % X::kScoreBufs], (i / X::kScoreBufs) & 1) && ok;
        tc_fence_after();
        float x[COLS];
        bool moved = w.t == w.t0;                // a segment's first tile goes straight to its maxima
        if (!moved) {
#pragma unroll
          for (int c0 = 0; c0 < COLS; c0 += CH) logits(at, c0, sk, lsv, clo, masked, sm.neg_m, x + c0);
          float top = x[0];
#pragma unroll
          for (int c = 1; c < COLS; ++c) top = fmaxf(top, x[c]);
          moved = top > kTop + kSlack;
        }
        if (group_sync_or(2, moved || !ok)) {
          // O of the tiles before is complete from here on
          ok = wait(&sm.p_free, (i & 1) ^ 1) && ok;
          if (lsv == INFINITY) sm.far = 1;
          if (tid == 0) sm.large = 0;
          if (group_sync_or(2, !ok)) return false;
          tc_fence_after();
          const bool far = sm.far;
          float exact[COLS];
          if (far) {
            float keep[COLS];
#pragma unroll
            for (int c = 0; c < COLS; ++c) keep[c] = l[c];
            const float own = base != INT_MAX ? log2f(scales(page).y) : 0.0f;
            far_tile(sm, tmem, at, sk, own, clo, w.t > w.t0 ? lref : 0.0f, keep, exact);
#pragma unroll
            for (int c = 0; c < COLS; ++c) l[c] = keep[c];
            lref = -INFINITY;
            isv = 0.0f;
            if (tid == 0) sm.far = 0;
          } else {
            tile_tops(at, sk, lsv, clo, masked);
            if (tid < COLS) {
              const float before = sm.neg_m[tid], now = fminf(before, kTop - tile_top());
              sm.corr[tid] = ex2(now - before);
              sm.neg_m[tid] = now;
              if (fabsf(now) > kKv8Large && now < -kNoMax) sm.large = 1;
            }
            group_sync(1);
          }
          if (w.t > w.t0) {
#pragma unroll 1
            for (int c0 = 0; c0 < X::kParts; c0 += 16) {
              uint32_t u[16];
              tmem_ld16(tmem + X::kOut + c0, u);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                asm volatile("" : "+r"(u[k]));
                u[k] = __float_as_uint(__uint_as_float(u[k]) * sm.corr[(c0 + k) % COLS]);
              }
              tmem_st16(tmem + X::kOut + c0, u);
            }
            tmem_st_wait();
          }
#pragma unroll
          for (int c = 0; c < COLS; ++c) l[c] *= far ? 1.0f : sm.corr[c];
          if (!far) {
#pragma unroll
            for (int c0 = 0; c0 < COLS; c0 += CH) logits(at, c0, sk, lsv, clo, masked, sm.neg_m, x + c0);
            if (sm.large) large_logits(sm, tmem, at, sk, lsv, clo, exact);
          }
          if (far || sm.large) {
#pragma unroll
            for (int c = 0; c < COLS; ++c) x[c] = exact[c];
          }
        } else {
          ok = wait(&sm.p_free, (i & 1) ^ 1) && ok;   // one that runs out ends the role at the next tile
        }
        // a warp's two chunks of keys lie in the same banks: their lanes store two columns in opposite order
        const int second = tid & 16;
        const uint32_t order = second ? 0x4401u : 0x4410u;
        uint8_t* p = sm.p + (tid >> 4) * X::kProbChunk + (tid & 15) + second;
        const int other = 16 - 2 * second;
#pragma unroll
        for (int c0 = 0; c0 < COLS; c0 += CH) {
#pragma unroll
          for (int k = 0; k < CH; k += 2) {
            const float y0 = ex2(x[c0 + k]), y1 = ex2(x[c0 + k + 1]);
            l[c0 + k] = fmaf(y0, isv, l[c0 + k]);
            l[c0 + k + 1] = fmaf(y1, isv, l[c0 + k + 1]);
            uint8_t* dst = p + ((c0 + k) >> 3) * X::kProbRows + ((c0 + k) & 7) * 16;
            const uint32_t hi = e4m3x2_of(y0, y1);
            const float2 h = e4m3x2_values(hi);
            const float r0 = y0 - h.x, r1 = y1 - h.y;
            const uint32_t mid = e4m3x2_of(r0 * kMid, r1 * kMid);
            const float2 m = e4m3x2_values(mid);
            const uint32_t lo = e4m3x2_of(fmaf(m.x, -kLo / kMid, r0 * kLo), fmaf(m.y, -kLo / kMid, r1 * kLo));
            const uint32_t codes[3] = {hi, mid, lo};
#pragma unroll
            for (int j = 0; j < 3; ++j) {
              const uint32_t z = __byte_perm(codes[j], 0u, order);
              dst[j * (COLS / 8) * X::kProbRows] = (uint8_t)z;
              dst[j * (COLS / 8) * X::kProbRows + other] = (uint8_t)(z >> 8);
            }
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        warp_arrive(&sm.p_full, lane);
      }
      // ---- the segment's output: sums over the keys' threads, then a dim a thread
      sm.red[warp][lane / (32 / COLS)] = warp_reduce_many<COLS, false>(l, lane);
      ok = wait(&sm.o_full, outs++ & 1) && ok;
      if (group_sync_or(2, !ok)) return false;   // sums visible, too
      tc_fence_after();
      const int slot = w.t0 > 0 ? 2 * (int)blockIdx.x : 2 * (int)blockIdx.x + 1;
      if (tid < COLS) {
        const float sum = (sm.red[0][tid] + sm.red[1][tid]) + (sm.red[2][tid] + sm.red[3][tid]);
        // O counts in 2^-neg_m, l in 2^m
        const bool far = lref == -INFINITY;
        const float m = far ? -sm.neg_l[tid] : -(sm.neg_m[tid] + lref);
        const float up = far ? ex2(-0.5f * sm.neg_m[tid]) : pow2((int)lref);   // by halves: all of it may pass fp32's range
        if (far) sm.neg_l[tid] = up;
        sm.corr[tid] = sum == 0.0f ? 0.0f : up / sum;
        if (whole) {
          if (a.lse && tid < cols) a.lse[sm.out_row[tid]] = sum == 0.0f ? -INFINITY : (log2f(sum) + m) * kLn2;
        } else {
          a.part_ml[((size_t)slot * 2) * COLS + tid] = m;
          a.part_ml[((size_t)slot * 2 + 1) * COLS + tid] = sum;
        }
      }
      group_sync(1);
      if (lref == -INFINITY) scale_out(sm, tmem);
#pragma unroll 1
      for (int c0 = 0; c0 < cols; c0 += CH) {
        float v[CH], mid[CH], lo[CH];
        load_raw(X::kOut + c0, v);
        load_raw(X::kOut + COLS + c0, mid);
        load_raw(X::kOut + 2 * COLS + c0, lo);
#pragma unroll
        for (int k = 0; k < CH; ++k) v[k] = fmaf(lo[k], 1.0f / kLo, fmaf(mid[k], 1.0f / kMid, v[k]));
        if (D == 64 && tid >= 64) continue;      // lanes past the last dim
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          if (c0 + k >= cols) break;
          const float f = sm.corr[c0 + k], o = f == 0.0f ? 0.0f : v[k] * f;
          if (whole) {
            const __nv_bfloat16 z = __float2bfloat16(o);
            a.out[(size_t)sm.out_row[c0 + k] * D + tid] = *reinterpret_cast<const uint16_t*>(&z);
          } else {
            a.part[((size_t)slot * COLS + c0 + k) * D + tid] = o;
          }
        }
        __syncwarp();
      }
      tc_fence_before();
    }
    return true;
  }
};

// CTAs per SM: as many as shared memory holds with two tiles (four of 64 dims) under way in each.
template <int COLS, int D>
constexpr int kPerSm = COLS <= 16 ? 3 : 2;

template <int COLS, int D>
__global__ void __launch_bounds__(kThreads, kPerSm<COLS, D>) k_kv8_attn(Kv8AttnArgs a, int RG) {
  extern __shared__ __align__(128) uint8_t s_raw[];
  using X = Shape<COLS, D>;
  Smem<COLS, D>& sm = *reinterpret_cast<Smem<COLS, D>*>(s_raw);
  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  pdl_trigger();
  if (tid == 0) {
    for (int k = 0; k < X::kStages; ++k) {
      mbar_init(&sm.full[k], 1);
      mbar_init(&sm.free[k], 1);
    }
    for (int k = 0; k < 2; ++k) mbar_init(&sm.s_full[k], 1);
    mbar_init(&sm.p_full, 4);
    mbar_init(&sm.p_free, 1);
    mbar_init(&sm.q_full, 4);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.drain, 1);
    sm.abort = sm.far = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&sm.tmem_base, X::kTmem);
  const Share sh = find_share<kThreads>(a, RG, sm.share);  // its barriers make the above visible
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  if (warp == kCopyWarp) {
    copy_pages<COLS, D>(a, sm, sh, RG);
  } else if (warp == kMmaWarp) {
    Products<COLS, D>{a, sm, tmem, false}.run(sh, RG);
  } else {
    int4 rec = make_int4(-1, 0, 0, 0);
    Softmax<COLS, D> role{{sm, tmem + ((uint32_t)(32 * warp) << 16), tid, warp, lane}, a};
    (void)role.run(sh, RG, rec);
    if (tid == 0) a.rec[blockIdx.x] = rec;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && sm.abort) raise_flag(a.status, CSA_FLAG_TIMEOUT);
  if (warp == kMmaWarp) tmem_dealloc(tmem, X::kTmem);
}

// ---- cut segments -----------------------------------------------------------------------------
// A row of CTAs a cut, W warps a column; a warp sums its parts' O / l by their weights l 2^m, in the
// parts' order.  A part's weight can be 2^-228 of another's and still bring most of the output, by its values (their
// scales span as much); where weights are that far apart they are applied as two factors.  Taken with l in [1, 2),
// the largest weight is 2^-11 of that: with fewer than 2^10 parts no sum leaves fp32's range at either end.
// Bound by latency: statistics and a warp's first 8 parts are asked for at once, some 3 us for the 33 parts
// of one token after 4096.  CTAs of 512 threads, with 64 registers each, took 0.5 us more, and 4 for 64 rows' lists.
constexpr int kMergeThreads = 256, kMergePerSm = 3;
constexpr float kPartUnit = 1.0f / 2048.0f, kDeep = -64.0f;
// A part's slot: 2 c0 + 1 of the first, then 2 (c0 + 1), 2 (c0 + 2), ...
__device__ __forceinline__ size_t part_slot(int first, int q) { return (size_t)(q == 0 ? 2 * first + 1 : 2 * (first + q)); }

template <int D>
__device__ __forceinline__ void write_column(uint16_t* out, float* lse, const float (&acc)[D / 32], float M, float L) {
  constexpr int N = D / 32;
  const int lane = lane_id();
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  uint32_t o[N / 2];
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const __nv_bfloat162 z = __floats2bfloat162_rn(inv == 0.0f ? 0.0f : acc[j] * inv, inv == 0.0f ? 0.0f : acc[j + 1] * inv);
    o[j / 2] = *reinterpret_cast<const uint32_t*>(&z);
  }
  uint16_t* dst = out + N * lane;
  if constexpr (N == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
  else *reinterpret_cast<uint32_t*>(dst) = o[0];
  if (lse && lane == 0) *lse = L == 0.0f ? -INFINITY : (M + log2f(L * (1.0f / kPartUnit))) * kLn2;
}
// (m, l) of a part, l as a number in [1, 2) whose power of two m takes up; 0, infinities and NaN as they are, or twice over.
__device__ __forceinline__ float2 part_stats(const float* part_ml, int cols_max, int c, int first, int q) {
  const float* ml = part_ml + part_slot(first, q) * 2 * cols_max + c;
  const float m = __ldcg(ml), l = __ldcg(ml + cols_max);
  const int e = l > 0.0f ? min(126, (int)(__float_as_uint(l) >> 23) - 127) : 0;
  return make_float2(m + (float)e, l * pow2(-e));
}
// A column whose parts' weights are far apart, by one warp.  Seldom called, and kept out of the way.
template <int D>
__device__ __noinline__ void deep_column(const float* part, const float* part_ml, int cols_max, int c, int first, int n,
                                         uint16_t* out, float* lse) {
  constexpr int N = D / 32;
  float M = kNoMax, L = 0.0f, acc[N];
#pragma unroll 1
  for (int q = 0; q < n; ++q) M = fmaxf(M, part_stats(part_ml, cols_max, c, first, q).x);
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.0f;
#pragma unroll 1
  for (int q = 0; q < n; ++q) {
    const float2 ml = part_stats(part_ml, cols_max, c, first, q);
    const float d = ml.x - M, f = ex2(d < kDeep ? 0.5f * d : d), g = d < kDeep ? f : 1.0f;
    const float w = f * ml.y * kPartUnit;
    L = fmaf(w, g, L);
    const float* v = part + (part_slot(first, q) * cols_max + c) * D + N * lane_id();
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = fmaf(w, __ldcg(v + j) * g, acc[j]);
  }
  write_column<D>(out, lse, acc, M, L);
}

template <int D>
__global__ void __launch_bounds__(kMergeThreads, kMergePerSm) k_kv8_merge(Kv8AttnArgs a, int cols_max) {
  constexpr int N = D / 32, kWarps = kMergeThreads / 32;
  __shared__ float s_o[kWarps][D];
  const int warp = warp_id(), lane = lane_id();
  pdl_wait();
  const int4 rec = __ldcg(a.rec + blockIdx.x);
  if (rec.x < 0) return;
  const int g = rec.y & 0xFFFF, h = rec.y >> 16, G = a.G, cols = g * G, n = rec.w - rec.z + 1;
  int W = 1;
  while (2 * W * cols <= kWarps) W *= 2;
  auto slot = [&](int q) { return part_slot(rec.z, q); };
  for (int c0 = blockIdx.y * (kWarps / W); c0 < cols; c0 += gridDim.y * (kWarps / W)) {
    const int c = c0 + warp / W, sub = warp % W;
    float M = kNoMax, L = 0.0f, acc[N];
    float least = INFINITY;                      // of the lane's parts' m
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.0f;
    if (c < cols) {
      // 32 parts at a time, a lane has one's (m, l); O / l of up to 8 of the warp's are asked for with them
#pragma unroll 1
      for (int base = 0; base < n; base += 32) {
        const int q = base + lane, end = min(32, n - base);
        float m = kNoMax, l = 0.0f;
        if (q < n) {
          const float2 ml = part_stats(a.part_ml, cols_max, c, rec.z, q);
          m = ml.x;
          l = ml.y;
        }
        float wgt = 0.0f;
#pragma unroll 1
        for (int k0 = sub; k0 < end || k0 == sub; k0 += 8 * W) {
          float v[8][N];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int k = min(k0 + i * W, end - 1);
            const float* src = a.part + (slot(base + k) * cols_max + c) * D + N * lane;
            if constexpr (N == 4) *reinterpret_cast<float4*>(v[i]) = __ldcg(reinterpret_cast<const float4*>(src));
            else *reinterpret_cast<float2*>(v[i]) = __ldcg(reinterpret_cast<const float2*>(src));
          }
          if (k0 == sub) {
            const float now = fmaxf(M, warp_top(m));
            const float corr = ex2(M - now);
            least = fminf(least, l == 0.0f ? INFINITY : m);
            M = now;
            wgt = ex2(m - now) * l * kPartUnit;
            L = fmaf(L, corr, wgt);
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] *= corr;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int k = k0 + i * W;
            const float wk = __shfl_sync(0xFFFFFFFFu, wgt, k & 31);
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = k < end ? fmaf(wk, v[i][j], acc[j]) : acc[j];
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
    }
    if (W > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < N; ++j) s_o[warp][N * lane + j] = acc[j];
      __syncthreads();
      if (sub == 0)
        for (int k = 1; k < W; ++k)
#pragma unroll
          for (int j = 0; j < N; ++j) acc[j] += s_o[warp + k][N * lane + j];
    }
    if (sub == 0 && c < cols) {
      const int i = c / G;
      const size_t row = (size_t)(rec.x + i) * a.heads * G + h * G + (c - i * G);
      uint16_t* out = a.out + row * D;
      float* lse = a.lse ? a.lse + row : nullptr;
      if (__any_sync(0xFFFFFFFFu, least - M < kDeep)) deep_column<D>(a.part, a.part_ml, cols_max, c, rec.z, n, out, lse);
      else write_column<D>(out, lse, acc, M, L);
    }
  }
}

// ---- launch ---------------------------------------------------------------------------------------
constexpr int kMaxPerSm = 3;
constexpr int kGap = 1;                          // units of work of a step between segments

// Columns that a group has here; 0: more than the kernel takes.  The fewest that hold the group's:
// 32 requests at 4k to 6k tokens, 4 key heads of 64, take 28 us with 7 columns in 8 and 34 in 16, 36 us
// with 14 in 16 and 50 in 32, 56 us with 28 in 32 and 66 in a wide group (8 key heads of 128, 32 columns:
// 103 and 148).  Two groups of 21 columns in 32 took 92 us where a wide one of 42 took 85, 69 by now.
int group_cols(int64_t wanted) { return wanted <= 8 ? 8 : (wanted <= 16 ? 16 : (wanted <= 32 ? 32 : 0)); }

template <int COLS, int D>
cudaError_t launch_cols(Kv8AttnArgs a, int RG, uint8_t* ws, int num_sms, cudaStream_t stream) {
  static_assert(kPerSm<COLS, D> <= kMaxPerSm && kPerSm<COLS, D> * Shape<COLS, D>::kTmem <= 512, "tensor memory");
  static_assert(kPerSm<COLS, D> * (sizeof(Smem<COLS, D>) + 1024) <= 233472, "shared memory");
  const int64_t pages = kv8_pages(a.rows.max_entries);
  const int grid = kv8_grid(a.rows.num_rows, a.heads, a.blocks ? std::min<int64_t>(pages, a.n_blocks) : pages,
                            num_sms * kPerSm<COLS, D>);
  kv8_place_parts(a, ws, grid, COLS);
  a.gap = kGap;
  constexpr int smem = (int)sizeof(Smem<COLS, D>);
  cudaError_t e = cudaFuncSetAttribute(k_kv8_attn<COLS, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_kernel(Order::kStream, k_kv8_attn<COLS, D>, dim3(grid), dim3(kThreads), smem, stream, a, RG);
  if (e != cudaSuccess || grid == 1) return e;
  return launch_kv8_merge(a, COLS, grid, stream);
}

template <int D>
cudaError_t launch_dim(const Kv8AttnArgs& a, uint8_t* ws, int num_sms, cudaStream_t stream) {
  const int64_t per = a.blocks ? 1 : std::min(a.rows.num_rows, a.rows.max_rows_per_req);
  const int cols = group_cols(a.G * per), RG = a.blocks ? 1 : cols / a.G;
  switch (cols) {
    case 8: return launch_cols<8, D>(a, RG, ws, num_sms, stream);
    case 16: return launch_cols<16, D>(a, RG, ws, num_sms, stream);
    case 32: return launch_cols<32, D>(a, RG, ws, num_sms, stream);
    default: return launch_kv8_wide(a, ws, num_sms, stream);
  }
}

}  // namespace

cudaError_t launch_kv8_merge(const Kv8AttnArgs& a, int cols, int grid, cudaStream_t stream) {
  if (a.dim == 64)
    return launch_kernel(Order::kChained, k_kv8_merge<64>, dim3(grid - 1, std::min((cols + 7) / 8, 16)), dim3(kMergeThreads), 0, stream, a, cols);
  return launch_kernel(Order::kChained, k_kv8_merge<128>, dim3(grid - 1, std::min((cols + 7) / 8, 16)), dim3(kMergeThreads), 0, stream, a, cols);
}

// For any split of the heads into groups and any number of pages up to max_entries'.
size_t kv8_attn_ws_bytes(int32_t num_rows, int32_t max_entries, int32_t n_heads, int num_sms) {
  const int64_t pages = kv8_pages(max_entries), most = (int64_t)num_rows * n_heads;
  const int cols = group_cols(most) ? group_cols(most) : 32;
  const size_t narrow = kv8_parts_bytes(kv8_grid(num_rows, n_heads, pages, num_sms * kMaxPerSm), cols, 128);
  if (most <= 32) return narrow;
  return std::max(narrow, kv8_parts_bytes(kv8_wide_grid(num_rows, n_heads, max_entries, num_sms), kKv8WideCols, 128));
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs& a, void* ws, int num_sms, cudaStream_t stream) {
  return a.dim == 64 ? launch_dim<64>(a, static_cast<uint8_t*>(ws), num_sms, stream)
                     : launch_dim<128>(a, static_cast<uint8_t*>(ws), num_sms, stream);
}

}  // namespace csa
