// csa_kv8_attn where a group has many columns (prompt chunks, verify rows of wide groups): two
// tiles of 128 columns share each tile of keys and values.
//
// Mathematics as in kv8_attn.cu with columns on the lanes: S = Q K^T (M = 128 columns, N = 128
// keys) in E4M3, Q's two parts one product after another into the same sums (the second part in
// the first one's units: exact down to 2^-9 of the query's largest element, below that to 2^-17
// of it); y = 2^(s + log2 sv - m) rounded once to fp16, at most 2^15 and at least 2^8 at the
// column's largest; O += y V in fp16, V converted from E4M3 (exact).  Two threads have a column, one
// with the keys of each page of a tile: their maximum, sum and correction need no other exchange.  Once a
// segment's value scales are far apart, or 0, the sum has a maximum and powers of two of its own there, too; such
// a tile's scales are infinite to the loop, so that it takes the way of a maximum that moves.
//
// Pipeline, one CTA per SM: 2 x 8 softmax warps (the halves' columns, a page of each tile each; two
// warps that share columns meet once a tile, to agree whether the maximum moves), 4 warps that
// convert values, one warp that copies keys, one that copies values, one that forms the tiles' scales,
// one that issues the products.  y takes the place of the S it came from in tensor memory and is the
// second product's A operand there.  Products alternate, O_a += y_a V of tile t, S_a of t + 1,
// then the same for b, so that the tensor core works for one half while the other half's softmax
// runs.  A segment of up to 128 columns has one tile of them: half b then takes every second tile
// of keys, with a maximum, sum and O of its own, which half a joins with its own at the end (both
// halves' lanes are the same columns, so a reads b's O in tensor memory as it is).
//
// What bounds it.  A tile of 128 keys and 2 x 128 columns of 128 dims is 32 MMAs of 65 clocks, 2080.
// Four prompts of 512 rows, 32 heads over 8, after 8k to 16k tokens take 310 us for 392 GFLOP, 1.26 PFLOP/s
// or 0.64 of the measured bf16 rate, where the queries' second part is work on top; the tensor pipe is
// active for 54 %, issue slots 53 %.  A tile takes some 2700 clocks, and shared memory's port is what it
// waits for: the products read 8 KB an MMA for S and 4 KB for O, 192 KB a tile, the conversion of the values
// moves 48 KB and the copies 32 KB, 2125 clocks at 128 bytes.  (Without any power of two, for a
// measurement, prompts took 302 us instead of 303.)  A step between segments takes 20 thousand, a share's search 10 thousand.  32
// requests of 6 rows and 7 queries a key head, 42 columns of 64 dims, take 53 us: half of the
// warps have columns that no query has.
// Eight softmax warps, a thread a column, took 330 and 69 us; two issuing warps were slower, as were one that
// sleeps at its barriers (366 against 347 us then) and one loop for both kinds of segments (326 against
// 314); of 768 threads each has 80 registers, and a split of 96 and 48 was no better (343 against 326), nor
// a quarter of the powers of two as polynomials (321 against 303).
#include <algorithm>

#include "kv8_list.cuh"

namespace csa {

namespace {

constexpr int kThreads = 768, kHalf = 128;
constexpr int kConvertWarp = 16, kKeyWarp = 20, kValueWarp = 21, kMmaWarp = 22, kScaleWarp = 23;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// y is 2^kTop at the running maximum, which moves when a page's y add up to more than kMost:
// none is above 2^15.
constexpr float kTop = 8.0f, kMost = 32768.0f;
constexpr float kNoMax = -3e38f;                 // running maximum of a column that has seen nothing
// Units of work of a step between segments: queries, outputs and the way to the first logits take the time of
// about 6 tiles (counted as 2, prompts of 4 x 512 rows took 337 us instead of 330).
constexpr int kGap = 6;

template <int D>
struct Shape {
  static constexpr int kKeyStages = 3, kValueStages = 2;
  // Tiles' scales.  Tile i's keys come when S of tile i - kKeyStages is complete, and that was issued after
  // y of the second tile before it, at the latest, had been formed.
  static constexpr int kTiles = kKeyStages + 3;
  static constexpr uint32_t kScores = 0, kOut = 256;          // tensor memory columns: S of both halves, then O
  static constexpr uint32_t kTmem = 512;
};
// What the softmax needs of a tile besides S.
struct Tile {
  float sk[2], lsv[2], isv[2];                   // key scale, log2 of the value scale, 2^lref over it
  float own[2];                                  // log2 of the value scale where lsv is infinite: far from the segment's first
  float lref;                                    // units of the segment's sums
  int first[2];                                  // position of a page's first slot; INT_MAX: no page
};
template <int D>
struct Smem {
  using X = Shape<D>;
  uint8_t q[2][2][kHalf * D];                    // [half][part]
  uint8_t k[X::kKeyStages][128 * D];
  uint8_t raw[X::kValueStages][128 * D];
  uint8_t v[2][256 * D];                         // fp16: 8 dims: 16 pieces of 8 keys
  float factor[2][kHalf];                        // of a column's logits (log2 units)
  float4 scales[X::kKeyStages][2];               // a page's key and value scales, as they lie behind its record
  Tile tile[X::kTiles];
  int k_first[X::kKeyStages][2], raw_first[X::kValueStages][2];
  uint64_t tile_full[X::kTiles];
  uint64_t k_full[X::kKeyStages], k_free[X::kKeyStages];
  uint64_t raw_full[X::kValueStages], raw_free[X::kValueStages];
  uint64_t v_full[2], v_free[2];
  uint64_t q_full[2], s_full[2], p_full[2], pv_done[2], drain;
  float2 joined[2][kHalf];                       // half b's -maximum and its pages' sums of a shared tile of columns
  float pair[2][2][kHalf];                       // [half][page]: what the two threads of a column tell one another
  // sums with a maximum of their own: a page's, minus the column's (NaN: not so), and what O counts from beside that
  float own_top[2][2][kHalf], own_neg[2][2][kHalf], own_rel[2][2][kHalf];
  uint64_t b_full, b_free;                       // these and half b's O: complete, read
  uint32_t tmem_base;
  volatile int abort;                            // a wait ran out: every role leaves
  ShareScratch<kThreads> share;
};

__device__ __forceinline__ uint32_t f16x2_of(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void group_pair_sync(int id) { asm volatile("barrier.cta.sync.aligned %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// ---- copies ------------------------------------------------------------------------------------
// One warp for each side: kKeys copies keys and the pages' scales, the other values.
template <int D, bool kKeys>
__device__ __forceinline__ void copy_side(const Kv8AttnArgs& a, Smem<D>& sm, const Share& sh, int RG) {
  using X = Shape<D>;
  constexpr int kStages = kKeys ? X::kKeyStages : X::kValueStages, kBytes = 64 * D;
  uint64_t* full = kKeys ? sm.k_full : sm.raw_full;
  uint64_t* free = kKeys ? sm.k_free : sm.raw_free;
  const int lane = lane_id();
  Walk w;
  uint32_t i = 0;
  bool ok = true;
  for (bool more = w.first(a, RG, sh); more && ok; more = w.next_segment(a, RG)) {
    if (w.t >= w.t_end) continue;
    int chunk = (w.t >> 4) - 1, above = -1;
    bool ended = false;
    Pages x{INT_MAX, -1}, next = pages_of<false>(a, w.gr, w.h, chunk + 1, above, ended);
    for (; w.t < w.t_end; ++w.t, ++i) {
      if (w.t >> 4 != chunk) {
        chunk = w.t >> 4;
        x = next;
        if (32 * (chunk + 1) < 2 * w.t_end) next = pages_of<false>(a, w.gr, w.h, chunk + 1, above, ended);
      }
      const uint32_t st = i % kStages;
      ok = __all_sync(0xFFFFFFFFu, wait_or_abort(&free[st], ((i / kStages) & 1) ^ 1, a.wait_budget, &sm.abort));
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
          (kKeys ? sm.k_first : sm.raw_first)[st][k] = j[k] == INT_MAX ? INT_MAX : j[k] * PAGE;
          if (j[k] != INT_MAX) bytes += kBytes + (kKeys ? 16 : 0);
        }
        mbar_expect_tx(&full[st], bytes);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (j[k] == INT_MAX) continue;
          const uint8_t* rec = a.pool + kv8_record<D>(page[k], a.heads, w.h);
          bulk_load((kKeys ? sm.k[st] : sm.raw[st]) + k * kBytes, kKeys ? rec : rec + kBytes, kBytes, &full[st]);
          if (kKeys) bulk_load(&sm.scales[st][k], rec + 2 * kBytes, 16, &full[st]);
        }
      }
      __syncwarp();
    }
  }
  // after a wait that ran out: what is still being copied must land before the CTA ends
  if (lane == 0)
    for (uint32_t k = i > kStages ? i - kStages : 0; k < i; ++k) (void)mbar_wait(&full[k % kStages], (k / kStages) & 1);
}

// ---- scales and values ------------------------------------------------------------------------------
// One warp: the tiles' scales as the softmax takes them, a lane each page's.
template <int D>
__device__ __forceinline__ void prepare_scales(const Kv8AttnArgs& a, Smem<D>& sm, const Share& sh, int RG) {
  using X = Shape<D>;
  const int lane = lane_id(), k = lane & 1;
  Walk w;
  uint32_t i = 0;
  float lref = 0.0f;
  bool far = false;
  for (bool more = w.first(a, RG, sh); more && w.settle(a, RG); ++i, ++w.t) {
    const uint32_t st = i % X::kKeyStages;
    if (!__all_sync(0xFFFFFFFFu, wait_or_abort(&sm.k_full[st], (i / X::kKeyStages) & 1, a.wait_budget, &sm.abort))) return;
    const float4 s = sm.scales[st][k];
    const int first = sm.k_first[st][k];
    const bool there = first != INT_MAX;
    const float own = log2f(there ? s.y : 1.0f);   // -inf where there are no values: to the sum they count as others do
    if (w.t == w.t0) {
      const uint32_t some = __ballot_sync(0xFFFFFFFFu, there && s.y > 0.0f);
      const float of0 = __shfl_sync(0xFFFFFFFFu, own, 0), of1 = __shfl_sync(0xFFFFFFFFu, own, 1);
      lref = rintf((some & 2u) ? of1 : ((some & 1u) ? of0 : 0.0f));
      far = false;
    }
    const float lsv = there ? own : lref;
    far = far || __any_sync(0xFFFFFFFFu, !(fabsf(lsv - lref) <= kKv8Near));
    Tile& t = sm.tile[i % X::kTiles];
    if (lane < 2) {
      t.sk[k] = first != INT_MAX ? s.x : 0.0f;
      t.lsv[k] = far ? INFINITY : lsv;
      t.isv[k] = far ? 0.0f : ex2(lref - lsv);
      t.own[k] = lsv;
      t.first[k] = first;
      t.lref = lref;
    }
    warp_arrive(&sm.tile_full[i % X::kTiles], lane);
    warp_arrive(&sm.k_free[st], lane);
  }
}

// Values to fp16, by four warps.  Pages' values are transposed already: 16 keys of a dim are two
// neighbouring pieces of 8.  A page that is not there becomes zeros, its place may hold anything.
template <int D>
__device__ __forceinline__ void convert_values(const Kv8AttnArgs& a, Smem<D>& sm, const Share& sh, int RG) {
  using X = Shape<D>;
  constexpr int N = D / 16;                      // a warp's pieces: 8 dims of a page
  const int lane = lane_id(), warp = warp_id() - kConvertWarp, k = warp & 1;
  Walk w;
  uint32_t i = 0;
  for (bool more = w.first(a, RG, sh); more && w.settle(a, RG); ++i, ++w.t) {
    const uint32_t st = i % X::kValueStages, vb = i & 1;
    bool ok = wait_or_abort(&sm.raw_full[st], (i / X::kValueStages) & 1, a.wait_budget, &sm.abort);
    if (!__all_sync(0xFFFFFFFFu, ok)) return;
    const bool there = sm.raw_first[st][k] != INT_MAX;
    ok = wait_or_abort(&sm.v_free[vb], ((i >> 1) & 1) ^ 1, a.wait_budget, &sm.abort);
    if (!__all_sync(0xFFFFFFFFu, ok)) return;
    // lane: dim lane % 8, 16 keys lane / 8
    uint8_t* dst = sm.v[vb] + (warp >> 1) * 2048 + (k * 8 + (lane >> 3) * 2) * 128 + (lane & 7) * 16;
#pragma unroll 2
    for (int j = 0; j < N; ++j) {
      uint32_t o[8];
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (there) x = *reinterpret_cast<const uint4*>(sm.raw[st] + k * 64 * D + (2 * j + (warp >> 1)) * 512 + lane * 16);
      const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t f[2];
        e4m3x4_to_f16(in[e], f);
        o[2 * e] = f[0];
        o[2 * e + 1] = f[1];
      }
      *reinterpret_cast<uint4*>(dst + j * 4096) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(dst + j * 4096 + 128) = make_uint4(o[4], o[5], o[6], o[7]);
    }
    fence_proxy_async_smem();
    warp_arrive(&sm.v_full[vb], lane);
    warp_arrive(&sm.raw_free[st], lane);
  }
}

// ---- products ------------------------------------------------------------------------------------
// The whole warp walks and waits, every operand's address is a constant or uniform, and one
// elected lane issues: with addresses formed in a lane of its own an MMA took 108 clocks to
// issue instead of the 65 that it runs.  The CTA holds all of the tensor memory, from column 0.
template <int D>
struct Products {
  using X = Shape<D>;
  const Kv8AttnArgs& a;
  Smem<D>& sm;
  uint32_t used = 0;                             // bit x: parity of half x's tiles so far

  // Up to three barriers at once, each polled by lanes of its own: one after another they took 150 clocks each.
  struct On {
    uint64_t* bar;
    uint32_t parity;
  };
  __device__ __forceinline__ bool wait(On p, On q, On r) {
    const int k = lane_id() % 3;
    uint64_t* bar = k == 0 ? p.bar : (k == 1 ? q.bar : r.bar);
    const uint32_t parity = k == 0 ? p.parity : (k == 1 ? q.parity : r.parity);
    return __all_sync(0xFFFFFFFFu, wait_or_abort<true>(bar, parity, a.wait_budget, &sm.abort));
  }
  __device__ __forceinline__ On keys(uint32_t i) { return On{&sm.k_full[i % X::kKeyStages], (i / X::kKeyStages) & 1}; }
  __device__ __forceinline__ On converted(uint32_t i) { return On{&sm.v_full[i & 1], (i >> 1) & 1}; }
  __device__ __forceinline__ On formed(int x) { return On{&sm.p_full[x], (used >> x) & 1}; }
  // S of half x and tile i, with the queries of half qx; the last half to use the keys gives them back
  __device__ __forceinline__ void scores(int x, int qx, uint32_t i, bool last_half) {
    constexpr uint32_t idesc = idesc_e4m3(128, 128);
    tc_fence_after();
    const uint64_t k = smem_desc(smem_u32(sm.k[0]), 128, 8 * D, kSwizzleNone) + (i % X::kKeyStages) * (8 * D);
    const uint64_t q = smem_desc(smem_u32(sm.q[0][0]), 128, 8 * D, kSwizzleNone) + qx * (kHalf * D / 8);
    if (elect_one()) {
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
          mma_f8(X::kScores + 128 * x, q + part * (kHalf * D / 16) + 16 * s, k + 16 * s, idesc, part + s > 0);
      tc_commit(&sm.s_full[x]);
      if (last_half) tc_commit(&sm.k_free[i % X::kKeyStages]);
    }
    __syncwarp();
  }
  // O of half x += y V of tile j
  __device__ __forceinline__ void values(int x, uint32_t j, bool first, bool last_half) {
    used ^= 1u << x;
    tc_fence_after();
    const uint64_t v = smem_desc(smem_u32(sm.v[0]), 128, 2048, kSwizzleNone) + (j & 1) * (16 * D);
    if (elect_one()) {
#pragma unroll
      for (int s = 0; s < 8; ++s)
        mma_f16_ts(X::kOut + 128 * x, X::kScores + 128 * x + 64 * (s >> 2) + 8 * (s & 3), v + 16 * s,
                   idesc_f16(128, D, 0, 0), s > 0 ? 1u : (uint32_t)!first);
      tc_commit(&sm.pv_done[x]);
      if (last_half) tc_commit(&sm.v_free[j & 1]);
    }
    __syncwarp();
  }
  // A loop for each kind of segment, as short as can be: what it holds is fetched anew each time round.
  __device__ __forceinline__ void run(const Share& sh, int RG) {
    Walk w;
    uint32_t i0 = 0, segs = 0, wides = 0;        // tiles, segments and those of two tiles of columns before this one
    bool ok = true;
    for (bool more = w.first(a, RG, sh); more && ok; more = ok && w.next_segment(a, RG)) {
      const int tiles = w.t_end - w.t;
      if (tiles <= 0) continue;
      const bool joint = w.gr.g * a.G <= kHalf;
      const On q0{&sm.q_full[0], segs & 1}, q1{&sm.q_full[1], wides & 1};
      if (joint) {                               // the halves in turn, a tile each
#pragma unroll 1
        for (int s = 0; s < tiles + 2; ++s) {
          const int x = s & 1;
          const uint32_t i = i0 + s;
          const bool next = s < tiles, before = s >= 2;
          if (!next && !before) continue;
          const On v = converted(i - 2), k = next ? keys(i) : v;
          if (!(ok = before ? wait(k, v, formed(x)) : wait(k, q0, k))) break;
          if (before) values(x, i - 2, s < 4, true);
          if (next) scores(x, 0, i, true);
        }
      } else {                                   // both halves, each tile
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
          const uint32_t i = i0 + t;
          const On k = keys(i);
          if (!(ok = t == 0 ? wait(k, q0, k) : wait(k, converted(i - 1), formed(0)))) break;
          if (t > 0) values(0, i - 1, t == 1, false);
          scores(0, 0, i, false);
          const On y = t == 0 ? q1 : formed(1);
          if (!(ok = wait(y, y, y))) break;
          if (t > 0) values(1, i - 1, t == 1, true);
          scores(1, 1, i, true);
        }
        for (int x = 0; x < 2 && ok; ++x) {
          const On v = converted(i0 + tiles - 1);
          if ((ok = wait(v, formed(x), v))) values(x, i0 + tiles - 1, tiles == 1, x > 0);
        }
      }
      i0 += tiles;
      ++segs;
      if (!joint) ++wides;
    }
    // everything issued is complete before the tensor memory is given back
    if (lane_id() == 0) {
      tc_commit(&sm.drain);
      (void)mbar_wait(&sm.drain, 0);
    }
    __syncwarp();
  }
};

// ---- queries ---------------------------------------------------------------------------------------
// A warp's own 32 columns to E4M3 parts.  Eight columns' pieces of 8 dims are copied at a time, each to
// where its dims' codes will be (16 dims have 32 bytes, and 16 of codes in either part); then a lane has a
// column, and the rest needs no other lane.  With 16 lanes a column, and shuffles for its maximum, a segment's
// queries took 15 thousand clocks.  A negative softmax scale turns the query round, so that a column's
// largest S is its largest logit.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool there) {            // zeros if not
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
// Two E4M3 codes of two fp16, low half first.
__device__ __forceinline__ uint32_t e4m3x2_of_f16(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}
template <int D>
__device__ __forceinline__ void convert_queries(const Kv8AttnArgs& a, Smem<D>& sm, const Group& gr, int h, int x) {
  const int lane = lane_id(), G = a.G, c0 = 32 * (warp_id() & 3), c = c0 + lane;
  const int over = (65536 + G - 1) / G;          // col / G is (col * over) >> 16 for columns below 256
  auto place = [&](int col, int piece) -> uint4* {
    return reinterpret_cast<uint4*>(sm.q[x][piece & 1] + (col >> 3) * 8 * D + (piece >> 1) * 128 + (col & 7) * 16);
  };
#pragma unroll 1
  for (int k = 0; k < 32; k += 8) {
    const int col = c0 + k + (lane & 7), at = kHalf * x + col, i = (at * over) >> 16;
    const bool there = i < gr.g;
    const uint16_t* src = there ? a.q + ((size_t)(gr.r0 + i) * a.heads * G + h * G + (at - i * G)) * D + 8 * (lane >> 3) : a.q;
#pragma unroll
    for (int p = 0; p < D / 8; p += 4) cp_async16(place(col, p + (lane >> 3)), there ? src + 8 * p : a.q, there);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  const Kv8Rope& rope = a.rows.rope;
  const int row = ((kHalf * x + c) * over) >> 16;
  if (rope.cos != nullptr && row < gr.g) {
    const int first = rope.first >> 3, half = rope.dims >> 4;
#pragma unroll 1
    for (int p = 0; p < half; ++p) {
      const uint4 low = *place(c, first + p), high = *place(c, first + half + p);
      *place(c, first + p) = turn8(low, high, rope, Kv8Turn{0, 8 * p, true}, gr.p0 + row);
      *place(c, first + half + p) = turn8(high, low, rope, Kv8Turn{0, 8 * p, false}, gr.p0 + row);
    }
  }
  auto two = [](uint32_t w) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)); };
  __nv_bfloat162 m = two(0u);
#pragma unroll 4
  for (int p = 0; p < D / 8; ++p) {
    const uint4 v = *place(c, p);
    m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(two(v.x), two(v.y)), __hmax2_nan(two(v.z), two(v.w))));
  }
  const float big = __low2float(__hmax2_nan(m, __lowhigh2highlow(m)));
  // 2^-e puts the largest magnitude in [128, 256); e >= -126 keeps it in fp32's range, and a
  // query of such small elements has no logit to speak of
  const int ex = (int)(__float_as_uint(big) >> 23);
  const int e = (ex > 0 && ex < 255) ? max(ex - 127 - 7, -126) : 0;
  const float f = a.softmax_scale < 0.0f ? -pow2(-e) : pow2(-e);
  // fp16 holds an element so scaled exactly down to 2^-16, and E4M3's steps end at 2^-9
#pragma unroll 1
  for (int s = 0; s < D / 16; ++s) {
    const uint4 v[2] = {*place(c, 2 * s), *place(c, 2 * s + 1)};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t w = k & 4 ? ((k & 2) ? (k & 1 ? v[1].w : v[1].z) : (k & 1 ? v[1].y : v[1].x))
                               : ((k & 2) ? (k & 1 ? v[0].w : v[0].z) : (k & 1 ? v[0].y : v[0].x));
      const uint32_t y = f16x2_of(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
      const uint32_t code = e4m3x2_of_f16(y), back = e4m3x2_to_f16((uint16_t)code);
      const __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&y), *reinterpret_cast<const __half2*>(&back));
      const uint32_t left = e4m3x2_of_f16(*reinterpret_cast<const uint32_t*>(&rest));
      hi[k >> 1] = (k & 1) ? hi[k >> 1] | (code << 16) : code;
      lo[k >> 1] = (k & 1) ? lo[k >> 1] | (left << 16) : left;
    }
    *place(c, 2 * s) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *place(c, 2 * s + 1) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  // NaN where an element is infinite or not a number
  sm.factor[x][c] = fmaf(big, 0.0f, fabsf(a.softmax_scale) * kLog2e * pow2(e));
}

// ---- softmax ---------------------------------------------------------------------------------------
// A tile of a column's page where sums have a maximum of their own: l, and the factor of O.  y goes over the S that it came
// from.  l counts from own_neg, minus the largest s, and O from own_neg + own_rel: a difference of two large numbers would
// say nothing of value scales.  In the first such tile l counts from neg + lref and O from neg.  The two warps that share
// the columns meet twice.  Seldom called, and kept out of the loop that calls it.
template <int D>
__device__ __noinline__ float2 far_tile(Smem<D>& sm, uint32_t scores, int x, int p, int c, int seen, float fs, float lsv, float neg,
                                        float lref, float l) {
  float a = sm.own_neg[x][p][c], rel = sm.own_rel[x][p][c];
  if (a != a) {
    a = neg + lref;
    rel = neg < -kNoMax ? -lref : neg;           // that of a column that has seen nothing stays so
  }
  float now = 0.0f, top = -INFINITY, most = -INFINITY, sum = 0.0f;
  auto pass = [&](auto each) {
#pragma unroll 1
    for (int k0 = 0; k0 < 64; k0 += 32) {
      uint32_t u[32];
      tmem_ld32(scores + k0, u);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        asm volatile("" : "+r"(u[k]));           // not before the wait
        const float z = __fmul_rn(__uint_as_float(u[k]), fs) + now;
        u[k] = __float_as_uint(k0 + k < seen ? z : -INFINITY);
      }
      each(k0, u);
    }
  };
  pass([&](int, const uint32_t (&u)[32]) {
#pragma unroll
    for (int k = 0; k < 32; ++k) top = fmaxf(top, __uint_as_float(u[k]));
  });
  sm.own_top[x][p][c] = top;
  group_pair_sync(1 + 4 * x + (c >> 5));
  now = fminf(a, -fmaxf(sm.own_top[x][0][c], sm.own_top[x][1][c]));
  pass([&](int, const uint32_t (&u)[32]) {
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      sum += ex2(__uint_as_float(u[k]));
      most = fmaxf(most, __uint_as_float(u[k]) + lsv);
    }
  });
  sm.pair[x][p][c] = most;
  group_pair_sync(1 + 4 * x + (c >> 5));
  most = fmaxf(sm.pair[x][0][c], sm.pair[x][1][c]);
  const float shift = now - a, next = fminf(rel < -kNoMax ? rel - shift : rel, kTop - most);
  pass([&](int k0, const uint32_t (&u)[32]) {
    uint32_t y[16];
#pragma unroll
    for (int k = 0; k < 32; k += 2)
      y[k / 2] = f16x2_of(ex2(__uint_as_float(u[k]) + (lsv + next)), ex2(__uint_as_float(u[k + 1]) + (lsv + next)));
    tmem_st16(scores + k0 / 2, y);
    tmem_st_wait();
  });
  sm.own_neg[x][p][c] = now;
  sm.own_rel[x][p][c] = next;
  return make_float2(fmaf(l, ex2(shift), sum), ex2(shift + (next - rel)));
}
// The halves of a shared tile of columns, at least one of them such: their O's weights and the sum of both (x, y, z).
template <int D>
__device__ __noinline__ float4 far_join(Smem<D>& sm, int p, int c, float neg, float neg_b, float lref, float l, float lb) {
  auto from = [&](float own, float rel, float n) {
    return own == own ? make_float2(own, rel) : make_float2(n + lref, n < -kNoMax ? -lref : n);
  };
  const float2 a = from(sm.own_neg[0][p][c], sm.own_rel[0][p][c], neg), b = from(sm.own_neg[1][0][c], sm.own_rel[1][0][c], neg_b);
  float4 w = make_float4(1.0f, 0.0f, l, 0.0f);
  float2 both = a;
  if (lb != 0.0f) {
    const float d = (b.x - a.x) + (b.y - a.y);
    both.x = fminf(a.x, b.x);
    both.y = d < 0.0f ? (b.x - both.x) + b.y : (a.x - both.x) + a.y;
    w = make_float4(ex2(fminf(d, 0.0f)), ex2(-fmaxf(d, 0.0f)), fmaf(lb, ex2(both.x - b.x), l * ex2(both.x - a.x)), 0.0f);
  }
  sm.own_neg[0][p][c] = both.x;
  sm.own_rel[0][p][c] = both.y;
  return w;
}
// y of the page's keys where maxima are large (kKv8Large), over the S that it came from; their sum.
__device__ __noinline__ float large_probabilities(uint32_t scores, int seen, float fs, float lsv, float neg) {
  float sum = 0.0f;
#pragma unroll 1
  for (int k0 = 0; k0 < 64; k0 += 32) {
    uint32_t u[32], y[16];
    tmem_ld32(scores + k0, u);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      float z[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        asm volatile("" : "+r"(u[k + j]));       // not before the wait
        // as `largest` rounds it; kTop minus the maximum is rounded, too, by up to 8
        const float t = fmaf(__uint_as_float(u[k + j]), fs, lsv) + neg;
        z[j] = k0 + k + j < seen ? ex2(t > 15.0f ? 15.0f : t) : 0.0f;            // what is no number stays so
        sum += z[j];
      }
      y[k / 2] = f16x2_of(z[0], z[1]);
    }
    tmem_st16(scores + k0 / 2, y);
    tmem_st_wait();
  }
  return sum;
}
template <int D>
struct Softmax {
  using X = Shape<D>;
  const Kv8AttnArgs& a;
  Smem<D>& sm;
  uint32_t scores, out;                          // tensor memory, with the warp's lanes
  int x, p, c, lane;                             // half, page of each tile, column of the half

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, wait_or_abort(bar, parity, a.wait_budget, &sm.abort));
  }
  // The two warps that share 32 columns meet; true if any thread of them says so.
  __device__ __forceinline__ bool either(bool on) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.aligned.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)on), "r"(1 + 4 * x + (c >> 5))
                 : "memory");
    return r != 0;
  }
  // S of the page's N keys from key at on; to be used after `arrived`.
  template <int N>
  __device__ __forceinline__ static void arrived(uint32_t (&u)[N]) {
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < N; ++k) asm volatile("" : "+r"(u[k]));       // not before the wait
  }
  // The largest of s + log2 sv over the page's keys that the column sees.
  __device__ __forceinline__ float largest(int seen, float fs, float lsv) {
    float top = -INFINITY;
#pragma unroll 1
    for (int k0 = 0; k0 < 64; k0 += 32) {
      const int left = seen - k0;
      uint32_t u[32];
      tmem_ld32(scores + k0, u);
      arrived(u);
      auto at = [&](int k) { return k < left ? __uint_as_float(u[k]) : -INFINITY; };
      float m[4] = {at(0), at(1), at(2), at(3)};
#pragma unroll
      for (int k = 4; k < 28; k += 8)
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = max3(m[j], at(k + j), at(k + 4 + j));
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = fmaxf(m[j], at(28 + j));
      top = fmaxf(top, fmaf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), fs, lsv));
    }
    return top;
  }
  // y of the page's keys, packed; their sum.
  template <bool kMasked>
  __device__ __forceinline__ float probabilities(int seen, float fs, float base, uint32_t (&y)[32]) {
    uint32_t u[2][16];
    tmem_ld16(scores, u[0]);
    const float2 f = make_float2(fs, fs), b = make_float2(base, base);
    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t (&v)[16] = u[j & 1];
      arrived(v);
      if (j < 3) tmem_ld16(scores + 16 * (j + 1), u[(j + 1) & 1]);    // while this one is worked on
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        float2 z = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), f, b);
        if (kMasked) {
          if (16 * j + k >= seen) z.x = -INFINITY;
          if (16 * j + k + 1 >= seen) z.y = -INFINITY;
        }
        z.x = ex2(z.x);
        z.y = ex2(z.y);
        sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], z);
        y[8 * j + k / 2] = f16x2_of(z.x, z.y);
      }
    }
    return (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
  }
  // A wait that runs out is told to the column's other warp where the two meet, and both end there; the
  // CTA's last barrier is all that follows.
  __device__ __forceinline__ void run(const Share& sh, int RG, int4& rec) {
    Walk w;
    uint32_t i = 0, n = 0;                       // tiles of the CTA, of this half
    uint32_t segs = 0, joints = 0;               // segments, those of one tile of columns
    bool joined = false;                         // the segment before was one
    bool ok = true;
    for (bool more = w.first(a, RG, sh); more; more = w.next_segment(a, RG)) {
      const Group& gr = w.gr;
      const bool whole = w.whole();
      if (gr.tiles > 0 && !whole && w.t0 == 0)
        rec = make_int4(gr.r0, gr.g | (w.h << 16), blockIdx.x,
                        (int)min((long long)gridDim.x - 1, blockIdx.x + quotient(gr.tiles - w.left + sh.per - 1, sh.per)));
      if (w.t >= w.t_end) {
        if (gr.tiles > 0 || x > 0 || p > 0) continue;   // the share begins behind the segment's last tile
        if (c == 0) raise_flag(a.status, CSA_FLAG_ROW_INVALID);
        const int heads = a.heads * a.G;
        uint4* dst = reinterpret_cast<uint4*>(a.out + (size_t)gr.r0 * heads * D);
        for (int k = c; k < heads * (D / 8); k += kHalf) dst[k] = make_uint4(0u, 0u, 0u, 0u);
        for (int k = c; k < heads && a.lse; k += kHalf) a.lse[(size_t)gr.r0 * heads + k] = -INFINITY;
        continue;
      }
      const int cols = gr.g * a.G;
      const bool joint = cols <= kHalf;
      if (x > 0 && joined) ok = wait(&sm.b_free, (joints - 1) & 1) && ok;         // half a has read O
      const int qx = joint ? 0 : x;
      if (p == 0 && (x == 0 || !joint)) {        // the segment before's last S of this half is complete
        convert_queries<D>(a, sm, gr, w.h, x);
        fence_proxy_async_smem();
        warp_arrive(&sm.q_full[x], lane);        // the warp's factors are visible to it
      } else {
        ok = wait(&sm.q_full[qx], (qx > 0 ? segs - joints : segs) & 1) && ok;
      }
      ++segs;
      joined = joint;
      const int col = joint ? c : kHalf * x + c, in_group = col / a.G;
      // a column that no query has sees all there is: only pages at a row's end need a mask; warps
      // of such columns leave S as it is
      const int pos = col < cols ? gr.p0 + in_group : INT_MAX - 1;
      const bool idle = col - lane >= cols;
      const float factor = sm.factor[qx][c];
      const uint32_t n0 = n;
      const int tiles = w.t_end - w.t, step = joint ? 2 : 1;
      float neg = -kNoMax, l = 0.0f, lref = 0.0f;
      sm.own_neg[x][p][c] = __int_as_float(0x7FFFFFFF);
#pragma unroll 1
      for (int at = joint ? x : 0; at < tiles; at += step, ++n) {
        const uint32_t ti = i + at;
        if (idle) {
          if (!(ok = wait(&sm.s_full[x], n & 1) && ok)) break;
          warp_arrive(&sm.p_full[x], lane);
          continue;
        }
        ok = wait(&sm.tile_full[ti % X::kTiles], (ti / X::kTiles) & 1) && ok;
        const Tile& t = sm.tile[ti % X::kTiles];
        if (n == n0) lref = t.lref;
        const int first = t.first[p], seen = first == INT_MAX ? 0 : min(64, max(0, pos - first + 1));
        const float fs = factor * t.sk[p], isv = t.isv[p];
        float lsv = t.lsv[p];
        const bool masked = __any_sync(0xFFFFFFFFu, seen < 64);
        ok = wait(&sm.s_full[x], n & 1) && ok;
        tc_fence_after();
        // With the maximum so far, first: sums of y up to 2^15 mean that none is too large.  Else the
        // maximum moves and y is formed anew; usually only in a segment's first tile.
        uint32_t y[32];
        float sum = 0.0f;
        bool moves = n == n0;
#pragma unroll 1
        for (;;) {
          if (moves) {
            const bool far = lsv == INFINITY;
            if (!far) sm.pair[x][p][c] = largest(seen, fs, lsv);
            ok = wait(&sm.pv_done[x], (n & 1) ^ 1) && ok;             // O of the tiles before is complete
            if (either(!ok)) return;
            tc_fence_after();
            float corr;
            if (far) {                           // the tile is here, so both warps say so
              const float2 r = far_tile(sm, scores, x, p, c, seen, fs, t.own[p], neg, lref, l);
              l = r.x;
              corr = r.y;
            } else {
              const float now = fminf(neg, kTop - fmaxf(sm.pair[x][0][c], sm.pair[x][1][c]));
              corr = ex2(now - neg);
              neg = now;
              l *= corr;
            }
            if (n > n0) {                        // a half of the dims each
#pragma unroll 1
              for (int d = p * (D / 2); d < (p + 1) * (D / 2); d += 16) {
                uint32_t u[16];
                tmem_ld16(out + d, u);
                arrived(u);
#pragma unroll
                for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * corr);
                tmem_st16(out + d, u);
              }
            }
            if (far) {
              tmem_ld32(scores, y);
              arrived(y);
              sum = 0.0f;                        // l has the tile already
              break;
            }
          }
          sum = masked ? probabilities<true>(seen, fs, neg + lsv, y) : probabilities<false>(seen, fs, neg + lsv, y);
          if (moves) {
            if (__any_sync(0xFFFFFFFFu, fabsf(neg) > kKv8Large && neg < -kNoMax)) {
              sum = large_probabilities(scores, seen, fs, lsv, neg);
              tmem_ld32(scores, y);
              arrived(y);
            }
            break;
          }
          if (!either(sum > kMost || !ok)) break;
          moves = true;
        }
        l = fmaf(sum, isv, l);
        // over the S that it came from
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
          uint32_t part[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) part[k] = y[j + k];
          tmem_st16(scores + j, part);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&sm.p_full[x], lane);
      }
      i += tiles;
      // ---- the segment's output: a column and half of its dims a thread
      if (n > n0) ok = wait(&sm.pv_done[x], (n - 1) & 1) && ok;
      if (joint && x > 0) {                      // half a's to write
        sm.joined[p][c] = make_float2(neg, n > n0 ? l : 0.0f);
        tc_fence_before();
        warp_arrive(&sm.b_full, lane);
        ++joints;
        continue;
      }
      if (joint) ok = wait(&sm.b_full, joints++ & 1) && ok;
      sm.pair[x][p][c] = l;
      if (either(!ok)) return;
      l = sm.pair[x][0][c] + sm.pair[x][1][c];
      float own = 1.0f, others = 0.0f;           // weights of the halves' O
      if (joint) {
        const float2 b = sm.joined[0][c];
        const float lb = b.y + sm.joined[1][c].y, na = sm.own_neg[0][p][c], nb = sm.own_neg[1][0][c];
        if (na == na || nb == nb) {
          const float4 w = far_join(sm, p, c, neg, b.x, lref, l, lb);
          own = w.x;
          others = w.y;
          l = w.z;
        } else {
          const float now = fminf(neg, b.x);
          own = ex2(now - neg);
          others = lb == 0.0f ? 0.0f : ex2(now - b.x);
          l = lb == 0.0f ? l * own : fmaf(lb, others, l * own);
          neg = now;
        }
      }
      const bool two = __any_sync(0xFFFFFFFFu, others != 0.0f);
      tc_fence_after();
      const int slot = w.t0 > 0 ? 2 * (int)blockIdx.x : 2 * (int)blockIdx.x + 1;
      float m = -(neg + lref), up = pow2((int)lref);
      const float own_neg = sm.own_neg[x][p][c];
      if (own_neg == own_neg) {                  // by halves, as all of the difference may pass fp32's range
        m = -own_neg;
        up = ex2(-0.5f * sm.own_rel[x][p][c]);
        own *= up;
        others *= up;
      }
      const float f = l == 0.0f ? 0.0f : up / l;
      if (col < cols && p == 0) {
        if (whole) {
          const size_t row = (size_t)(gr.r0 + in_group) * a.heads * a.G + w.h * a.G + (col - in_group * a.G);
          if (a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (log2f(l) + m) * kLn2;
        } else {
          a.part_ml[(size_t)slot * 2 * 2 * kHalf + col] = m;
          a.part_ml[((size_t)slot * 2 + 1) * 2 * kHalf + col] = l;
        }
      }
      // Through the place of the columns' own queries (their first parts' for one warp, the second's for
      // the other), D bytes of a column at a time: rows of as many bytes go out together.  Stored from where
      // they are, a column's dims at a stride of its row, they took 11 thousand clocks a segment.
      constexpr int kPieces = D / 16;            // of 16 bytes
      uint8_t* stage = sm.q[x][p] + (c - lane) * D;
      auto place = [&](int column, int piece) -> uint4* {
        return reinterpret_cast<uint4*>(stage + column * D + 16 * (piece ^ (column * kPieces / 8 & (kPieces - 1))));
      };
      const size_t base = whole ? ((size_t)gr.r0 * a.heads * a.G + w.h * a.G) * (2 * D) : (size_t)slot * 2 * kHalf * (4 * D);
      uint8_t* dst = (whole ? reinterpret_cast<uint8_t*>(a.out) : reinterpret_cast<uint8_t*>(a.part)) + base;
      const int line = whole ? 2 * D : 4 * D;    // bytes of a column
      const int mine = whole ? in_group * (a.heads - 1) * a.G + col : col;       // lines from dst on
#pragma unroll 1
      for (int from = p * (line / 2); from < (p + 1) * (line / 2) && !idle; from += D) {
        const int d0 = whole ? from >> 1 : from >> 2, dims = whole ? D / 2 : D / 4;
#pragma unroll 1
        for (int d = 0; d < dims; d += 16) {
          uint32_t u[16];
          tmem_ld16(out + d0 + d, u);
          arrived(u);
          float o[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __uint_as_float(u[k]) * own;
          if (two) {
            tmem_ld16(out + kHalf + d0 + d, u);
            arrived(u);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (others != 0.0f) o[k] = fmaf(__uint_as_float(u[k]), others, o[k]);
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = f == 0.0f ? 0.0f : o[k] * f;
          if (whole) {
            uint32_t z[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]);
              z[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *place(lane, d / 8) = make_uint4(z[0], z[1], z[2], z[3]);
            *place(lane, d / 8 + 1) = make_uint4(z[4], z[5], z[6], z[7]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *place(lane, d / 4 + k) = make_uint4(__float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]),
                                                   __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3]));
          }
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
          const int column = k * (32 / kPieces) + lane / kPieces, piece = lane % kPieces;
          const int to = __shfl_sync(0xFFFFFFFFu, mine, column);
          const uint4 v = *place(column, piece);
          if (col - lane + column < cols) *reinterpret_cast<uint4*>(dst + (size_t)to * line + from + 16 * piece) = v;
        }
        __syncwarp();
      }
      tc_fence_before();
      if (joint) warp_arrive(&sm.b_free, lane);
      (void)either(false);                       // both are done with the queries' place and with `pair`
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_kv8_wide(Kv8AttnArgs a, int RG) {
  extern __shared__ __align__(128) uint8_t s_raw[];
  using X = Shape<D>;
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(s_raw);
  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  pdl_trigger();
  if (tid == 0) {
    for (int k = 0; k < X::kKeyStages; ++k) {
      mbar_init(&sm.k_full[k], 1);
      mbar_init(&sm.k_free[k], 2);
    }
    for (int k = 0; k < X::kTiles; ++k) mbar_init(&sm.tile_full[k], 1);
    for (int k = 0; k < X::kValueStages; ++k) {
      mbar_init(&sm.raw_full[k], 1);
      mbar_init(&sm.raw_free[k], 4);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&sm.v_full[k], 4);
      mbar_init(&sm.v_free[k], 1);
      mbar_init(&sm.q_full[k], 4);
      mbar_init(&sm.s_full[k], 1);
      mbar_init(&sm.p_full[k], 8);
      mbar_init(&sm.pv_done[k], 1);
    }
    mbar_init(&sm.b_full, 8);
    mbar_init(&sm.b_free, 8);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&sm.tmem_base, X::kTmem);
  const Share sh = find_share<kThreads>(a, RG, sm.share);   // its barriers make the above visible
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  if (warp < kConvertWarp) {
    int4 rec = make_int4(-1, 0, 0, 0);
    const int x = (warp >> 2) & 1, p = warp >> 3;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    Softmax<D> role{a, sm, lanes + X::kScores + 128 * x + 64 * p, lanes + X::kOut + 128 * x, x, p, tid & (kHalf - 1), lane};
    role.run(sh, RG, rec);
    if (tid == 0) a.rec[blockIdx.x] = rec;
  } else {
    if (warp == kKeyWarp) copy_side<D, true>(a, sm, sh, RG);
    else if (warp == kValueWarp) copy_side<D, false>(a, sm, sh, RG);
    else if (warp == kMmaWarp) Products<D>{a, sm, 0}.run(sh, RG);
    else if (warp == kScaleWarp) prepare_scales<D>(a, sm, sh, RG);
    else convert_values<D>(a, sm, sh, RG);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && sm.abort) raise_flag(a.status, CSA_FLAG_TIMEOUT);
  if (warp == kMmaWarp) tmem_dealloc(tmem, X::kTmem);
}

template <int D>
cudaError_t launch_dim(Kv8AttnArgs a, uint8_t* ws, int num_sms, cudaStream_t stream) {
  static_assert(sizeof(Smem<D>) <= 232448, "shared memory");
  const int grid = kv8_wide_grid(a.rows.num_rows, a.heads, a.rows.max_entries, num_sms);
  kv8_place_parts(a, ws, grid, 2 * kHalf);
  a.gap = kGap;
  constexpr int smem = (int)sizeof(Smem<D>);
  cudaError_t e = cudaFuncSetAttribute(k_kv8_wide<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_kernel(Order::kStream, k_kv8_wide<D>, dim3(grid), dim3(kThreads), smem, stream, a,
                    a.blocks ? 1 : 2 * kHalf / a.G);
  if (e != cudaSuccess || grid == 1) return e;
  return launch_kv8_merge(a, 2 * kHalf, grid, stream);
}

}  // namespace

cudaError_t launch_kv8_wide(const Kv8AttnArgs& a, uint8_t* ws, int num_sms, cudaStream_t stream) {
  return a.dim == 64 ? launch_dim<64>(a, ws, num_sms, stream) : launch_dim<128>(a, ws, num_sms, stream);
}

}  // namespace csa
