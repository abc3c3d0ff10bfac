// csa_dense_attn: MQA softmax attention of each row's heads over every visible
// FP4 main-KV entry and the FP8 local window, for single tokens, verify rows and
// whole prompt chunks.
//
// Mathematics.  A group is up to G = COLS / H rows of one request at consecutive
// positions; its COLS = G * H columns are independent queries that share keys.
// Its keys are one list: the W window tokens of the group's rows, padded to whole
// tiles, then the n entries that its last row sees (so a tile of entries is two
// whole pages, and finding its rows takes a few instructions); column c (row i) attends to the window
// positions in [max(0, t_i - 127), t_i] and the entries below (t_i + 1) / P.
// Per 128-key tile: S^T = K Q^T (M = 128 keys, N = COLS), p = 2^(s - m) with a
// running max m per column, O^T += V^T P^T (M = 128 dims x 4, N = COLS); keys and
// values are the same fp16 tile, read K-major by the first product and MN-major
// by the second.  Entries are exact in fp16 (e2m1 x E4M3); a window token is its
// E4M3 codes times 2^e, e in [-14, 7], also exact, and the rest of its scale, mu,
// multiplies its logits and p; rotated, e is at most 6, as a rotated pair may be sqrt(2)
// times larger than its codes.  A query is scaled by a power of two so that its
// largest element is in [128, 256), which undoes itself in the logit's factor.
// A rotated query has more bits than fp16 holds: its last 64 dims are split into
// fp16 high and low parts (22 bits), the low part four more steps of the first
// product.  Rounding it once would put the logit of a key four times the usual
// size off by about 2e-4.
//
// Work: the tiles of all groups, in row order, are one list; CTA i takes the i-th
// equal share.  A group inside one share is written out directly.  A cut group's
// parts leave unnormalised O and (m, l) in the workspace (at most two per CTA),
// and k_dense_merge joins them in CTA order.
//
// Pipeline.  One CTA per SM, roles that meet only at mbarriers:
//   8 dequantising warps (two warpgroups, two 128-dim chunks of a tile each),
//   8 softmax warps (32 keys x half of the columns each), also queries and output,
//   2 warps that issue the MMAs, one for each product, one that prefetches entries
//   into L2, and one that fetches the next queries.
// Shared memory holds Q (64 KB), P and one fp16 tile (128 KB), not two.  So the
// first product does not read it: the dequantising warps write each 128-dim chunk
// to tensor memory (two 64-column slots) as its A operand, and S of tile t + 1 is
// computed while tile t still occupies shared memory, during its softmax.  Of a
// warpgroup's two chunks the first waits in registers and the second in its slot
// until the second product has used tile t's.  That also takes 4 of the 6 KB per
// MMA off the shared-memory port, which the second product alone fills.
//
// What bounds it.  At N = 64 an MMA of M128 K16 takes 32 clocks with A in tensor
// memory and 48 with both operands in shared memory: a tile's 64 take 2700 clocks
// together.  A tile takes 5600: its shared-memory traffic (second product 1540, first
// product's Q 510, values stored 1150, the rest 300) fills the port for 3500, and the
// loads and stores queue behind the second product's, which lengthens the chain of
// two tiles (convert, S, softmax, O^T, store) that one tile of space allows.  512
// rows of 64 heads over 4 caches run at 755 TFLOP/s, 128 rows over 128 caches at 776,
// 0.40 and 0.41 of what cuBLAS reaches in bf16.  A step between groups costs about three tiles
// more (queries in, first maximum, output); one token of a short context is all step.
// One kernel is 130 KB of code and the parts that run once per group are fetched
// cold, at several clocks per instruction; loops there stay rolled.
// Measured on the way (128 rows over 128 caches, us): one serial role per tile 868;
// three roles, S from tensor memory 569; MMA loops rolled 488; entry tiles aligned to
// pages, output by plain stores 485; the list of work with the steps' cost, cuts joined
// in one wave 428; 8 softmax warps for 4, the first tile straight to its maxima 414;
// a window's cost in the list 399 (2 x 999 rows: 535, 580, 595, 435, 202, 182, 177).
#include <algorithm>

#include "attn_device.cuh"
#include "csa_internal.h"

namespace csa {

namespace {

constexpr int kThreads = 640;                    // 8 dequantising, 8 softmax, 2 MMA, 1 prefetching, 1 query-fetching warp
constexpr int kTileKeys = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running max moves when a logit exceeds it by this (log2 units): p <= 16159,
// times a window key's mu < 4, stays inside fp16 (65504), and a column rarely moves
// again after its first tile (at 8 a column of widely spread logits still moved in most
// early tiles).
constexpr float kRescaleLog2 = 13.98f;

// ---- the list of work ----------------------------------------------------------------
struct Group {
  int r0, g, b, p0;                              // first row, rows, request, first position
  int W, Wp, wlo;                                // window keys, padded to tiles, and the first one's position
  int n, tiles;                                  // tiles 0: the rows see nothing (or are invalid)
};

constexpr int kMaxPos = INT32_MAX - 1024;        // keys and positions stay within 32 bits

// Entries complete at position pos (P is 1 or 2).
__device__ __forceinline__ int entries_at(const DenseArgs& a, int pos) { return (pos + 1) >> (a.P - 1); }
__device__ __forceinline__ bool row_valid(const DenseArgs& a, int b, int pos) {
  return b >= 0 && b < a.num_requests && pos >= 0 && pos < kMaxPos && (a.rope_cos == nullptr || pos < a.rope_rows) &&
         entries_at(a, pos) <= (int64_t)a.max_pages * PAGE;
}
// Row r continues row r - 1: same request, next position, both valid.
__device__ __forceinline__ bool row_continues(const DenseArgs& a, int r) {
  if (r <= 0) return false;
  const int b = __ldg(a.row_req + r), p = __ldg(a.row_pos + r);
  return b == __ldg(a.row_req + r - 1) && p - 1 == __ldg(a.row_pos + r - 1) && p > 0 && row_valid(a, b, p) &&
         row_valid(a, b, p - 1);
}
__device__ __forceinline__ Group group_at(const DenseArgs& a, int r, int G) {
  Group q;
  q.r0 = r;
  q.b = __ldg(a.row_req + r);
  q.p0 = __ldg(a.row_pos + r);
  q.g = 1;
  if (!row_valid(a, q.b, q.p0)) {
    q.W = q.Wp = q.wlo = q.n = q.tiles = 0;
    return q;
  }
#pragma unroll 1
  while (q.g < G && r + q.g < a.num_rows && row_continues(a, r + q.g)) ++q.g;
  const int last = q.p0 + q.g - 1;
  q.wlo = max(0, q.p0 - (WIN - 1));
  q.W = a.win_codes ? last - q.wlo + 1 : 0;
  q.Wp = (q.W + kTileKeys - 1) / kTileKeys * kTileKeys;
  q.n = entries_at(a, last);
  q.tiles = (q.Wp + q.n + kTileKeys - 1) / kTileKeys;
  return q;
}
// Units of work: a tile is one; the step from one group to the next, which drains the
// pipeline and fills it again, counts as kGap, and a window, whose tile is gathered from
// the ring and converted twice, as kNear more.  Without them a share of many short
// groups takes far longer than a part of one long one.  2 x 999 rows without a window,
// up to 8 tiles each, and 128 rows of 17 to 513 tiles, us, by (kGap, kNear):
// (0, 0) 391, 473; (4, 0) 182, 411; (3, 2) 177, 403; (3, 3) 177, 399; (2, 3) 179, 403.
// Both are calls of 64 columns without rotary tables; 16 and 32 columns, and rotated
// windows, which take longer, use the same two numbers.
// A group of no tiles takes one unit: its rows are written out empty.
constexpr int kGap = 3, kNear = 3;
__device__ __forceinline__ int group_units(const Group& q) {
  return q.tiles > 0 ? q.tiles + kGap + (q.W > 0 ? kNear : 0) : 1;
}

struct Share {
  int row, t0;                                   // the first group's row, and the share's first unit in it
  int units, per;                                // units of this share (0: none) and of a whole one
};

// Inclusive running sum (or maximum) over the block's threads.
template <bool kMax, typename T>
__device__ __forceinline__ T block_scan(T v, T* s_warp) {
  const int lane = lane_id(), warp = warp_id();
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v = kMax ? max(v, y) : v + y;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  T below = kMax ? (T)-1 : (T)0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w)
    if (w < warp) below = kMax ? max(below, s_warp[w]) : below + s_warp[w];
  return kMax ? max(v, below) : v + below;
}

// This CTA's share of the list; every thread of the block takes part.
struct ShareScratch {
  long long sums[kThreads / 32], total;
  int starts[kThreads / 32], run[kThreads / 32];
  Share out;
};
__device__ __forceinline__ Share find_share(const DenseArgs& a, int G, ShareScratch& s) {
  const int tid = threadIdx.x, R = a.num_rows;
  const int each = (R + kThreads - 1) / kThreads;
  const int r_lo = min(R, tid * each), r_hi = min(R, r_lo + each);
  // the start of the run that reaches into this thread's rows
  int run = -1;
  if (G > 1) {
    int start = -1;
#pragma unroll 1
    for (int r = r_lo; r < r_hi; ++r)
      if (!row_continues(a, r)) start = r;
    const int upto = block_scan<true>(start, s.starts);
    run = __shfl_up_sync(0xFFFFFFFFu, upto, 1);
    if (lane_id() == 31) s.run[warp_id()] = upto;
    __syncthreads();
    if (lane_id() == 0) run = tid > 0 ? s.run[warp_id() - 1] : -1;
  }
  // twice over the groups that begin in this thread's rows: their units, then, in the
  // one thread whose groups hold this share's first unit, the group that does
  long long sum = 0, upto = 0, lo = 0, per = 0, units = 0, u = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int from = run;
#pragma unroll 1
    for (int r = r_lo; r < r_hi; ++r) {
      if (G > 1 && row_continues(a, r)) {
        if ((r - from) % G != 0) continue;
      } else {
        from = r;
      }
      const int n = group_units(group_at(a, r, G));
      if (pass == 0) {
        sum += n;
      } else if (lo >= u + n) {
        u += n;
      } else {
        s.out.row = r;
        s.out.t0 = (int)(lo - u);
        break;
      }
    }
    if (pass > 0) break;
    upto = block_scan<false>(sum, s.sums);
    if (tid == kThreads - 1) s.total = upto;
    __syncthreads();
    const long long total = s.total;
    per = (max(1ll, total - kGap - kNear) + gridDim.x - 1) / gridDim.x;   // nothing follows the last group
    lo = min(total, (long long)blockIdx.x * per);
    units = (blockIdx.x + 1 == gridDim.x ? total : min(total, lo + per)) - lo;
    u = upto - sum;
    if (units == 0 || lo < u || lo >= upto) break;
  }
  __syncthreads();
  Share h = s.out;
  h.units = (int)units;                          // a share is far below 2^31 tiles
  h.per = (int)per;
  return h;
}

// ---- shared memory ---------------------------------------------------------------------
constexpr int kDequantWarps = 8, kSoftmaxWarps = 8;
// Of the softmax warps those that work: two for each quarter of the keys, half of the
// columns each, but no fewer than 16.
template <int COLS>
constexpr int kSoftmaxUsed = COLS < 32 ? 4 : kSoftmaxWarps;
constexpr int kMmaWarp = kDequantWarps + kSoftmaxWarps;
// Running max of a column that has seen nothing: its first visible key's logit exceeds
// it by far, so the key moves it like any other that does.  (With one max of 0 for all
// such columns, one whose logits lie far below 0 lost its p to fp16.)
constexpr float kNoMax = -3e38f;

// Tensor memory columns: O^T chunk c at 64 c, S^T of even and odd tiles, and
// the two chunks of K.
constexpr uint32_t kTmemS = 256, kTmemK = 384;

template <int COLS>
struct Smem {
  uint8_t k[kTileKeys * D * 2];                  // values: 64-dim atoms of 16 KB: (key/8)*1024 + (key%8)*128
  uint8_t q[COLS * D * 2];                       // 64-position atoms of COLS * 128 B: (c/8)*1024 + (c%8)*128
  uint8_t q_lo[COLS * 256];                      // low parts of the rotated dims, zero elsewhere: chunk 3's two atoms
  uint8_t p[kTileKeys * 128];                    // (key/8)*1024 + (key%8)*128, columns along the row
  float mu[2][kTileKeys];                        // per tile: factor of a key's logit and p; < 0: left out;
  uint32_t odd[2][4];                            // read where set: 32 keys some of which are window keys or left out
  float factor[COLS];                            // of a column's logits (log2 units)
  float neg_m[COLS];                             // minus the running max
  float red[4][COLS];                            // per softmax warp: maxima of a tile, sums of p
  float corr[COLS];                              // correction of a column whose max moved; after a segment's last
                                                 // tile 1 / l (0: nothing seen)
  uint64_t k_full[2], k_free[2];                 // a chunk of K in tensor memory
  uint64_t v_full[4], v_free[4];                 // a 128-dim chunk of the tile in shared memory
  uint64_t s_full[2], s_free[2];                 // S^T of a tile
  uint64_t p_full, p_free, q_raw, q_full, q_free, o_full, o_free, drain;
  uint32_t moved[2];                             // bit c: column c's max moved
  uint32_t tmem_base;
  volatile int abort;                            // a wait ran out: every role leaves
  volatile int tile_now;                         // tiles whose S is issued; the prefetch runs ahead of it
};

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_top(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// D += A B with A in tensor memory (M = 128 lanes, two fp16 per column).
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 lanes x 64 columns: register 4g + e of lane l is row l/4 (+ 8 for e >= 2),
// column 8g + 2(l%4) + (e & 1).
__device__ __forceinline__ void tmem_st_16x64(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 16 lanes x 32 columns, laid out likewise.
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// (tmem_ld_wait before use)
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Bounded wait; false once any role's wait ran out.
template <bool kPoll = false>
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, long long budget, volatile int* abort) {
  auto probe = [&] { return kPoll ? mbar_try_wait_poll(bar, parity) : mbar_try_wait(bar, parity); };
  if (probe()) return true;
  const long long t0 = clock64();
  while (!probe()) {
    if (*abort) return false;
    if (clock64() - t0 > budget) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// The softmax warps' barriers.
template <int COLS>
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftmaxUsed<COLS>) : "memory");
}
template <int COLS>
__device__ __forceinline__ bool softmax_sync_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 2, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(32 * kSoftmaxUsed<COLS>)
      : "memory");
  return r != 0;
}
// The warp's writes are done: one arrival.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// ---- this CTA's tiles, segment by segment ------------------------------------------------
struct Walk {
  Group gr;
  int left;                                      // units of the share from this segment's first one on
  int t0, t, t_end;                              // the segment's tiles and the current one
  __device__ __forceinline__ bool open(const DenseArgs& a, int G, int row, int first) {
    if (left <= 0) return false;
    gr = group_at(a, row, G);
    t0 = t = first;
    t_end = min(gr.tiles, first + left);
    return true;
  }
  // the share's first segment; false when the share is empty
  __device__ __forceinline__ bool first(const DenseArgs& a, int G, const Share& s) {
    left = s.units;
    return open(a, G, s.row, s.t0);
  }
  __device__ __forceinline__ bool next_segment(const DenseArgs& a, int G) {
    left -= group_units(gr) - t0;
    return open(a, G, gr.r0 + gr.g, 0);
  }
  // the first tile at or after t; false at the share's end
  __device__ __forceinline__ bool settle(const DenseArgs& a, int G) {
    while (t >= t_end)
      if (!next_segment(a, G)) return false;
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && left >= gr.tiles; }
};

// ---- dequantising ------------------------------------------------------------------------
// A warp holds 32 keys (its tensor-memory quarter); its warpgroup takes chunks 2 wg
// and 2 wg + 1, 128 dims each.  Lane 4r + q holds rows r, r + 8, r + 16, r + 24, of
// each chunk the 32 dims from 32 q (16 bytes: four words of 8 dims, two scales).
// Four dims sit in two neighbouring columns of tensor memory; S sums over dims in
// any order, and Q is laid out to match: dims d .. d + 3 (d a multiple of 4) of a chunk
// are place d / 32, of four, in its 16-dim step (d / 4) % 8.  In shared memory lanes q >= 2
// put word i where word i ^ 2 belongs, so that a quarter-warp's 16-byte stores hit
// distinct banks; that permutes rows of O^T, and write_out undoes it.
struct Raw {
  uint4 w[2][4];                                 // [chunk][row]
  uint16_t sc[2][4];                             // [chunk][row]: the lane's two scales
};

// Where a warp's 32 entries lie: half a page.  A warp with nothing to read (past the
// last entry, or a page outside the pool) takes some page's codes, and scales of zero.
struct Rows {
  const uint8_t *data, *scales;                  // the lane's bytes of its first row
  uint32_t valid;                                // bit s: row s is there to read
  // pg: the page table's word; e: the lane's first entry
  __device__ __forceinline__ void set(const DenseArgs& a, int pg, int e, int n, int wg, int q) {
    const bool ok = (uint32_t)pg < (uint32_t)a.num_pages;
    const uint8_t* page = a.kv_pool + (size_t)(ok ? pg : 0) * KV_PAGE;
    const int slot = e & (PAGE - 1);
    data = page + slot * 256 + wg * 128 + 16 * q;
    scales = page + KV_SCALE_OFF + slot * 32 + wg * 16 + 2 * q;
    const int rows = ok ? min(4, max(0, (n - e + 7) >> 3)) : 0;
    valid = (1u << rows) - 1u;
  }
  __device__ __forceinline__ void fetch(Raw& x) const {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x.w[h][s] = ldg_nc_v4(data + s * 2048 + h * 64);
        x.sc[h][s] = 0;
        if ((valid >> s) & 1u) x.sc[h][s] = ldg_nc_u16(scales + s * 256 + h * 8);
      }
  }
};
// The page table's word for the warp's 32 entries from e0 on; -1 past the last one.
__device__ __forceinline__ int find_page(const int32_t* row, int e0, int n) {
  return e0 < n ? __ldg(row + (e0 >> 6)) : -1;
}

// h: tensor-memory register order of two rows (r, r + 8): pair k (two dims) of row j
// of the thread's 16 pairs.
__device__ __forceinline__ constexpr int h_at(int j, int k) { return 4 * (k / 2) + 2 * j + k % 2; }

// Two words of an entry: 16 dims, one scale (in both halves).
__device__ __forceinline__ void words_to_f16(uint32_t w0, uint32_t w1, __half2 scale, uint32_t (&o)[8]) {
  uint32_t f[4];
  e2m1x8_to_f16(w0, f);
#pragma unroll
  for (int g = 0; g < 4; ++g) o[g] = hmul2_u32(f[g], scale);
  e2m1x8_to_f16(w1, f);
#pragma unroll
  for (int g = 0; g < 4; ++g) o[4 + g] = hmul2_u32(f[g], scale);
}

// The rotated dims of a window row, in fp32, rounded once: u, v hold the lane's 32
// codes, pu, pv its partner's (the other halves of the pairs).  Out of line: lanes
// q >= 2 of chunk 3 of the tiles with window keys.
__device__ __noinline__ void rotate_window(const float* cos, const float* sin, bool lower, float pw, uint4 u, uint4 v,
                                           uint4 pu, uint4 pv, uint32_t (&o)[16]) {
  const uint32_t mine[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  const uint32_t other[8] = {pu.x, pu.y, pu.z, pu.w, pv.x, pv.y, pv.z, pv.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t f[2], g[2];
    e4m3x4_to_f16(mine[i], f);
    e4m3x4_to_f16(other[i], g);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 m = __half22float2(*reinterpret_cast<const __half2*>(&f[k]));
      const float2 n = __half22float2(*reinterpret_cast<const __half2*>(&g[k]));
      const float mx[2] = {m.x * pw, m.y * pw}, nx[2] = {n.x * pw, n.y * pw};
      float r[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float c = __ldg(cos + 4 * i + 2 * k + t), s = __ldg(sin + 4 * i + 2 * k + t);
        r[t] = lower ? __fsub_rn(__fmul_rn(mx[t], c), __fmul_rn(nx[t], s))
                     : __fadd_rn(__fmul_rn(mx[t], c), __fmul_rn(nx[t], s));
      }
      const __half2 z = __floats2half2_rn(r[0], r[1]);
      o[2 * i + k] = *reinterpret_cast<const uint32_t*>(&z);
    }
  }
}

// One warpgroup's chunks, 2 wg and 2 wg + 1, of every tile.
template <int COLS>
struct Dequant {
  using S = Smem<COLS>;
  const DenseArgs& a;
  S& sm;
  int lane, wg, q, key0;                         // key0: the thread's first row in the tile
  uint32_t tslot;                                // the warp's lanes of the warpgroup's K slot

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, wait_or_abort(bar, parity, a.wait_budget, &sm.abort));
  }
  // word i of row s of chunk c
  __device__ __forceinline__ static uint8_t* value_at(S& sm, int c, int key0, int s, int q, int i) {
    return sm.k + (2 * c + (q >> 1)) * 16384 + ((key0 >> 3) + s) * 1024 + swz128(key0 & 7, 4 * (q & 1) + (i ^ (q & 2)));
  }

  // A chunk of a tile with window keys, for the first product (values: for the
  // second).  A window token is its codes times 2^e, e in [-14, 7] (exact); the rest
  // of its scale is mu, below 2 for scales up to 2^8.  448 * 2^7 fits fp16 and
  // 448 * 2^7 * sqrt(2) does not, so with rotary tables e ends at 6 and mu below 4.
  // ki: the thread's first key.
  __device__ __noinline__ static bool near_chunk(const DenseArgs& a, S& sm, bool values, int lane, int wg, int q,
                                                 int key0, uint32_t tslot, int h, uint32_t tile, int ki, int W,
                                                 int wlo, int b) {
    const int c = 2 * wg + h;
    const bool turn = c == 3 && q >= 2 && a.rope_cos != nullptr;
    const int top = a.rope_cos ? 6 : 7;          // of all chunks: a token has one mu
    if (!values && c == 0 && lane == 0) sm.odd[tile & 1][key0 >> 5] = 1u;
    // the four rows' codes, before the wait
    uint4 u[4], v[4];
    float ws[4];
    const uint8_t* src[4];
    int at = (wlo + ki) % a.win_cap;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u[s] = v[s] = make_uint4(0u, 0u, 0u, 0u);
      ws[s] = 0.0f;
      const size_t ring = (size_t)b * a.win_cap + at;
      src[s] = a.win_codes + ring * D + c * 128 + 32 * q;
      if (ki + 8 * s < W) {
        u[s] = ldg_nc_v4(src[s]);
        v[s] = ldg_nc_v4(src[s] + 16);
        ws[s] = ldg_nc_f32(a.win_scale + ring);
      }
      at += 8;
      while (at >= a.win_cap) at -= a.win_cap;
    }
    const bool ok = wait_or_abort(values ? &sm.v_free[c] : &sm.k_free[wg], values ? (tile & 1) ^ 1 : h ^ 1,
                                  a.wait_budget, &sm.abort);
    if (!__all_sync(0xFFFFFFFFu, ok)) return false;
    tc_fence_after();
#pragma unroll
    for (int s0 = 0; s0 < 4; s0 += 2) {          // two rows, r and r + 8
      uint32_t o[2][16];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = ki + 8 * (s0 + j);
        const float scale = ws[s0 + j];
        const int ex = min(top, max(-14, (int)((__float_as_uint(scale) >> 23) & 255u) - 127));
        const float pw = copysignf(pow2(ex), scale);
        if (turn && k < W) {
          const size_t row = (size_t)(wlo + k) * 32;
          uint32_t t[16];
          const uint8_t* other = src[s0 + j] + 32 * (5 - 2 * q);   // dims 448 + 32 (q - 2): the halves are q = 2 and 3
          rotate_window(a.rope_cos + row, a.rope_sin + row, q == 2, pw, u[s0 + j], v[s0 + j], ldg_nc_v4(other),
                        ldg_nc_v4(other + 16), t);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[j][i] = t[i];
        } else {
          const __half2 hp = __float2half2_rn(pw);
          const uint4 x = u[s0 + j], y = v[s0 + j];
          const uint32_t cw[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t f[2];
            e4m3x4_to_f16(cw[i], f);
            o[j][2 * i] = hmul2_u32(f[0], hp);
            o[j][2 * i + 1] = hmul2_u32(f[1], hp);
          }
        }
        if (!values && c == 0 && q == 0) {
          // an infinite scale gives NaN, like NaN itself: the rows that see the token become
          // NaN, and P is 0 in the others, which an infinite mu would turn into NaN as well
          const float mu = fabsf(scale) * pow2(-ex);
          sm.mu[tile & 1][key0 + 8 * (s0 + j)] = k < W ? fmaf(mu, 0.0f, mu) : -1.0f;
        }
      }
      __syncwarp();
      if (!values) {
        uint32_t t[32];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          t[h_at(0, k)] = o[0][k];
          t[h_at(1, k)] = o[1][k];
        }
        tmem_st_16x64(tslot + ((uint32_t)(8 * s0) << 16), t);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(value_at(sm, c, key0, s0 + j, q, i)) =
                make_uint4(o[j][4 * i], o[j][4 * i + 1], o[j][4 * i + 2], o[j][4 * i + 3]);
      }
    }
    if (!values) {
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&sm.k_full[wg], lane);
    } else {
      fence_proxy_async_smem();
      warp_arrive(&sm.v_full[c], lane);
    }
    return true;
  }

  __device__ __forceinline__ void run(const Share& sh, int G) {
    Walk w;
    uint32_t tile = 0;
    for (bool more = w.first(a, G, sh); more; more = w.next_segment(a, G)) {
      const int32_t* row = a.page_table + (size_t)w.gr.b * a.max_pages;
      const int n = w.gr.n;
      int left = w.t_end - w.t;                  // tiles of the segment
      int ki = w.t * kTileKeys + key0;           // the thread's first key
#pragma unroll 1
      for (; left > 0 && ki < w.gr.Wp; --left, ki += kTileKeys, ++tile) {
#pragma unroll 1
        for (int part = 0; part < 4; ++part)     // both chunks for the first product, then for the second
          if (!near_chunk(a, sm, part >= 2, lane, wg, q, key0, tslot, part & 1, tile, ki, w.gr.W, w.gr.wlo, w.gr.b))
            return;
      }
      if (left <= 0) continue;
      int e = ki - w.gr.Wp;                      // the thread's first entry
      Raw x;
      Rows at;
      at.set(a, find_page(row, e & ~31, n), e, n, wg, q);
      at.fetch(x);
#pragma unroll 1
      for (; left > 0; --left, ++tile) {
        int next = find_page(row, (e & ~31) + kTileKeys, n);
        if (wg == 0) {                           // keys past the last one and in bad pages are left out
          const bool odd = __any_sync(0xFFFFFFFFu, at.valid != 15u);
          if (lane == 0) sm.odd[tile & 1][key0 >> 5] = odd;
          if (odd && q == 0) {
#pragma unroll 1
            for (int s = 0; s < 4; ++s) {
              const bool in = (at.valid >> s) & 1u;
              sm.mu[tile & 1][key0 + 8 * s] = in ? 1.0f : -1.0f;
              if (!in && e + 8 * s < n) raise_flag(a.status, CSA_FLAG_PAGE_OOB);
            }
          }
        }
        // ---- the first product's A operand: one chunk, whose values stay in registers,
        // then the other, which stays in the slot
        uint32_t t[4][16];                       // [2 pair + half]
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!wait(&sm.k_free[wg], h ^ 1)) return;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k) {          // 32 columns: words 2 half and 2 half + 1 of two rows
            uint32_t u[16];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint4 v = x.w[h][2 * (k >> 1) + j];
              const uint32_t sp = e4m3x2_to_f16(x.sc[h][2 * (k >> 1) + j]);
              const __half2 hs = *reinterpret_cast<const __half2*>(&sp);
              uint32_t o[8];
              words_to_f16(k & 1 ? v.z : v.x, k & 1 ? v.w : v.y, k & 1 ? __high2half2(hs) : __low2half2(hs), o);
#pragma unroll
              for (int i = 0; i < 8; ++i) u[h_at(j, i)] = o[i];
            }
            tmem_st_16x32(tslot + ((uint32_t)(16 * (k >> 1)) << 16) + 32 * (k & 1), u);
            if (h == 0) {
#pragma unroll
              for (int i = 0; i < 16; ++i) t[k][i] = u[i];
            }
          }
          tmem_st_wait();
          tc_fence_before();
          warp_arrive(&sm.k_full[wg], lane);
        }
        // ---- the second product's, as the previous tile's chunks are used up; the next
        // tile's bytes are fetched meanwhile
        e += kTileKeys;
        asm volatile("" : "+r"(next));           // not looked at before here
        at.set(a, next, e, n, wg, q);            // past the last tile: nothing to read
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!wait(&sm.v_free[2 * wg + h], (tile & 1) ^ 1)) return;
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int r = h_at(j, 4 * i);
                *reinterpret_cast<uint4*>(value_at(sm, 2 * wg + h, key0, 2 * (k >> 1) + j, q, 2 * (k & 1) + i)) =
                    make_uint4(t[k][r], t[k][r + 1], t[k][r + 4], t[k][r + 5]);
              }
          tc_fence_before();
          fence_proxy_async_smem();
          warp_arrive(&sm.v_full[2 * wg + h], lane);
          if (h == 0) {
            at.fetch(x);
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_ld_16x32(tslot + ((uint32_t)(16 * (k >> 1)) << 16) + 32 * (k & 1), t[k]);
            tmem_ld_wait();
          }
        }
      }
    }
  }
};

// ---- one warp that runs ahead ------------------------------------------------------------
// The entries of the next tiles into L2, page by page: the dequantising warps fetch
// their bytes one tile ahead only, less than a trip to memory.
constexpr int kAhead = 6;
template <int COLS>
__device__ __forceinline__ void prefetch_tiles(const DenseArgs& a, Smem<COLS>& sm, const Share& sh, int G) {
  Walk w;
  if (!w.first(a, G, sh)) return;
#pragma unroll 1
  for (int i = 0; w.settle(a, G); ++i, ++w.t) {
    if (w.t == w.t0 && i > 0 && lane_id() < COLS / 8) {   // a new segment's queries
      const int c = 8 * lane_id();
      if (c < w.gr.g * a.H) prefetch_l2(a.q + ((size_t)w.gr.r0 * a.H + c) * D, 8 * D * 2);
    }
    while (i - kAhead > sm.tile_now) __nanosleep(200);   // ends: S's issuer sets the last value on leaving
    const int lo = max(0, w.t * kTileKeys - w.gr.Wp), hi = min(w.gr.n, (w.t + 1) * kTileKeys - w.gr.Wp);
    const int page = (lo >> 6) + lane_id();
    if (lo < hi && page <= (hi - 1) >> 6) {
      const int pg = __ldg(a.page_table + (size_t)w.gr.b * a.max_pages + page);
      if ((uint32_t)pg < (uint32_t)a.num_pages) {
        const int from = max(lo, page * PAGE) & (PAGE - 1), rows = min(hi, (page + 1) * PAGE) - max(lo, page * PAGE);
        const uint8_t* src = a.kv_pool + (size_t)pg * KV_PAGE;
        prefetch_l2(src + from * 256, rows * 256);
        prefetch_l2(src + KV_SCALE_OFF + from * 32, rows * 32);
      }
    }
    __syncwarp();
  }
}

// ---- the warps that issue the MMAs ------------------------------------------------------
// One issues S, one O^T, each tile by tile and chunk by chunk (0, 2, 1, 3: the
// warpgroups take turns), so neither product waits for the other's operands.  The
// whole warp walks and waits, and every operand's address is a constant or uniform;
// one elected lane issues (with addresses formed per lane an MMA took ~110 clocks to
// issue instead of the 32 to 48 that it takes to run, and one warp choosing between
// the streams ~600 clocks per choice).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
  return r != 0;
}

template <int COLS>
struct Issue {
  using S = Smem<COLS>;
  const DenseArgs& a;
  S& sm;

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, wait_or_abort<true>(bar, parity, a.wait_budget, &sm.abort));
  }
  // step 0..3 of tile i's S: chunk (step / 2) of warpgroup (step % 2).  The step is a
  // constant, so that every operand's address is one.
  __device__ __forceinline__ bool scores(uint32_t i, int step, bool last) {
    if (!wait(&sm.k_full[step & 1], step >> 1)) return false;
    const uint64_t dQ = smem_desc(smem_u32(sm.q), 16, 1024, kSwizzle128B);
    const uint64_t dQl = smem_desc(smem_u32(sm.q_lo), 16, 1024, kSwizzle128B);
    constexpr uint32_t id = idesc_f16(128, COLS, 0, 0);
    const uint32_t ts = kTmemS + 64 * (i & 1), ta = kTmemK + 64 * (step & 1);
    const int c = 2 * (step & 1) + (step >> 1);
    tc_fence_after();
    if (elect_one()) {
      const uint64_t dq = dQ + (uint64_t)(c * 2 * (COLS * 8));
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        mma_f16_ts(ts, ta + 8 * ks, dq + (uint64_t)((ks >> 2) * (COLS * 8) + (ks & 3) * 2), id,
                   ks > 0 ? 1u : (uint32_t)(step > 0));
      if (step == 3 && a.rope_cos) {             // chunk 3 again, by the rotated dims' low parts
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_f16_ts(ts, ta + 8 * ks, dQl + (uint64_t)((ks >> 2) * (COLS * 8) + (ks & 3) * 2), id, 1u);
      }
      tc_commit(&sm.k_free[step & 1]);
      if (step == 3) {
        tc_commit(&sm.s_full[i & 1]);
        if (last) tc_commit(&sm.q_free);         // of the segment
        mbar_arrive(&sm.s_full[i & 1]);          // orders the tile's mu before its softmax
      }
    }
    __syncwarp();
    return true;
  }
  // step 0..3 of a tile's O^T; first, last: of its segment
  __device__ __forceinline__ bool values(uint32_t i, int step, bool first, bool last) {
    if (!wait(&sm.v_full[2 * (step & 1) + (step >> 1)], i & 1)) return false;
    const uint64_t dV = smem_desc(smem_u32(sm.k), 16384, 1024, kSwizzle128B);
    const uint64_t dP = smem_desc(smem_u32(sm.p), 8192, 1024, kSwizzle128B);
    constexpr uint32_t id = idesc_f16(128, COLS, 1, 1);
    const int c = 2 * (step & 1) + (step >> 1);
    tc_fence_after();
    if (elect_one()) {
      const uint64_t dv = dV + (uint64_t)(c * 2048);
#pragma unroll
      for (int ks = 0; ks < kTileKeys / 16; ++ks)
        mma_f16(64 * c, dv + (uint64_t)(ks * 128), dP + (uint64_t)(ks * 128), id, ks > 0 ? 1u : (uint32_t)!first);
      tc_commit(&sm.v_free[c]);
      if (step == 3) {
        tc_commit(&sm.p_free);
        if (last) tc_commit(&sm.o_full);
      }
    }
    __syncwarp();
    return true;
  }
  __device__ __forceinline__ void run_scores(const Share& sh, int G) {
    Walk w;
    uint32_t i = 0, seg = 0;
    for (bool more = w.first(a, G, sh); more && w.settle(a, G); ++i, ++w.t) {
      if (w.t == w.t0 && !wait(&sm.q_full, seg++ & 1)) break;
      if (!wait(&sm.s_free[i & 1], ((i >> 1) & 1) ^ 1)) break;
      bool ok = true;
#pragma unroll 1
      for (int step = 0; step < 4 && ok; ++step) ok = scores(i, step, w.t + 1 == w.t_end);
      if (!ok) break;
      if (lane_id() == 0) sm.tile_now = (int)i;
    }
    if (lane_id() == 0) sm.tile_now = INT32_MAX;   // lets the prefetching warp go
  }
  __device__ __forceinline__ void run_values(const Share& sh, int G) {
    Walk w;
    uint32_t i = 0, seg = 0;
    for (bool more = w.first(a, G, sh); more && w.settle(a, G); ++i, ++w.t) {
      const bool first = w.t == w.t0, last = w.t + 1 == w.t_end;
      if (!wait(&sm.p_full, i & 1)) break;
      if (first && !wait(&sm.o_free, (seg++ & 1) ^ 1)) break;
      bool ok = true;
#pragma unroll 1
      for (int step = 0; step < 4 && ok; ++step) ok = values(i, step, first, last);
      if (!ok) break;
    }
  }
};

__device__ __forceinline__ void swap2(uint2& a, uint2& b) {
  const uint2 t = a;
  a = b;
  b = t;
}
// ---- queries ------------------------------------------------------------------------------
// One warp copies the next segment's bf16 queries to Q's place as soon as the last S
// of the segment before is complete, while that segment's last softmax and O^T run.
// Column c's 128-byte piece of an atom lies where the fp16 ones will; pieces of 16
// bytes swap places in odd atoms, so that the warp that converts a column reads
// without bank conflicts.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, uint32_t bytes) {   // the rest is zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
template <int COLS>
__device__ __forceinline__ void fetch_queries(const DenseArgs& a, Smem<COLS>& sm, const Share& sh, int G) {
  Walk w;
  uint32_t seg = 0;
#pragma unroll 1
  for (bool more = w.first(a, G, sh); more; more = w.next_segment(a, G)) {
    if (w.t >= w.t_end) continue;
    if (seg > 0) {
      const bool ok = wait_or_abort(&sm.q_free, (seg - 1) & 1, a.wait_budget, &sm.abort);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
    }
    const int cols = w.gr.g * a.H;
    const uint8_t* src = reinterpret_cast<const uint8_t*>(a.q + (size_t)w.gr.r0 * a.H * D);
#pragma unroll 8
    for (int k = lane_id(); k < COLS * 64; k += 32) {
      const int c = k >> 6, atom = (k >> 3) & 7;
      const bool in = c < cols;
      cp_async16(sm.q + atom * (COLS * 128) + c * 128 + 16 * ((k & 7) ^ (atom & 1)), src + (in ? 16 * k : 0),
                 in ? 16u : 0u);
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sm.q_raw)) : "memory");
    ++seg;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// A softmax warp's share of the columns to fp16, in place: a column's 512 dims are
// one warp's, 16 consecutive ones a lane, and are all read before any is written.
template <int COLS>
__device__ __forceinline__ void convert_queries(const DenseArgs& a, Smem<COLS>& sm, const Group& gr, int warp, int lane) {
  constexpr int N = 2;                           // columns at a time
  constexpr int kMine = COLS / kSoftmaxUsed<COLS>;
  const int c_lo = warp * kMine;
  const bool rope = a.rope_cos != nullptr && c_lo < gr.g * a.H;
  // the rotated pairs (448 + j, 480 + j) are one a lane, j = lane
  float cs = 1.0f, sn = 0.0f;
  if (rope) {
    const size_t at = (size_t)(gr.p0 + c_lo / a.H) * 32 + lane;
    cs = __ldg(a.rope_cos + at);
    sn = __ldg(a.rope_sin + at);
  }
#pragma unroll 1
  for (int c = c_lo; c < c_lo + kMine; c += N) {
    uint32_t w[N][8];
    float big[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint8_t* src = sm.q + (lane >> 2) * (COLS * 128) + (c + j) * 128 + 32 * (lane & 3);
      const uint4 r0 = *reinterpret_cast<const uint4*>(src + 16 * ((lane >> 2) & 1));
      const uint4 r1 = *reinterpret_cast<const uint4*>(src + 16 * (((lane >> 2) & 1) ^ 1));
      const uint32_t r[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
      __nv_bfloat162 top = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&r[0]));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[j][i] = r[i];
        if (i > 0) top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&r[i])));
      }
      big[j] = fmaxf(__low2float(top), __high2float(top));
    }
    float turned[N][2];
    if (rope) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint8_t* src = sm.q + 7 * (COLS * 128) + (c + j) * 128 + 16 * ((lane >> 3) ^ 1) + 2 * (lane & 7);
        const float x = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(src) << 16);
        const float y = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(src + 64) << 16);
        turned[j][0] = __fsub_rn(__fmul_rn(x, cs), __fmul_rn(y, sn));
        turned[j][1] = __fadd_rn(__fmul_rn(y, cs), __fmul_rn(x, sn));
        big[j] = fmaxf(lane < 28 ? big[j] : 0.0f, fmaxf(fabsf(turned[j][0]), fabsf(turned[j][1])));
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) big[j] = warp_top(big[j]);
    __syncwarp();                                // both columns have been read
#pragma unroll
    for (int j = 0; j < N; ++j) {
      // 2^-e puts the largest magnitude in [128, 256); e >= -126 keeps it in fp32's
      // range, and a query of such small elements has no logit to speak of
      const int ex = (int)(__float_as_uint(big[j]) >> 23);
      const int e = (ex > 0 && ex < 255) ? max(ex - 127 - 7, -126) : 0;
      if (lane == 0) sm.factor[c + j] = a.softmax_scale * kLog2e * pow2(e);
      const float s1 = pow2(-e);
      uint2 hi[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {              // 4 dims at a time
        const uint32_t x = w[j][2 * u], y = w[j][2 * u + 1];
        const __half2 h0 = __floats2half2_rn(__uint_as_float(x << 16) * s1, __uint_as_float(x & 0xFFFF0000u) * s1);
        const __half2 h1 = __floats2half2_rn(__uint_as_float(y << 16) * s1, __uint_as_float(y & 0xFFFF0000u) * s1);
        hi[u].x = *reinterpret_cast<const uint32_t*>(&h0);
        hi[u].y = *reinterpret_cast<const uint32_t*>(&h1);
      }
      // lanes of different atoms begin with different steps: their banks differ
      const int first = (lane & 1) | ((lane >> 2) & 2);
#pragma unroll
      for (int u = 0; u < 4; u += 2)
        if (first & 1) swap2(hi[u], hi[u + 1]);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (first & 2) swap2(hi[u], hi[u + 2]);
      const int place = (lane >> 1) & 3;         // of dims 16 (lane % 8) + 4 u of a chunk; the step is 4 (lane % 2) + u
      uint8_t* dst = sm.q + (2 * (lane >> 3) + (lane & 1)) * (COLS * 128) + ((c + j) >> 3) * 1024 + 8 * (place & 1);
      if (!rope || lane < 28) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<uint2*>(dst + swz128((c + j) & 7, 2 * (u ^ first) + (place >> 1))) = hi[u];
      }
      if (rope) {
        // dims 64 + lane and 96 + lane of chunk 3 are places 2 and 3 of a step
        const int at = (lane >> 4) * (COLS * 128) + ((c + j) >> 3) * 1024 +
                       swz128((c + j) & 7, 2 * ((lane >> 2) & 3) + 1) + 2 * (lane & 3);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float x = turned[j][k] * s1;
          const __half h = __float2half_rn(x), l = __float2half_rn(x - __half2float(h));
          *reinterpret_cast<__half*>(sm.q + 6 * (COLS * 128) + at + 8 * k) = h;
          *reinterpret_cast<__half*>(sm.q_lo + at + 8 * k) = l;
        }
      }
    }
  }
}

// ---- output -------------------------------------------------------------------------------
// O^T of a segment to its rows (kParts: to a part), by the softmax warps.  Each lane
// holds a dim of 16 columns at a time, so a store of a column is one run of 32 dims;
// neighbours swap halves of two columns to store pairs of bf16.  (Put together in
// shared memory and sent as bulk copies, 64 columns took 19000 clocks, most of them
// waiting for the copies to read.)
template <int COLS, bool kParts>
__device__ __forceinline__ void write_out(const DenseArgs& a, Smem<COLS>& sm, int warp, int lane, int r0, int cols,
                                          int slot) {
  const int quarter = warp & 3;
  const int d = 32 * quarter + (lane ^ (8 * (quarter & 2)));   // the lane's dim in a chunk, as the tile was laid out
  // with two warps for a quarter of the dims, each takes two of the four chunks
  constexpr int kStep = kSoftmaxUsed<COLS> / 4;
#pragma unroll 1
  for (int j = kStep > 1 ? warp >> 2 : 0; j < cols / 8; j += kStep) {   // 16 columns of two chunks
    const int c0 = 16 * (j >> 1), dc = 2 * (j & 1);
    const uint32_t ta = 64 * dc + ((uint32_t)(32 * quarter) << 16) + c0;
    uint32_t v[2][16];
    tmem_ld16(ta, v[0]);
    tmem_ld16(ta + 64, v[1]);
    tmem_ld_wait();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int k = 0; k < 16; ++k) asm volatile("" : "+r"(v[h][k]));   // not before the wait
      if constexpr (kParts) {
        float* dst = a.part + ((size_t)slot * COLS + c0) * D + 128 * (dc + h) + d;
#pragma unroll
        for (int k = 0; k < 16; ++k) dst[k * D] = __uint_as_float(v[h][k]);
      } else {
        // the even lane of a pair stores column k, the odd one column k + 1
        const int odd = lane & 1;
        uint16_t* dst = a.out + ((size_t)r0 * a.H + c0 + odd) * D + 128 * (dc + h) + (d & ~1);
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const float x0 = __uint_as_float(v[h][k]) * sm.corr[c0 + k];
          const float x1 = __uint_as_float(v[h][k + 1]) * sm.corr[c0 + k + 1];
          const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? x0 : x1, 1);
          const __nv_bfloat162 o = odd ? __floats2bfloat162_rn(got, x1) : __floats2bfloat162_rn(x0, got);
          *reinterpret_cast<__nv_bfloat162*>(dst + k * D) = o;
        }
      }
    }
  }
}

// ---- softmax ------------------------------------------------------------------------------
template <int COLS>
struct Softmax {
  using S = Smem<COLS>;
  const DenseArgs& a;
  S& sm;
  int lane, warp;                                // 32 keys (warp % 4) and, of the tile, kCols columns (warp / 4)
  static constexpr int kCols = 4 * COLS / kSoftmaxUsed<COLS>;

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    return wait_or_abort(bar, parity, a.wait_budget, &sm.abort);
  }

  // 16 consecutive columns of the thread's lane, in pairs; tmem_ld_wait before use.
  __device__ __forceinline__ static void tmem_ld16_pairs(uint32_t taddr, float2* x) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(x[0].x), "=f"(x[0].y), "=f"(x[1].x), "=f"(x[1].y), "=f"(x[2].x), "=f"(x[2].y), "=f"(x[3].x),
          "=f"(x[3].y), "=f"(x[4].x), "=f"(x[4].y), "=f"(x[5].x), "=f"(x[5].y), "=f"(x[6].x), "=f"(x[6].y),
          "=f"(x[7].x), "=f"(x[7].y)
        : "r"(taddr));
  }
  __device__ __forceinline__ bool run(const Share& sh, int G, int4& rec) {
    Walk w;
    uint32_t i = 0, outs = 0, segs = 0;
    int prev_r0 = -1, prev_cols = 0, prev_slot = 0;
    const int quarter = warp & 3, cb = warp >> 2 ? kCols : 0;   // the first column
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    const int mykey = 32 * quarter + lane, tid = 32 * warp + lane;
    bool more = w.first(a, G, sh);
#pragma unroll 1
    for (;; more = w.next_segment(a, G)) {
      const int cols = more ? w.gr.g * a.H : 0;
      const bool whole = w.whole();
      const int slot = whole ? -1 : (w.t0 > 0 ? 2 * (int)blockIdx.x : 2 * (int)blockIdx.x + 1);
      if (more && !whole && w.t0 == 0)
        rec = make_int4(w.gr.r0, w.gr.g, blockIdx.x,
                        min((int)gridDim.x - 1, (int)blockIdx.x + (w.gr.tiles - w.left + sh.per - 1) / sh.per));
      if (more && w.t >= w.t_end) {
        if (w.gr.tiles > 0) continue;            // the share begins behind the group's last tile
        // rows that see nothing
        if (!row_valid(a, w.gr.b, w.gr.p0) && tid == 0) raise_flag(a.status, CSA_FLAG_ROW_INVALID);
        uint4* dst = reinterpret_cast<uint4*>(a.out + (size_t)w.gr.r0 * a.H * D);
        for (int k = tid; k < cols * (D / 8); k += 32 * kSoftmaxUsed<COLS>) dst[k] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse && tid < cols) a.lse[(size_t)w.gr.r0 * a.H + tid] = -INFINITY;
        continue;
      }
      if (more) {
        (void)wait(&sm.q_raw, segs++ & 1);       // one that runs out ends the role at S's wait
        convert_queries<COLS>(a, sm, w.gr, warp, lane);
        if (tid < COLS) sm.neg_m[tid] = -kNoMax;
        fence_proxy_async_smem();
        warp_arrive(&sm.q_full, lane);
        softmax_sync<COLS>();                    // factors and maxima visible to all softmax warps
      }
      if (prev_r0 >= 0) {                        // the segment before, once its last O^T is complete
        const bool ok = wait(&sm.o_full, outs & 1);
        if (softmax_sync_or<COLS>(!ok)) return false;
        ++outs;
        tc_fence_after();
        if (prev_slot < 0) write_out<COLS, false>(a, sm, warp, lane, prev_r0, prev_cols, 0);
        else write_out<COLS, true>(a, sm, warp, lane, prev_r0, prev_cols, prev_slot);
        tc_fence_before();
        warp_arrive(&sm.o_free, lane);
        prev_r0 = -1;
      }
      if (!more) break;
      bool fresh = true;                         // no column has seen a key of the segment yet
      // keys that every column sees (window keys aside); none when columns are unused
      const int all_see = cols == COLS ? w.gr.Wp + entries_at(a, w.gr.p0) : 0;
      float2 lpart[kCols / 2];                   // this key's share of the columns' sums of p
#pragma unroll
      for (int k = 0; k < kCols / 2; ++k) lpart[k] = make_float2(0.0f, 0.0f);
#pragma unroll 1
      for (; w.t < w.t_end; ++w.t, ++i) {
        const bool ok = wait(&sm.s_full[i & 1], (i >> 1) & 1);
        bool ok_warp = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        const uint32_t ts = kTmemS + 64 * (i & 1) + cb + lane_off;
        // the columns that see this key; usually all, and none is a window key
        const int ki = w.t * kTileKeys + mykey;
        int clo = 0, chi = kCols;                 // from cb on
        float mu = 1.0f;
        const bool plain = (w.t + 1) * kTileKeys <= all_see && !sm.odd[i & 1][quarter];
        if (!plain) {
          if (sm.odd[i & 1][quarter]) mu = sm.mu[i & 1][mykey];
          int ilo = 0, ihi = -1;                 // rows of the group
          if (!(mu < 0.0f)) {
            if (ki < w.gr.Wp) {
              ilo = max(0, w.gr.wlo + ki - w.gr.p0);
              ihi = min(w.gr.g - 1, w.gr.wlo + ki + (WIN - 1) - w.gr.p0);
            } else {
              ilo = max(0, ((ki - w.gr.Wp + 1) << (a.P - 1)) - 1 - w.gr.p0);
              ihi = w.gr.g - 1;
            }
          }
          clo = ilo * a.H - cb;
          chi = (ihi + 1) * a.H - cb;
        }
        const float4* fac = reinterpret_cast<const float4*>(sm.factor + cb);
        const float4* mr = reinterpret_cast<const float4*>(sm.neg_m + cb);
        const float4* al = reinterpret_cast<const float4*>(sm.corr + cb);
        float2 x[kCols / 2];
        bool moved = false;
#pragma unroll 1
        for (;;) {                               // again once the running max has moved
          if (!fresh || moved) {
            // x = logit - m; a column that does not see the key: -inf
#pragma unroll
            for (int k = 0; k < kCols; k += 16) tmem_ld16_pairs(ts + k, &x[k / 2]);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < kCols / 2; ++k) asm volatile("" : "+f"(x[k].x), "+f"(x[k].y));   // not before the wait
            if (!plain) {
#pragma unroll
              for (int k = 0; k < kCols / 2; ++k) x[k] = make_float2(x[k].x * mu, x[k].y * mu);
            }
#pragma unroll
            for (int k = 0; k < kCols; k += 4) {
              const float4 f = fac[k / 4], m = mr[k / 4];
              x[k / 2] = fma2(x[k / 2], make_float2(f.x, f.y), make_float2(m.x, m.y));
              x[k / 2 + 1] = fma2(x[k / 2 + 1], make_float2(f.z, f.w), make_float2(m.z, m.w));
            }
            if (!plain) {
#pragma unroll
              for (int k = 0; k < kCols; k += 2) {
                if (k < clo || k >= chi) x[k / 2].x = -INFINITY;
                if (k + 1 < clo || k + 1 >= chi) x[k / 2].y = -INFINITY;
              }
            }
            if (moved) break;
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < kCols / 2; ++k) top = fmaxf(fmaxf(top, x[k].x), x[k].y);
            // The running max moves only when a logit exceeds it by kRescaleLog2, or at the
            // column's first key; usually it stays, and then no max or sum is reduced.
            if (!softmax_sync_or<COLS>(!ok_warp || top > kRescaleLog2)) break;
          }
          // a failed wait ends the role here, for all of its warps alike; O^T of the
          // tile before is complete from here on
          ok_warp = __all_sync(0xFFFFFFFFu, wait(&sm.p_free, (i & 1) ^ 1)) && ok_warp;
          if (softmax_sync_or<COLS>(!ok_warp)) return false;
          tc_fence_after();
          // the columns' maxima, from S once more: 16 columns at a time keep the code of
          // what happens once or twice in a segment small
#pragma unroll 1
          for (int c0 = 0; c0 < kCols; c0 += 16) {
            float2 y[8];
            tmem_ld16_pairs(ts + c0, y);
            tmem_ld_wait();
            float t[16];
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              const float4 f = fac[(c0 + k) / 4];
              asm volatile("" : "+f"(y[k / 2].x), "+f"(y[k / 2].y), "+f"(y[k / 2 + 1].x), "+f"(y[k / 2 + 1].y));
              t[k] = y[k / 2].x * mu * f.x;
              t[k + 1] = y[k / 2].y * mu * f.y;
              t[k + 2] = y[k / 2 + 1].x * mu * f.z;
              t[k + 3] = y[k / 2 + 1].y * mu * f.w;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (c0 + k < clo || c0 + k >= chi) t[k] = -INFINITY;
#pragma unroll
            for (int k = 0; k < 16; ++k) t[k] = warp_top(t[k]);
            if (lane == 0) {
#pragma unroll
              for (int k = 0; k < 16; k += 4)
                *reinterpret_cast<float4*>(&sm.red[quarter][cb + c0 + k]) = make_float4(t[k], t[k + 1], t[k + 2], t[k + 3]);
            }
          }
          softmax_sync<COLS>();
          bool seen = false;
          if (tid < COLS) {                      // the column's new max
            const float t = fmaxf(fmaxf(sm.red[0][tid], sm.red[1][tid]), fmaxf(sm.red[2][tid], sm.red[3][tid]));
            seen = t != -INFINITY;
            // with one column every one that has grown moves, as the event is what costs;
            // one that had seen nothing takes its first max, whatever its sign, and has no
            // sum or O to correct
            const float old = sm.neg_m[tid];
            const bool had = old != -kNoMax;
            const float now = (had ? t + old > 1.0f : seen) ? -t : old;
            sm.neg_m[tid] = now;
            sm.corr[tid] = had ? ex2(now - old) : 1.0f;
            const uint32_t m = __ballot_sync(COLS < 32 ? 0xFFFFu : 0xFFFFFFFFu, now != old);
            if (lane == 0) sm.moved[warp] = m;
          }
          const bool was_fresh = fresh;
          fresh = !softmax_sync_or<COLS>(seen) && fresh;   // the new maxima are visible
          moved = true;
          if (was_fresh) continue;
#pragma unroll
          for (int k = 0; k < kCols; k += 4) {
            const float4 f = al[k / 4];
            lpart[k / 2] = make_float2(lpart[k / 2].x * f.x, lpart[k / 2].y * f.y);
            lpart[k / 2 + 1] = make_float2(lpart[k / 2 + 1].x * f.z, lpart[k / 2 + 1].y * f.w);
          }
#pragma unroll 1
          for (int j = 0; j < 2 * (kCols / 16); ++j) {   // 16 columns of two chunks
            const int c0 = 16 * (j >> 1);
            if (!((sm.moved[(cb + c0) / 32] >> ((cb + c0) & 31)) & 0xFFFFu)) continue;
            const uint32_t ta = lane_off + 128 * (j & 1) + cb + c0;
            float2 v[2][8];
            tmem_ld16_pairs(ta, v[0]);
            tmem_ld16_pairs(ta + 64, v[1]);
            tmem_ld_wait();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t u[16];
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                const float4 f = al[(c0 + k) / 4];
                asm volatile("" : "+f"(v[h][k / 2].x), "+f"(v[h][k / 2].y), "+f"(v[h][k / 2 + 1].x),
                             "+f"(v[h][k / 2 + 1].y));   // not before the wait
                u[k] = __float_as_uint(v[h][k / 2].x * f.x);
                u[k + 1] = __float_as_uint(v[h][k / 2].y * f.y);
                u[k + 2] = __float_as_uint(v[h][k / 2 + 1].x * f.z);
                u[k + 3] = __float_as_uint(v[h][k / 2 + 1].y * f.w);
              }
              tmem_st16(ta + 64 * h, u);
            }
          }
          tmem_st_wait();
        }
        tc_fence_before();
        warp_arrive(&sm.s_free[i & 1], lane);
        uint32_t packed[kCols / 2];
#pragma unroll
        for (int k = 0; k < kCols / 2; ++k) {
          float2 p = make_float2(ex2(x[k].x), ex2(x[k].y));
          lpart[k] = add2(lpart[k], p);
          if (!plain) p = make_float2(p.x * fmaxf(mu, 0.0f), p.y * fmaxf(mu, 0.0f));   // of NaN: 0
          const __half2 hv = __floats2half2_rn(p.x, p.y);
          packed[k] = *reinterpret_cast<const uint32_t*>(&hv);
        }
        // P of the tile before is used up.  A wait that runs out here raises the abort
        // flag, and the next barrier of the role ends it.
        (void)wait(&sm.p_free, (i & 1) ^ 1);
        __syncwarp();
        uint8_t* prow = sm.p + (mykey >> 3) * 1024;
#pragma unroll
        for (int k = 0; k < kCols / 8; ++k)
          *reinterpret_cast<uint4*>(prow + swz128(mykey & 7, cb / 8 + k)) =
              make_uint4(packed[4 * k], packed[4 * k + 1], packed[4 * k + 2], packed[4 * k + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&sm.p_full, lane);
      }
      // ---- the columns' sums
#pragma unroll
      for (int n = 0; n < kCols; n += 16) {
        float t[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) t[k] = (k & 1) ? lpart[(n + k) / 2].y : lpart[(n + k) / 2].x;
        const float sum = warp_reduce_many<16, false>(t, lane);
        if ((lane & 1) == 0) sm.red[quarter][cb + n + (lane >> 1)] = sum;
      }
      softmax_sync<COLS>();
      if (tid < COLS) {
        const float l = (sm.red[0][tid] + sm.red[1][tid]) + (sm.red[2][tid] + sm.red[3][tid]);
        const float m = l == 0.0f ? kNoMax : -sm.neg_m[tid];
        sm.corr[tid] = l == 0.0f ? 0.0f : 1.0f / l;
        if (tid < cols) {
          if (!whole) {
            a.part_ml[(size_t)slot * 2 * COLS + tid] = m;
            a.part_ml[(size_t)slot * 2 * COLS + COLS + tid] = l;
          } else if (a.lse) {
            a.lse[(size_t)w.gr.r0 * a.H + tid] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
          }
        }
      }
      softmax_sync<COLS>();
      prev_r0 = w.gr.r0;
      prev_cols = cols;
      prev_slot = slot;
    }
    return true;
  }
};

template <int COLS>
__global__ void __launch_bounds__(kThreads, 1) k_dense_attn(const __grid_constant__ DenseArgs a) {
  // addressed through the declared array, so that accesses compile to shared-memory
  // instructions; its 1024-byte alignment is what the 128-byte swizzle needs
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  using S = Smem<COLS>;
  S& sm = *reinterpret_cast<S*>(smem_raw);
  // the warp's number from one lane: known to be the same in all of them
  const int tid = threadIdx.x, lane = lane_id(), warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  const int G = COLS / a.H;
  pdl_trigger();
  if (smem_u32(smem_raw) & 1023u) {              // not where it was declared to be: nothing runs
    if (tid == 0) {
      raise_flag(a.status, CSA_FLAG_TIMEOUT);
      a.rec[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    return;
  }
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i], 4);
      mbar_init(&sm.k_free[i], 1);
      mbar_init(&sm.s_full[i], 2);
      mbar_init(&sm.s_free[i], kSoftmaxUsed<COLS>);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.v_full[i], 4);
      mbar_init(&sm.v_free[i], 1);
    }
    mbar_init(&sm.p_full, kSoftmaxUsed<COLS>);
    mbar_init(&sm.p_free, 1);
    mbar_init(&sm.q_raw, 32);
    mbar_init(&sm.q_full, kSoftmaxUsed<COLS>);
    mbar_init(&sm.q_free, 1);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_free, kSoftmaxUsed<COLS>);
    mbar_init(&sm.drain, 2);
    fence_barrier_init();
    sm.abort = 0;
    sm.tile_now = 0;
  }
  if (a.rope_cos)                                // the low parts' image is zero where nothing is rotated
    for (int i = tid; i < COLS * 16; i += kThreads) reinterpret_cast<uint4*>(sm.q_lo)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (warp == kMmaWarp) tmem_alloc(&sm.tmem_base, 512);
  const Share sh = find_share(a, G, *reinterpret_cast<ShareScratch*>(sm.p));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // all 512 columns are this CTA's, so they start at address 0
  // registers: 640 x 96 at launch = 256 x 128 + 256 x 96 + 128 x 32
  if (warp < kDequantWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    Dequant<COLS> d{a, sm, lane, warp >> 2, lane & 3, 32 * (warp & 3) + (lane >> 2),
                    kTmemK + 64 * (warp >> 2) + ((uint32_t)(32 * (warp & 3)) << 16)};
    d.run(sh, G);
  } else if (warp < kMmaWarp) {
    const int v = warp - kDequantWarps;
    if (v < kSoftmaxUsed<COLS>) {
      int4 rec = make_int4(-1, 0, 0, 0);
      Softmax<COLS> s{a, sm, lane, v};
      const bool ok = s.run(sh, G, rec);
      if (v == 0 && lane == 0) a.rec[blockIdx.x] = ok ? rec : make_int4(-1, 0, 0, 0);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp < kMmaWarp + 2) {
      Issue<COLS> m{a, sm};
      if (warp == kMmaWarp) m.run_scores(sh, G);
      else m.run_values(sh, G);
      // nothing of this CTA's is in flight when its memory is given back
      __syncwarp();
      if (elect_one()) tc_commit(&sm.drain);
      __syncwarp();
      if (!mbar_wait(&sm.drain, 0)) sm.abort = 1;
    } else if (warp == kMmaWarp + 2) {
      prefetch_tiles<COLS>(a, sm, sh, G);
    } else {
      fetch_queries<COLS>(a, sm, sh, G);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm.abort) raise_flag(a.status, CSA_FLAG_TIMEOUT);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(sm.tmem_base, 512);
  }
}

// Joins the parts of the groups cut between CTAs:
// O = sum_q 2^(m_q - M) O_q / sum_q 2^(m_q - M) l_q.  One wave of CTAs, each of one
// column (a CTA for every cut and column spent most of its time on being launched and
// finding nothing to do).  Thread = 4 dims.  A cut of few parts is the work of a
// quarter of a CTA, which needs no barrier; of one of many parts each quarter sums
// every fourth, and the four sums are joined in a fixed order.  129 parts of 64
// columns (17 MB) take about 9 us, 25 with a CTA for every cut and column; bound by
// the trips to L2, eight parts in flight a thread.
constexpr int kMergeSplit = 4, kMergeLoads = 8, kMergeThreads = 128 * kMergeSplit;
__device__ __forceinline__ void merge_store(const DenseArgs& a, size_t col, int d, float M, float L, float4 o) {
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv, o.y * inv), y = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  uint2 st;
  st.x = *reinterpret_cast<const uint32_t*>(&x);
  st.y = *reinterpret_cast<const uint32_t*>(&y);
  *(reinterpret_cast<uint2*>(a.out + col * D) + d) = st;
  if (a.lse && d == 0) a.lse[col] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
}
__device__ __forceinline__ void add_scaled(float4& o, float w, const float4& v) {
  o.x += w * v.x;
  o.y += w * v.y;
  o.z += w * v.z;
  o.w += w * v.w;
}
__global__ void __launch_bounds__(kMergeThreads, 2) k_dense_merge(DenseArgs a, int cols_max, int num_recs) {
  __shared__ int4 s_rec[kMergeThreads];          // cuts of few parts from the front, of many from the back
  __shared__ int2 s_count[kMergeThreads / 32];   // of each kind, by warp
  __shared__ float s_w[kMergeThreads];           // a group has at most one part per SM
  __shared__ float s_m[kMergeThreads / 32], s_l[kMergeThreads / 32];
  __shared__ float4 s_o[kMergeSplit - 1][128];
  const int tid = threadIdx.x, k = tid >> 7, d = tid & 127, c = blockIdx.y;
  pdl_wait();
  // the cuts of this column, in the same order in every CTA that shares them out
  const int4 mine = tid < num_recs ? __ldcg(a.rec + tid) : make_int4(-1, 0, 0, 0);
  const bool used = mine.x >= 0 && c < mine.y * a.H, is_few = mine.w - mine.z < kMergeLoads;
  const uint32_t b_few = __ballot_sync(0xFFFFFFFFu, used && is_few), b_many = __ballot_sync(0xFFFFFFFFu, used && !is_few);
  if (lane_id() == 0) s_count[tid >> 5] = make_int2(__popc(b_few), __popc(b_many));
  __syncthreads();
  int few = 0, many = 0, at_few = 0, at_many = 0;
#pragma unroll
  for (int w = 0; w < kMergeThreads / 32; ++w) {
    if (w == tid >> 5) {
      at_few = few;
      at_many = many;
    }
    few += s_count[w].x;
    many += s_count[w].y;
  }
  const uint32_t below = (1u << lane_id()) - 1u;
  if (used) s_rec[is_few ? at_few + __popc(b_few & below) : kMergeThreads - 1 - at_many - __popc(b_many & below)] = mine;
  __syncthreads();
  // a part's slot: 2 c0 + 1 of the first, then 2 (c0 + 1), 2 (c0 + 2), ...
  auto slot = [](const int4& rec, int q) { return (size_t)(q == 0 ? 2 * rec.z + 1 : 2 * (rec.z + q)); };
  const float* part = a.part + (size_t)c * D + 4 * d;
#pragma unroll 1
  for (int i = blockIdx.x * kMergeSplit + k; i < few; i += gridDim.x * kMergeSplit) {
    const int4 rec = s_rec[i];
    const int n = rec.w - rec.z + 1;
    float4 v[kMergeLoads];
    float m[kMergeLoads], l[kMergeLoads], M = kNoMax;
#pragma unroll
    for (int q = 0; q < kMergeLoads; ++q) {
      v[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      m[q] = kNoMax;
      l[q] = 0.0f;
      if (q < n) {
        const float* ml = a.part_ml + slot(rec, q) * 2 * cols_max + c;
        m[q] = __ldcg(ml);
        l[q] = __ldcg(ml + cols_max);
        v[q] = __ldcg(reinterpret_cast<const float4*>(part + slot(rec, q) * cols_max * D));
      }
    }
#pragma unroll
    for (int q = 0; q < kMergeLoads; ++q) M = fmaxf(M, m[q]);
    float L = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int q = 0; q < kMergeLoads; ++q) {
      if (q < n) {
        const float w = ex2(m[q] - M);
        L += w * l[q];
        add_scaled(o, w, v[q]);
      }
    }
    merge_store(a, (size_t)rec.x * a.H + c, d, M, L, o);
  }
#pragma unroll 1
  for (int i = blockIdx.x; i < many; i += gridDim.x) {
    const int4 rec = s_rec[kMergeThreads - 1 - i];
    const int n = rec.w - rec.z + 1;
    float m = kNoMax, l = 0.0f;
    if (tid < n) {
      const float* ml = a.part_ml + slot(rec, tid) * 2 * cols_max + c;
      m = __ldcg(ml);
      l = __ldcg(ml + cols_max);
    }
    float4 v[kMergeLoads];
    auto load = [&](int q0) {
#pragma unroll
      for (int j = 0; j < kMergeLoads; ++j) {
        const int q = q0 + j * kMergeSplit;
        v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (q < n) v[j] = __ldcg(reinterpret_cast<const float4*>(part + slot(rec, q) * cols_max * D));
      }
    };
    load(k);                                     // before the weights are known
    const float m_warp = warp_top(m);
    if (lane_id() == 0) s_m[tid >> 5] = m_warp;
    __syncthreads();
    float M = s_m[0];
#pragma unroll
    for (int w = 1; w < kMergeThreads / 32; ++w) M = fmaxf(M, s_m[w]);
    const float weight = ex2(m - M);
    s_w[tid] = tid < n ? weight : 0.0f;
    float l_warp = weight * l;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l_warp += __shfl_xor_sync(0xFFFFFFFFu, l_warp, x);
    if (lane_id() == 0) s_l[tid >> 5] = l_warp;
    __syncthreads();
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int q0 = k; q0 < n; q0 += kMergeLoads * kMergeSplit) {
      if (q0 != k) load(q0);
#pragma unroll
      for (int j = 0; j < kMergeLoads; ++j) {
        const int q = q0 + j * kMergeSplit;
        if (q < n) add_scaled(o, s_w[q], v[j]);
      }
    }
    if (k > 0) s_o[k - 1][d] = o;
    __syncthreads();
    if (k == 0) {
      float L = s_l[0];
#pragma unroll
      for (int w = 1; w < kMergeThreads / 32; ++w) L += s_l[w];
#pragma unroll
      for (int j = 1; j < kMergeSplit; ++j) add_scaled(o, 1.0f, s_o[j - 1][d]);
      merge_store(a, (size_t)rec.x * a.H + c, d, M, L, o);
    }
    __syncthreads();                             // the next cut uses the same places
  }
}

constexpr size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Columns of a group: rows of a request taken together, up to 64.
int group_cols(int rows, int H) {
  int c = 16;
  while (c < 64 && c < (int64_t)rows * H) c *= 2;
  return std::max(c, H);
}

// CTAs: one per SM, no more than the tiles that the host's bounds allow.
int dense_grid(int num_rows, int max_entries, int num_sms) {
  const int64_t tiles = ((int64_t)max_entries + kTileKeys - 1) / kTileKeys + 2;   // a group's window: at most two
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(num_sms, kMergeThreads), tiles * num_rows));
}

template <int COLS>
cudaError_t launch_cols(DenseArgs a, int grid, int num_sms, cudaStream_t stream) {
  static_assert(sizeof(Smem<COLS>) <= 232448, "shared memory of one CTA");
  const size_t smem = sizeof(Smem<COLS>);
  cudaError_t e = cudaFuncSetAttribute(k_dense_attn<COLS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_kernel(Order::kStream, k_dense_attn<COLS>, dim3(grid), dim3(kThreads), smem, stream, a);
  if (e != cudaSuccess || grid == 1) return e;
  // two CTAs fit an SM, and a grid has a CTA per SM at most
  const dim3 merge(std::max(1, 2 * num_sms / COLS), COLS);
  return launch_kernel(Order::kChained, k_dense_merge, merge, dim3(kMergeThreads), 0, stream, a, COLS, grid - 1);
}

}  // namespace

size_t dense_ws_bytes(int32_t num_rows, int32_t max_entries, int32_t H, int num_sms) {
  const size_t grid = dense_grid(num_rows, max_entries, num_sms), cols = group_cols(num_rows, H);
  return up256(grid * sizeof(int4)) + up256(2 * grid * 2 * cols * sizeof(float)) + 2 * grid * cols * D * sizeof(float);
}

cudaError_t launch_dense_attn(DenseArgs a, void* ws, int num_sms, cudaStream_t stream) {
  const int grid = dense_grid(a.num_rows, a.max_entries, num_sms);
  const int cols = group_cols(std::min(a.num_rows, a.max_rows_per_req), a.H);
  uint8_t* p = static_cast<uint8_t*>(ws);
  a.rec = reinterpret_cast<int4*>(p);
  p += up256((size_t)grid * sizeof(int4));
  a.part_ml = reinterpret_cast<float*>(p);
  p += up256((size_t)2 * grid * 2 * cols * sizeof(float));
  a.part = reinterpret_cast<float*>(p);
  switch (cols) {
    case 16: return launch_cols<16>(a, grid, num_sms, stream);
    case 32: return launch_cols<32>(a, grid, num_sms, stream);
    default: return launch_cols<64>(a, grid, num_sms, stream);
  }
}

}  // namespace csa
