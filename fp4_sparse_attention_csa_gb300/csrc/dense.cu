// csa_dense_attn: MQA softmax attention of each row's heads over every visible
// FP4 main-KV entry and the FP8 local window, for single tokens, verify rows and
// whole prompt chunks.
//
// Mathematics.  A group is up to G = COLS / H rows of one request at consecutive
// positions; its COLS = G * H columns are independent queries that share keys.
// Its keys are one list: the W window tokens of the group's rows, then the n
// entries that its last row sees; column c (row i) attends to the window
// positions in [max(0, t_i - 127), t_i] and the entries below (t_i + 1) / P.
// Per 128-key tile: S^T = K Q^T (M = 128 keys, N = COLS), p = 2^(s - m) with a
// running max m per column, O^T += V^T P^T (M = 128 dims x 4, N = COLS); keys and
// values are the same fp16 tile, read K-major by the first product and MN-major
// by the second.  Entries are exact in fp16 (e2m1 x E4M3); a window token is its
// E4M3 codes times 2^e, e in [-14, 7], also exact, and the rest of its scale, mu,
// multiplies its logits and p.  A query is scaled by a power of two so that its
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
// Pipeline.  One CTA per SM, three roles that meet only at mbarriers:
//   8 dequantising warps (two warpgroups, 128 dims of a tile at a time each),
//   4 softmax warps (32 keys x all columns each), also queries and output,
//   2 warps that issue the MMAs, one for each product, and one that prefetches
//   entries into L2.
// The tensor pipe takes 48 clocks per M128 K16 MMA up to N = 64 (64 at N = 128),
// so a tile costs at least 64 x 48 = 3072; the roles have to hide behind that.
// Shared memory holds Q (64 KB), P and one fp16 tile (128 KB), not two.  So the
// first product does not read it: the dequantising warps write each 128-dim chunk
// to tensor memory (two 64-column slots) as its A operand, and S of tile t + 1 is
// computed while tile t still occupies shared memory, during its softmax.  Of a
// warpgroup's two chunks the first waits in registers and the second in its slot
// until the second product has used tile t's.  That also takes 4 of the 6 KB per
// MMA off the shared-memory port, which the second product alone fills.
#include <algorithm>

#include "attn_device.cuh"
#include "csa_internal.h"

namespace csa {

namespace {

constexpr int kThreads = 512;                    // 8 dequantising, 4 softmax, 2 MMA, 1 prefetching warp (and 1 idle)
constexpr int kTileKeys = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running max moves when a logit exceeds it by this (log2 units): p <= 2^14,
// times a window key's mu < 2, stays inside fp16, and a column rarely moves again
// after its first tile (at 2^8 a column of widely spread logits still moved in
// most early tiles).
constexpr float kRescaleLog2 = 14.0f;

// ---- the list of work ----------------------------------------------------------------
struct Group {
  int r0, g, b, p0;                              // first row, rows, request, first position
  int W, wlo;                                    // window keys and the first one's position
  int keys, tiles;                               // tiles 0: the rows see nothing (or are invalid)
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
    q.W = q.wlo = q.keys = q.tiles = 0;
    return q;
  }
  while (q.g < G && r + q.g < a.num_rows && row_continues(a, r + q.g)) ++q.g;
  const int last = q.p0 + q.g - 1;
  q.wlo = max(0, q.p0 - (WIN - 1));
  q.W = a.win_codes ? last - q.wlo + 1 : 0;
  q.keys = q.W + entries_at(a, last);
  q.tiles = (q.keys + kTileKeys - 1) / kTileKeys;
  return q;
}
// A group of no tiles still takes one unit: its rows are written out empty.
__device__ __forceinline__ int group_units(const Group& q) { return max(1, q.tiles); }

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
    for (int r = r_lo; r < r_hi; ++r)
      if (!row_continues(a, r)) start = r;
    const int upto = block_scan<true>(start, s.starts);
    run = __shfl_up_sync(0xFFFFFFFFu, upto, 1);
    if (lane_id() == 31) s.run[warp_id()] = upto;
    __syncthreads();
    if (lane_id() == 0) run = tid > 0 ? s.run[warp_id() - 1] : -1;
  }
  // visits the groups that begin in this thread's rows: f(row, units) until it is true
  auto groups = [&](auto f) {
    int from = run;
    for (int r = r_lo; r < r_hi; ++r) {
      if (G > 1 && row_continues(a, r)) {
        if ((r - from) % G != 0) continue;
      } else {
        from = r;
      }
      if (f(r, group_units(group_at(a, r, G)))) break;
    }
  };
  long long sum = 0;
  groups([&](int, int n) {
    sum += n;
    return false;
  });
  const long long upto = block_scan<false>(sum, s.sums);
  if (tid == kThreads - 1) s.total = upto;
  __syncthreads();
  const long long total = s.total, per = (total + gridDim.x - 1) / gridDim.x;
  const long long lo = min(total, (long long)blockIdx.x * per), hi = min(total, lo + per);
  long long u = upto - sum;
  if (lo < hi && u <= lo && lo < upto) {         // exactly one thread
    groups([&](int r, int n) {
      if (lo >= u + n) {
        u += n;
        return false;
      }
      s.out.row = r;
      s.out.t0 = (int)(lo - u);
      return true;
    });
  }
  __syncthreads();
  Share h = s.out;
  h.units = (int)(hi - lo);                      // a share is far below 2^31 tiles
  h.per = (int)per;
  return h;
}

// ---- shared memory ---------------------------------------------------------------------
constexpr int kDequantWarps = 8, kSoftmaxWarps = 4;
constexpr int kMmaWarp = kDequantWarps + kSoftmaxWarps;
constexpr float kNoMax = -3e38f;                 // running max of a column that has seen nothing

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
  uint64_t p_full, p_free, q_full, o_full, o_free, drain;
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
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool softmax_sync_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v)
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
  __device__ __forceinline__ bool whole() const { return t0 == 0 && left >= group_units(gr); }
};

// ---- dequantising ------------------------------------------------------------------------
// A warp holds 32 keys (its tensor-memory quarter); its warpgroup takes chunks 2 wg
// and 2 wg + 1, 128 dims each.  Lane 4r + q holds rows r, r + 8, r + 16, r + 24, of
// each chunk the 32 dims from 32 q (16 bytes: four words of 8 dims, two scales).
// Four dims sit in two neighbouring columns of tensor memory; S sums over dims in
// any order, and Q is laid out to match (q_place).  In shared memory lanes q >= 2
// put word i where word i ^ 2 belongs, so that a quarter-warp's 16-byte stores hit
// distinct banks; that permutes rows of O^T, and write_out undoes it.
struct Raw {
  uint4 w[2][4];                                 // [chunk][row]
  uint32_t sc[4];                                // [row]: the lane's quarter of the 16 scales of both chunks
};

// Where the 4 dims from d (a multiple of 4) of a chunk sit: the 16-dim step of the
// product and the place, of four, in it.
__device__ __forceinline__ void q_place(int d, int& step, int& place) {
  place = d >> 5;
  step = (d >> 2) & 7;
}

__device__ __forceinline__ uint32_t ldg_nc_u32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// A thread's four rows lie within 32 consecutive keys, so in one page or two
// neighbouring ones.
struct Pages {
  int lo, hi;                                    // table words of the first row's page and the last row's
};
// e: the first row's entry; past the n entries, or a window key: -1.  Nothing looks
// at the words until their bytes are fetched, a tile later.
__device__ __forceinline__ Pages find_pages(const int32_t* row, int e, int n) {
  Pages p{-1, -1};
  if (e + 24 >= 0 && e < n) {
    p.lo = __ldg(row + (max(e, 0) >> 6));
    p.hi = __ldg(row + (min(e + 24, n - 1) >> 6));
  }
  return p;
}
// The page of row s, -1 when there is nothing to read (a page outside the pool
// among them).
__device__ __forceinline__ int page_of(const DenseArgs& a, const Pages& p, int e, int s, int n) {
  const int x = e + 8 * s;
  const int pg = (x >> 6) == (max(e, 0) >> 6) ? p.lo : p.hi;
  return (x >= 0 && x < n && (uint32_t)pg < (uint32_t)a.num_pages) ? pg : -1;
}

// Row s's bytes of one chunk (h) or its scales.  A row with nothing to read takes
// page 0's codes, and scales of zero.
__device__ __forceinline__ const uint8_t* row_data(const DenseArgs& a, int pg, int slot, int chunk, int q) {
  return a.kv_pool + (size_t)max(pg, 0) * KV_PAGE + slot * 256 + chunk * 64 + 16 * q;
}
__device__ __forceinline__ uint32_t row_scales(const DenseArgs& a, int pg, int slot, int wg, int q) {
  return pg >= 0 ? ldg_nc_u32(a.kv_pool + (size_t)pg * KV_PAGE + KV_SCALE_OFF + slot * 32 + wg * 16 + 4 * q) : 0u;
}
// Where the thread's four rows of a tile of entries lie.
struct Rows {
  const uint8_t* data[2];                        // row 0's bytes, were it in the first or the second page
  const uint8_t* scales[2];
  int slot0;
  uint32_t valid;                                // bit s: row s is there to read
  __device__ __forceinline__ void set(const DenseArgs& a, const Pages& p, int e, int n, int wg, int q) {
    slot0 = e & (PAGE - 1);
    const bool ok[2] = {(uint32_t)p.lo < (uint32_t)a.num_pages, (uint32_t)p.hi < (uint32_t)a.num_pages};
    valid = 0;
#pragma unroll
    for (int s = 0; s < 4; ++s) valid |= (uint32_t)(e + 8 * s < n && ok[slot0 + 8 * s >= PAGE]) << s;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint8_t* page = a.kv_pool + (size_t)(ok[k] ? (k ? p.hi : p.lo) : 0) * KV_PAGE;
      data[k] = page + (slot0 - k * PAGE) * 256 + wg * 128 + 16 * q;
      scales[k] = page + KV_SCALE_OFF + (slot0 - k * PAGE) * 32 + wg * 16 + 4 * q;
    }
  }
  // chunk h's bytes, and with the second the scales.  A row with nothing to read
  // takes some page's codes, and scales of zero.
  __device__ __forceinline__ void fetch(Raw& x, int h) const {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = slot0 + 8 * s >= PAGE;
      x.w[h][s] = ldg_nc_v4((k ? data[1] : data[0]) + s * 2048 + h * 64);
      if (h == 1) {
        x.sc[s] = 0u;
        if ((valid >> s) & 1u) x.sc[s] = ldg_nc_u32((k ? scales[1] : scales[0]) + s * 256);
      }
    }
  }
};
// The lane's four scales, chunk 0's two in the low half, from its group's quarters.
__device__ __forceinline__ uint32_t own_scales(uint32_t sc, int q) {
  const uint32_t lo = __shfl_sync(0xFFFFFFFFu, sc, q >> 1, 4), hi = __shfl_sync(0xFFFFFFFFu, sc, 2 + (q >> 1), 4);
  return __byte_perm(lo, hi, (q & 1) ? 0x7632 : 0x5410);
}

// h: tensor-memory register order of two rows (r, r + 8): pair k (two dims) of row j
// of the thread's 16 pairs.
__device__ __forceinline__ constexpr int h_at(int j, int k) { return 4 * (k / 2) + 2 * j + k % 2; }

// The 16 pairs of an entry row's chunk; sc: its two scales.
__device__ __forceinline__ void entry_to_f16(uint4 v, uint32_t sc, uint32_t (&o)[16]) {
  const uint32_t sp = e4m3x2_to_f16((uint16_t)sc);
  const __half2 hs0 = __low2half2(*reinterpret_cast<const __half2*>(&sp));
  const __half2 hs1 = __high2half2(*reinterpret_cast<const __half2*>(&sp));
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t f[4];
    e2m1x8_to_f16(w[i], f);
#pragma unroll
    for (int g = 0; g < 4; ++g) o[4 * i + g] = hmul2_u32(f[g], i < 2 ? hs0 : hs1);
  }
}

// Two words (16 dims, one scale, in both halves) of it.
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
  // of its scale is mu.  ki: the thread's first key.
  __device__ __noinline__ static bool near_chunk(const DenseArgs& a, S& sm, bool values, int lane, int wg, int q,
                                                 int key0, uint32_t tslot, int h, uint32_t tile, int ki, int W, int n,
                                                 int wlo, int b, Pages p) {
    const int c = 2 * wg + h, e = ki - W;
    const bool turn = c == 3 && q >= 2 && a.rope_cos != nullptr;
    uint4 u[4], v[4];                            // 32 window codes, or an entry's 16 bytes in u
    uint32_t sc[4];                              // a window token's scale, or an entry's scales
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u[s] = v[s] = make_uint4(0u, 0u, 0u, 0u);
      const int slot = (e + 8 * s) & (PAGE - 1), pg = page_of(a, p, e, s, n);
      sc[s] = row_scales(a, pg, slot, wg, q);
      if (ki + 8 * s < W) {
        const size_t ring = (size_t)b * a.win_cap + (size_t)((wlo + ki + 8 * s) % a.win_cap);
        const uint8_t* src = a.win_codes + ring * D + c * 128 + 32 * q;
        u[s] = ldg_nc_v4(src);
        v[s] = ldg_nc_v4(src + 16);
        sc[s] = __float_as_uint(__ldg(a.win_scale + ring));
      } else if (pg >= 0) {
        u[s] = ldg_nc_v4(row_data(a, pg, slot, c, q));
      }
    }
    auto row = [&](int s, uint32_t (&o)[16]) {
      const uint32_t own = own_scales(sc[s], q) >> (16 * h);   // by all lanes
      float mu = page_of(a, p, e, s, n) >= 0 ? 1.0f : -1.0f;
      if (ki + 8 * s < W) {
        const float ws = __uint_as_float(sc[s]);
        const int ex = ws > 0.0f ? min(7, max(-14, (int)(__float_as_uint(ws) >> 23) - 127)) : -14;
        const float pw = pow2(ex);
        mu = ws * pow2(-ex);
        const __half2 hp = __float2half2_rn(pw);
        const uint32_t cw[8] = {u[s].x, u[s].y, u[s].z, u[s].w, v[s].x, v[s].y, v[s].z, v[s].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t f[2];
          e4m3x4_to_f16(cw[i], f);
          o[2 * i] = hmul2_u32(f[0], hp);
          o[2 * i + 1] = hmul2_u32(f[1], hp);
        }
        if (turn) {                              // dims 448 + 32 (q - 2): the halves are q = 2 and 3
          const int at = wlo + ki + 8 * s;
          const size_t ring = (size_t)b * a.win_cap + (size_t)(at % a.win_cap);
          const uint8_t* src = a.win_codes + ring * D + c * 128 + 32 * (5 - q);
          uint32_t t[16];
          rotate_window(a.rope_cos + (size_t)at * 32, a.rope_sin + (size_t)at * 32, q == 2, pw, u[s], v[s],
                        ldg_nc_v4(src), ldg_nc_v4(src + 16), t);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = t[k];
        }
      } else {
        entry_to_f16(u[s], own, o);
      }
      if (!values && c == 0 && q == 0) {
        sm.mu[tile & 1][key0 + 8 * s] = mu;
        if (mu < 0.0f && e + 8 * s < n) raise_flag(a.status, CSA_FLAG_PAGE_OOB);
      }
      __syncwarp();
    };
    if (!values && c == 0 && lane == 0) sm.odd[tile & 1][key0 >> 5] = 1u;
    const bool ok = wait_or_abort(values ? &sm.v_free[c] : &sm.k_free[wg], values ? (tile & 1) ^ 1 : h ^ 1,
                                  a.wait_budget, &sm.abort);
    if (!__all_sync(0xFFFFFFFFu, ok)) return false;
    tc_fence_after();
#pragma unroll
    for (int pair = 0; pair < 2; ++pair) {
      uint32_t o[2][16];
      row(2 * pair, o[0]);
      row(2 * pair + 1, o[1]);
      if (!values) {
        uint32_t t[32];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          t[h_at(0, k)] = o[0][k];
          t[h_at(1, k)] = o[1][k];
        }
        tmem_st_16x64(tslot + ((uint32_t)(16 * pair) << 16), t);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(value_at(sm, c, key0, 2 * pair + j, q, i)) =
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
      const int W = w.gr.W, n = w.gr.keys - W;
      int left = w.t_end - w.t;                  // tiles of the segment
      int ki = w.t * kTileKeys + key0;           // the thread's first key
#pragma unroll 1
      for (; left > 0 && ki - key0 < W; --left, ki += kTileKeys, ++tile) {
        const Pages p = find_pages(row, ki - W, n);
#pragma unroll 1
        for (int part = 0; part < 4; ++part)     // both chunks for the first product, then for the second
          if (!near_chunk(a, sm, part >= 2, lane, wg, q, key0, tslot, part & 1, tile, ki, W, n, w.gr.wlo, w.gr.b, p))
            return;
      }
      if (left <= 0) continue;
      int e = ki - W;                            // the first row's entry
      Raw x;
      Rows at;
      Pages next = find_pages(row, e, n);
      at.set(a, next, e, n, wg, q);
      at.fetch(x, 0);
      at.fetch(x, 1);
#pragma unroll 1
      for (; left > 0; --left, ++tile) {
        next = find_pages(row, e + kTileKeys, n);
        if (wg == 0) {                           // keys past the last one and in bad pages are left out
          const bool odd = __any_sync(0xFFFFFFFFu, at.valid != 15u);
          if (lane == 0) sm.odd[tile & 1][key0 >> 5] = odd;
          if (odd && q == 0) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const bool in = (at.valid >> s) & 1u;
              sm.mu[tile & 1][key0 + 8 * s] = in ? 1.0f : -1.0f;
              if (!in && e + 8 * s < n) raise_flag(a.status, CSA_FLAG_PAGE_OOB);
            }
          }
        }
        uint32_t sc[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) sc[s] = own_scales(x.sc[s], q);
        // ---- the first product's A operand: one chunk, whose values stay in registers,
        // then the other, which stays in the slot
        if (!wait(&sm.k_free[wg], 1)) return;
        tc_fence_after();
        uint32_t t[2][32];
#pragma unroll
        for (int pair = 0; pair < 2; ++pair) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t o[16];
            entry_to_f16(x.w[0][2 * pair + j], sc[2 * pair + j], o);
#pragma unroll
            for (int k = 0; k < 16; ++k) t[pair][h_at(j, k)] = o[k];
          }
          tmem_st_16x64(tslot + ((uint32_t)(16 * pair) << 16), t[pair]);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&sm.k_full[wg], lane);
        if (!wait(&sm.k_free[wg], 0)) return;
        tc_fence_after();
#pragma unroll
        for (int pair = 0; pair < 2; ++pair) {
#pragma unroll
          for (int half = 0; half < 2; ++half) { // 32 columns: words 2 half and 2 half + 1 of two rows
            uint32_t u[16];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint4 v = x.w[1][2 * pair + j];
              const uint32_t sp = e4m3x2_to_f16((uint16_t)(sc[2 * pair + j] >> 16));
              const __half2 hs = *reinterpret_cast<const __half2*>(&sp);
              uint32_t o[8];
              words_to_f16(half ? v.z : v.x, half ? v.w : v.y, half ? __high2half2(hs) : __low2half2(hs), o);
#pragma unroll
              for (int k = 0; k < 8; ++k) u[h_at(j, k)] = o[k];
            }
            tmem_st_16x32(tslot + ((uint32_t)(16 * pair) << 16) + 32 * half, u);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&sm.k_full[wg], lane);
        // ---- the second product's, as the previous tile's chunks are used up; the next
        // tile's bytes are fetched meanwhile
        e += kTileKeys;
        asm volatile("" : "+r"(next.lo), "+r"(next.hi));   // not looked at before here
        at.set(a, next, e, n, wg, q);            // past the last tile: nothing to read
        if (!wait(&sm.v_free[2 * wg], (tile & 1) ^ 1)) return;
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t* r = t[s / 2] + h_at(s % 2, 4 * i);
            *reinterpret_cast<uint4*>(value_at(sm, 2 * wg, key0, s, q, i)) = make_uint4(r[0], r[1], r[4], r[5]);
          }
        fence_proxy_async_smem();
        warp_arrive(&sm.v_full[2 * wg], lane);
        at.fetch(x, 0);
        at.fetch(x, 1);
        uint32_t u[4][16];                       // [2 pair + half]
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld_16x32(tslot + ((uint32_t)(16 * (k >> 1)) << 16) + 32 * (k & 1), u[k]);
        tmem_ld_wait();
        if (!wait(&sm.v_free[2 * wg + 1], (tile & 1) ^ 1)) return;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = h_at(j, 4 * i);
              *reinterpret_cast<uint4*>(value_at(sm, 2 * wg + 1, key0, 2 * (k >> 1) + j, q, 2 * (k & 1) + i)) =
                  make_uint4(u[k][r], u[k][r + 1], u[k][r + 4], u[k][r + 5]);
            }
        tc_fence_before();
        fence_proxy_async_smem();
        warp_arrive(&sm.v_full[2 * wg + 1], lane);
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
    const int lo = max(0, w.t * kTileKeys - w.gr.W), hi = min(w.gr.keys, (w.t + 1) * kTileKeys) - w.gr.W;
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
  template <int step>
  __device__ __forceinline__ bool scores(uint32_t i) {
    if (!wait(&sm.k_full[step & 1], step >> 1)) return false;
    const uint64_t dQ = smem_desc(smem_u32(sm.q), 16, 1024, kSwizzle128B);
    const uint64_t dQl = smem_desc(smem_u32(sm.q_lo), 16, 1024, kSwizzle128B);
    constexpr uint32_t id = idesc_f16(128, COLS, 0, 0);
    const uint32_t ts = kTmemS + 64 * (i & 1), ta = kTmemK + 64 * (step & 1);
    constexpr int c = 2 * (step & 1) + (step >> 1);
    tc_fence_after();
    if (elect_one()) {
      const uint64_t dq = dQ + (uint64_t)(c * 2 * (COLS * 8));
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        mma_f16_ts(ts, ta + 8 * ks, dq + (uint64_t)((ks >> 2) * (COLS * 8) + (ks & 3) * 2), id,
                   (ks > 0 || step > 0) ? 1u : 0u);
      if (step == 3 && a.rope_cos) {             // chunk 3 again, by the rotated dims' low parts
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_f16_ts(ts, ta + 8 * ks, dQl + (uint64_t)((ks >> 2) * (COLS * 8) + (ks & 3) * 2), id, 1u);
      }
      tc_commit(&sm.k_free[step & 1]);
      if (step == 3) {
        tc_commit(&sm.s_full[i & 1]);
        mbar_arrive(&sm.s_full[i & 1]);          // orders the tile's mu before its softmax
      }
    }
    __syncwarp();
    return true;
  }
  // step 0..3 of a tile's O^T; first, last: of its segment
  template <int step>
  __device__ __forceinline__ bool values(uint32_t i, bool first, bool last) {
    if (!wait(&sm.v_full[2 * (step & 1) + (step >> 1)], i & 1)) return false;
    const uint64_t dV = smem_desc(smem_u32(sm.k), 16384, 1024, kSwizzle128B);
    const uint64_t dP = smem_desc(smem_u32(sm.p), 8192, 1024, kSwizzle128B);
    constexpr uint32_t id = idesc_f16(128, COLS, 1, 1);
    constexpr int c = 2 * (step & 1) + (step >> 1);
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
      if (!scores<0>(i) || !scores<1>(i) || !scores<2>(i) || !scores<3>(i)) break;
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
      if (!values<0>(i, first, last) || !values<1>(i, first, last) || !values<2>(i, first, last) ||
          !values<3>(i, first, last))
        break;
    }
  }
};

// ---- queries ------------------------------------------------------------------------------
// Columns c0 .. c0 + n - 1, of one row, to shared memory, fp16, by one warp: N at a
// time, the next N in flight meanwhile.
template <int COLS, int N>
__device__ __forceinline__ void load_queries(const DenseArgs& a, Smem<COLS>& sm, const Group& gr, int c0, int n) {
  const int lane = lane_id();
  const bool in = c0 < gr.g * a.H, rope = a.rope_cos != nullptr && in;
  const uint4* src = reinterpret_cast<const uint4*>(a.q + ((size_t)gr.r0 * a.H + c0) * D) + 2 * lane;
  uint4 raw[N][2];
  float cs[16], sn[16];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    raw[j][0] = raw[j][1] = make_uint4(0u, 0u, 0u, 0u);
    if (in) {
      raw[j][0] = __ldg(src + j * (D / 8));
      raw[j][1] = __ldg(src + j * (D / 8) + 1);
    }
  }
  if (rope && lane >= 28) {                      // the row's table entries of this lane's 16 dims
    const size_t at = (size_t)(gr.p0 + c0 / a.H) * 32 + 16 * (lane & 1);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      cs[i] = __ldg(a.rope_cos + at + i);
      sn[i] = __ldg(a.rope_sin + at + i);
    }
  }
#pragma unroll 1
  for (int done = 0; done < n; done += N) {
    float f[N][16];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t w[8] = {raw[j][0].x, raw[j][0].y, raw[j][0].z, raw[j][0].w,
                             raw[j][1].x, raw[j][1].y, raw[j][1].z, raw[j][1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[j][2 * i] = __uint_as_float(w[i] << 16);
        f[j][2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
    if (in && done + N < n) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        raw[j][0] = __ldg(src + (done + N + j) * (D / 8));
        raw[j][1] = __ldg(src + (done + N + j) * (D / 8) + 1);
      }
    }
    if (rope) {                                  // dims 448.. are lanes 28, 29 and 30, 31
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float other = __shfl_xor_sync(0xFFFFFFFFu, f[j][i], 2);
          if (lane >= 28)
            f[j][i] = lane < 30 ? __fsub_rn(__fmul_rn(f[j][i], cs[i]), __fmul_rn(other, sn[i]))
                                : __fadd_rn(__fmul_rn(f[j][i], cs[i]), __fmul_rn(other, sn[i]));
        }
    }
    float big[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      big[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) big[j] = fmaxf(big[j], fabsf(f[j][i]));
    }
#pragma unroll
    for (int j = 0; j < N; ++j) big[j] = warp_top(big[j]);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = c0 + done + j;
      // 2^-e puts the largest magnitude in [128, 256); in two factors, as 2^-e may be
      // past the fp32 range
      const int ex = max(1, (int)(__float_as_uint(big[j]) >> 23));
      const int e = (big[j] > 0.0f && ex < 255) ? ex - 127 - 7 : 0, e1 = e / 2, e2 = e - e1;
      if (lane == 0) sm.factor[c] = a.softmax_scale * kLog2e * pow2(e1) * pow2(e2);
      const float s1 = pow2(-e1), s2 = pow2(-e2);
      const int row = (c >> 3) * 1024;
#pragma unroll
      for (int u = 0; u < 4; ++u) {              // 4 dims at a time
        const float x0 = f[j][4 * u] * s1 * s2, x1 = f[j][4 * u + 1] * s1 * s2;
        const float x2 = f[j][4 * u + 2] * s1 * s2, x3 = f[j][4 * u + 3] * s1 * s2;
        const __half2 h0 = __floats2half2_rn(x0, x1), h1 = __floats2half2_rn(x2, x3);
        int stp, place;
        q_place(16 * (lane & 7) + 4 * u, stp, place);
        const uint32_t at = row + swz128(c & 7, 2 * (stp & 3) + (place >> 1)) + 8 * (place & 1);
        uint2 v;
        v.x = *reinterpret_cast<const uint32_t*>(&h0);
        v.y = *reinterpret_cast<const uint32_t*>(&h1);
        *reinterpret_cast<uint2*>(sm.q + (2 * (lane >> 3) + (stp >> 2)) * (COLS * 128) + at) = v;
        if (rope && lane >= 28) {
          const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
          const __half2 l0 = __floats2half2_rn(x0 - f0.x, x1 - f0.y), l1 = __floats2half2_rn(x2 - f1.x, x3 - f1.y);
          v.x = *reinterpret_cast<const uint32_t*>(&l0);
          v.y = *reinterpret_cast<const uint32_t*>(&l1);
          *reinterpret_cast<uint2*>(sm.q_lo + (stp >> 2) * (COLS * 128) + at) = v;
        }
      }
    }
  }
}

// ---- output -------------------------------------------------------------------------------
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// O^T of a segment to its rows (kParts: to a part), by the softmax warps.  Each lane
// holds a dim: the columns are put together in P's place, which no product uses now,
// and leave as one bulk copy each.
template <int COLS, bool kParts>
__device__ __forceinline__ void write_out(const DenseArgs& a, Smem<COLS>& sm, int warp, int lane, int r0, int cols,
                                          int slot) {
  constexpr int kRound = kParts ? 8 : 16;        // columns put together at a time
  constexpr int kElem = kParts ? 4 : 2, kRow = D * kElem;
  const int d = 32 * warp + (lane ^ (8 * (warp & 2)));   // the lane's dim in a chunk, as the tile was laid out
#pragma unroll 1
  for (int c0 = 0; c0 < cols; c0 += kRound) {
    if (c0 > 0) {                                // the round before has been read
      if (warp == 0) bulk_wait_read();
      softmax_sync();
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {       // two chunks at a time
      uint32_t v[2][kRound];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t ta = 64 * (2 * half + j) + ((uint32_t)(32 * warp) << 16) + c0;
        if constexpr (kParts) {
#pragma unroll
          for (int k = 0; k < kRound; k += 4) {
            uint32_t u[4];
            tmem_ld4(ta + k, u);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][k + i] = u[i];
          }
        } else {
          tmem_ld16(ta, v[j]);
        }
      }
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint8_t* dst = sm.p + kElem * (128 * (2 * half + j) + d);
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
          asm volatile("" : "+r"(v[j][k]));      // not before the wait
          if constexpr (kParts) {
            *reinterpret_cast<uint32_t*>(dst + k * kRow) = v[j][k];
          } else {
            const __nv_bfloat16 o = __float2bfloat16_rn(__uint_as_float(v[j][k]) * sm.corr[c0 + k]);
            *reinterpret_cast<uint16_t*>(dst + k * kRow) = *reinterpret_cast<const uint16_t*>(&o);
          }
        }
      }
    }
    fence_proxy_async_smem();
    softmax_sync();
    if (warp == 0 && lane < kRound) {
      uint8_t* to = kParts ? reinterpret_cast<uint8_t*>(a.part + ((size_t)slot * COLS + c0 + lane) * D)
                           : reinterpret_cast<uint8_t*>(a.out + ((size_t)r0 * a.H + c0 + lane) * D);
      bulk_store(to, sm.p + lane * kRow, kRow);
      bulk_commit();
    }
  }
}

// ---- softmax ------------------------------------------------------------------------------
template <int COLS>
struct Softmax {
  using S = Smem<COLS>;
  static constexpr int HB = COLS < 32 ? COLS : 32, NB = COLS / HB;   // columns reduced at a time
  const DenseArgs& a;
  S& sm;
  int lane, warp;                                // warp 0..3: 32 keys, and 32 dims of each chunk

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
    uint32_t i = 0, outs = 0;
    int prev_r0 = -1, prev_cols = 0, prev_slot = 0;
    const uint32_t lane_off = (uint32_t)(32 * warp) << 16;
    const int mykey = 32 * warp + lane, tid = mykey;
    constexpr int kShift = RedShift<HB>::v;
    // the previous segment's output, once its last O^T is complete
    auto flush = [&]() -> bool {
      if (prev_r0 < 0) return true;
      const bool ok = wait(&sm.o_full, outs & 1);
      if (softmax_sync_or(!ok)) return false;
      ++outs;
      tc_fence_after();
      if (prev_slot < 0) write_out<COLS, false>(a, sm, warp, lane, prev_r0, prev_cols, 0);
      else write_out<COLS, true>(a, sm, warp, lane, prev_r0, prev_cols, prev_slot);
      if (warp == 0) bulk_wait_read();           // P may be written again
      softmax_sync();
      tc_fence_before();
      warp_arrive(&sm.o_free, lane);
      prev_r0 = -1;
      return true;
    };
    for (bool more = w.first(a, G, sh); more; more = w.next_segment(a, G)) {
      const int cols = w.gr.g * a.H;
      const bool whole = w.whole();
      const int slot = whole ? -1 : (w.t0 > 0 ? 2 * (int)blockIdx.x : 2 * (int)blockIdx.x + 1);
      if (!whole && w.t0 == 0)
        rec = make_int4(w.gr.r0, w.gr.g, blockIdx.x, blockIdx.x + (group_units(w.gr) - w.left + sh.per - 1) / sh.per);
      if (w.t >= w.t_end) {                      // rows that see nothing
        if (!row_valid(a, w.gr.b, w.gr.p0) && tid == 0) raise_flag(a.status, CSA_FLAG_ROW_INVALID);
        uint4* dst = reinterpret_cast<uint4*>(a.out + (size_t)w.gr.r0 * a.H * D);
        for (int k = tid; k < cols * (D / 8); k += 32 * kSoftmaxWarps) dst[k] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse && tid < cols) a.lse[(size_t)w.gr.r0 * a.H + tid] = -INFINITY;
        continue;
      }
      if (i > 0) load_queries<COLS, 4>(a, sm, w.gr, warp * (COLS / 4), COLS / 4);   // a quarter of the columns
      if (tid < COLS) sm.neg_m[tid] = 0.0f;
      fence_proxy_async_smem();
      warp_arrive(&sm.q_full, lane);
      softmax_sync();                            // factors and maxima visible to all softmax warps
      if (!flush()) return false;
      bool fresh = true;                         // no key of the segment seen yet: neg_m is not a max
      // keys that every column sees (window keys aside); none when columns are unused
      const int all_see = cols == COLS ? w.gr.W + entries_at(a, w.gr.p0) : 0;
      float2 lpart[COLS / 2];                    // this key's share of the columns' sums of p
#pragma unroll
      for (int k = 0; k < COLS / 2; ++k) lpart[k] = make_float2(0.0f, 0.0f);
#pragma unroll 1
      for (; w.t < w.t_end; ++w.t, ++i) {
        const bool ok = wait(&sm.s_full[i & 1], (i >> 1) & 1);
        bool ok_warp = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        const uint32_t ts = kTmemS + 64 * (i & 1) + lane_off;
        // the columns that see this key; usually all, and none is a window key
        const int ki = w.t * kTileKeys + mykey;
        int clo = 0, chi = COLS;
        float mu = 1.0f;
        const bool plain = (w.t + 1) * kTileKeys <= all_see && !sm.odd[i & 1][warp];
        if (!plain) {
          if (sm.odd[i & 1][warp]) mu = sm.mu[i & 1][mykey];
          int ilo = 0, ihi = -1;                 // rows of the group
          if (mu >= 0.0f) {
            if (ki < w.gr.W) {
              ilo = max(0, w.gr.wlo + ki - w.gr.p0);
              ihi = min(w.gr.g - 1, w.gr.wlo + ki + (WIN - 1) - w.gr.p0);
            } else {
              ilo = max(0, ((ki - w.gr.W + 1) << (a.P - 1)) - 1 - w.gr.p0);
              ihi = w.gr.g - 1;
            }
          }
          clo = ilo * a.H;
          chi = (ihi + 1) * a.H;
        }
        // x = logit - m; a column that does not see the key: -inf
        float2 x[COLS / 2];
#pragma unroll
        for (int k = 0; k < COLS; k += 16) tmem_ld16_pairs(ts + k, &x[k / 2]);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < COLS / 2; ++k) asm volatile("" : "+f"(x[k].x), "+f"(x[k].y));   // not before the wait
        tc_fence_before();
        warp_arrive(&sm.s_free[i & 1], lane);
        const float4* fac = reinterpret_cast<const float4*>(sm.factor);
        const float4* mr = reinterpret_cast<const float4*>(sm.neg_m);
        if (!plain) {
#pragma unroll
          for (int k = 0; k < COLS / 2; ++k) x[k] = make_float2(x[k].x * mu, x[k].y * mu);
        }
#pragma unroll
        for (int k = 0; k < COLS; k += 4) {
          const float4 f = fac[k / 4], m = mr[k / 4];
          x[k / 2] = fma2(x[k / 2], make_float2(f.x, f.y), make_float2(m.x, m.y));
          x[k / 2 + 1] = fma2(x[k / 2 + 1], make_float2(f.z, f.w), make_float2(m.z, m.w));
        }
        if (!plain) {
#pragma unroll
          for (int k = 0; k < COLS; k += 2) {
            if (k < clo || k >= chi) x[k / 2].x = -INFINITY;
            if (k + 1 < clo || k + 1 >= chi) x[k / 2].y = -INFINITY;
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < COLS / 2; ++k) top = fmaxf(fmaxf(top, x[k].x), x[k].y);
        // The running max moves only when a logit exceeds it by more than 2^14, or at
        // the segment's first key; usually it stays, and then no max or sum is reduced.
        if (softmax_sync_or(!ok_warp || fresh || top > kRescaleLog2)) {
          // a failed wait ends the role here, for all of its warps alike; O^T of the
          // tile before is complete from here on
          ok_warp = __all_sync(0xFFFFFFFFu, wait(&sm.p_free, (i & 1) ^ 1)) && ok_warp;
          if (softmax_sync_or(!ok_warp)) return false;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < COLS; k += 4) {
            const float4 v = make_float4(warp_top(x[k / 2].x), warp_top(x[k / 2].y), warp_top(x[k / 2 + 1].x),
                                         warp_top(x[k / 2 + 1].y));
            if (lane == 0) *reinterpret_cast<float4*>(&sm.red[warp][k]) = v;
          }
          softmax_sync();
          bool seen = false;
          if (tid < COLS) {                      // by how much the column's max moves
            const float t = fmaxf(fmaxf(sm.red[0][tid], sm.red[1][tid]), fmaxf(sm.red[2][tid], sm.red[3][tid]));
            seen = t != -INFINITY;
            // with one column every one that has grown moves, as the event is what costs
            const float by = (fresh ? seen : t > 1.0f) ? t : 0.0f;
            sm.neg_m[tid] -= by;
            sm.red[0][tid] = -by;              // this thread alone has read the column's tops
            sm.corr[tid] = fresh ? 1.0f : ex2(-by);
            const uint32_t m = __ballot_sync(COLS < 32 ? 0xFFFFu : 0xFFFFFFFFu, by != 0.0f);
            if (lane == 0) sm.moved[warp] = m;
          }
          const bool was_fresh = fresh;
          fresh = !softmax_sync_or(seen) && fresh;   // the new maxima are visible
          const float4* mv = reinterpret_cast<const float4*>(sm.red[0]);
          const float4* al = reinterpret_cast<const float4*>(sm.corr);
#pragma unroll
          for (int k = 0; k < COLS; k += 4) {
            const float4 d = mv[k / 4], f = al[k / 4];
            x[k / 2] = add2(x[k / 2], make_float2(d.x, d.y));
            x[k / 2 + 1] = add2(x[k / 2 + 1], make_float2(d.z, d.w));
            lpart[k / 2] = make_float2(lpart[k / 2].x * f.x, lpart[k / 2].y * f.y);
            lpart[k / 2 + 1] = make_float2(lpart[k / 2 + 1].x * f.z, lpart[k / 2 + 1].y * f.w);
          }
          if (!was_fresh) {
#pragma unroll 1
            for (int j = 0; j < 2 * (COLS / 16); ++j) {   // 16 columns of two chunks
              const int c0 = 16 * (j >> 1);
              if (!((sm.moved[c0 / 32] >> (c0 & 31)) & 0xFFFFu)) continue;
              const uint32_t ta = lane_off + 128 * (j & 1) + c0;
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
        }
        uint32_t packed[COLS / 2];
#pragma unroll
        for (int k = 0; k < COLS / 2; ++k) {
          float2 p = make_float2(ex2(x[k].x), ex2(x[k].y));
          lpart[k] = add2(lpart[k], p);
          if (!plain) p = make_float2(p.x * fmaxf(mu, 0.0f), p.y * fmaxf(mu, 0.0f));
          const __half2 hv = __floats2half2_rn(p.x, p.y);
          packed[k] = *reinterpret_cast<const uint32_t*>(&hv);
        }
        // P of the tile before is used up.  A wait that runs out here raises the abort
        // flag, and the next barrier of the role ends it.
        (void)wait(&sm.p_free, (i & 1) ^ 1);
        __syncwarp();
        uint8_t* prow = sm.p + (mykey >> 3) * 1024;
#pragma unroll
        for (int k = 0; k < COLS / 8; ++k)
          *reinterpret_cast<uint4*>(prow + swz128(mykey & 7, k)) =
              make_uint4(packed[4 * k], packed[4 * k + 1], packed[4 * k + 2], packed[4 * k + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&sm.p_full, lane);
      }
      // ---- the columns' sums
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        float tmp[HB];
#pragma unroll
        for (int k = 0; k < HB; ++k) tmp[k] = (k & 1) ? lpart[(n * HB + k) / 2].y : lpart[(n * HB + k) / 2].x;
        const float sum = warp_reduce_many<HB, false>(tmp, lane);
        if ((lane & ((1 << kShift) - 1)) == 0) sm.red[warp][n * HB + (lane >> kShift)] = sum;
      }
      softmax_sync();
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
      softmax_sync();
      prev_r0 = w.gr.r0;
      prev_cols = cols;
      prev_slot = slot;
    }
    const bool ok = flush();
    if (warp == 0) bulk_wait_all();
    return ok;
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
      mbar_init(&sm.s_free[i], kSoftmaxWarps);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.v_full[i], 4);
      mbar_init(&sm.v_free[i], 1);
    }
    mbar_init(&sm.p_full, kSoftmaxWarps);
    mbar_init(&sm.p_free, 1);
    mbar_init(&sm.q_full, kSoftmaxWarps);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_free, kSoftmaxWarps);
    mbar_init(&sm.drain, 2);
    fence_barrier_init();
    sm.abort = 0;
    sm.tile_now = 0;
  }
  if (a.rope_cos)                                // the low parts' image is zero where nothing is rotated
    for (int i = tid; i < COLS * 16; i += kThreads) reinterpret_cast<uint4*>(sm.q_lo)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (warp == kMmaWarp) tmem_alloc(&sm.tmem_base, 512);
  const Share sh = find_share(a, G, *reinterpret_cast<ShareScratch*>(sm.p));
  __syncthreads();                               // the zeros come before the low parts
  {
    // the first queries, by every warp; later ones by the softmax warps
    Walk w;
    if (w.first(a, G, sh) && w.settle(a, G)) load_queries<COLS, COLS / 16>(a, sm, w.gr, warp * (COLS / 16), COLS / 16);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // all 512 columns are this CTA's, so they start at address 0
  // registers: 512 x 128 at launch = 256 x 128 + 128 x 208 + 128 x 48
  if (warp < kDequantWarps) {
    Dequant<COLS> d{a, sm, lane, warp >> 2, lane & 3, 32 * (warp & 3) + (lane >> 2),
                    kTmemK + 64 * (warp >> 2) + ((uint32_t)(32 * (warp & 3)) << 16)};
    d.run(sh, G);
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int v = warp - kDequantWarps;
    int4 rec = make_int4(-1, 0, 0, 0);
    Softmax<COLS> s{a, sm, lane, v};
    const bool ok = s.run(sh, G, rec);
    if (v == 0 && lane == 0) a.rec[blockIdx.x] = ok ? rec : make_int4(-1, 0, 0, 0);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
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

// Joins the parts of the groups cut between CTAs: one CTA per (cut, column),
// thread = 4 dims; O = sum_q 2^(m_q - M) O_q / sum_q 2^(m_q - M) l_q in CTA order.
__global__ void __launch_bounds__(128) k_dense_merge(DenseArgs a, int cols_max) {
  pdl_wait();
  const int4 rec = __ldcg(a.rec + blockIdx.x);
  const int c = blockIdx.y;
  if (rec.x < 0 || c >= rec.y * a.H) return;
  const int n = rec.w - rec.z + 1;               // parts: slot 2 c0 + 1, then 2 (c0 + 1), 2 (c0 + 2), ...
  auto slot = [&](int q) { return q == 0 ? 2 * rec.z + 1 : 2 * (rec.z + q); };
  float M = kNoMax;
  for (int q = 0; q < n; ++q) M = fmaxf(M, __ldcg(a.part_ml + (size_t)slot(q) * 2 * cols_max + c));
  float L = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int q = 0; q < n; ++q) {
    const float* ml = a.part_ml + (size_t)slot(q) * 2 * cols_max + c;
    const float m = __ldcg(ml), l = __ldcg(ml + cols_max);
    const float w = ex2(m - M);
    const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part + ((size_t)slot(q) * cols_max + c) * D) + threadIdx.x);
    L += w * l;
    o.x += w * v.x;
    o.y += w * v.y;
    o.z += w * v.z;
    o.w += w * v.w;
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv, o.y * inv), y = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  uint2 st;
  st.x = *reinterpret_cast<const uint32_t*>(&x);
  st.y = *reinterpret_cast<const uint32_t*>(&y);
  const size_t col = (size_t)rec.x * a.H + c;
  *(reinterpret_cast<uint2*>(a.out + col * D) + threadIdx.x) = st;
  if (a.lse && threadIdx.x == 0) a.lse[col] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
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
  const int64_t tiles = ((int64_t)max_entries + 2 * WIN + kTileKeys - 1) / kTileKeys;
  return (int)std::max<int64_t>(1, std::min<int64_t>(num_sms, tiles * num_rows));
}

template <int COLS>
cudaError_t launch_cols(DenseArgs a, int grid, cudaStream_t stream) {
  static_assert(sizeof(Smem<COLS>) <= 232448, "shared memory of one CTA");
  const size_t smem = sizeof(Smem<COLS>);
  cudaError_t e = cudaFuncSetAttribute(k_dense_attn<COLS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_kernel(Order::kStream, k_dense_attn<COLS>, dim3(grid), dim3(kThreads), smem, stream, a);
  if (e != cudaSuccess || grid == 1) return e;
  return launch_kernel(Order::kChained, k_dense_merge, dim3(grid - 1, COLS), dim3(128), 0, stream, a, COLS);
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
    case 16: return launch_cols<16>(a, grid, stream);
    case 32: return launch_cols<32>(a, grid, stream);
    default: return launch_cols<64>(a, grid, stream);
  }
}

}  // namespace csa
