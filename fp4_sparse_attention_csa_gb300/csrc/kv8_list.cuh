// What the attention kernels of the 8-bit cache share: groups of rows, the list of work and a
// CTA's share of it, and the pages of a segment's tiles.
//
// A segment is one key head of a group, up to RG rows of one request at consecutive positions
// (one row where pages are listed).  The tiles (two pages) of all segments, in row and head
// order, are one list; CTA i takes the i-th equal share.  A step from one segment to the next
// counts as a.gap tiles.
#pragma once

#include "kv8_device.cuh"

namespace csa {

// ---- products ----------------------------------------------------------------------
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kind::f8f6f4, E4M3 operands, fp32 sums, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// ---- the list of work ----------------------------------------------------------------
struct Group {
  int r0, g, b, p0;                              // first row, rows, request, first position
  int tiles;                                     // of each head; 0: the row is invalid
};

// Tiles of each head of g rows from position p0 on; 0: the rows are invalid.
__device__ __forceinline__ int group_tiles(const Kv8AttnArgs& a, int b, int p0, int g) {
  if (!kv8_row_valid(a.rows, b, p0)) return 0;
  int pages = ((p0 + g - 1) >> 6) + 1;
  if (a.blocks) pages = min(pages, a.n_blocks);
  return (pages + 1) >> 1;
}
// The group that begins at row r, of at most RG rows; a whole warp looks for its end.
__device__ __forceinline__ Group group_at(const Kv8AttnArgs& a, int r, int RG) {
  Group q;
  q.r0 = r;
  q.b = __ldg(a.rows.row_req + r);
  q.p0 = __ldg(a.rows.row_pos + r);
  q.g = 1;
  if (kv8_row_valid(a.rows, q.b, q.p0)) {
    const int most = min(min(RG, a.rows.num_rows - r), kv8_pos_limit(a.rows) - q.p0);
#pragma unroll 1
    while (q.g < most) {
      const int k = q.g + lane_id();
      const bool on = k < most && __ldg(a.rows.row_req + r + k) == q.b && __ldg(a.rows.row_pos + r + k) == q.p0 + k;
      const uint32_t off = ~__ballot_sync(0xFFFFFFFFu, on);
      q.g += off ? __ffs(off) - 1 : 32;
      if (off) break;
    }
  }
  q.tiles = group_tiles(a, q.b, q.p0, q.g);
  return q;
}
__device__ __forceinline__ long long group_units(const Kv8AttnArgs& a, int tiles) {
  return tiles > 0 ? (long long)a.heads * (tiles + a.gap) : 1;
}

// Quotients of numbers that are small in all but the longest lists: a division in 64 bits is some
// hundred instructions.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

struct Share {
  int row;                                       // the first group's row
  long long first, units, per;                   // the share's first unit in it, its units, those of a whole share
};
template <int T>
struct ShareScratch {
  long long sums[T / 32];
  int starts[T / 32];
  Share out;
};

// This CTA's share of the list; every thread of the block takes part.
template <int T>
__device__ __forceinline__ Share find_share(const Kv8AttnArgs& a, int RG, ShareScratch<T>& s) {
  const int tid = threadIdx.x, lane = lane_id(), warp = warp_id(), R = a.rows.num_rows;
  if (R == 1) {                                  // the list is one row's heads: nothing to look for
    Share h;
    const long long total = group_units(a, group_tiles(a, __ldg(a.rows.row_req), __ldg(a.rows.row_pos), 1));
    h.per = quotient(max(1ll, total - a.gap) + gridDim.x - 1, gridDim.x);
    h.row = 0;
    h.first = min(total, (long long)blockIdx.x * h.per);
    h.units = (blockIdx.x + 1 == gridDim.x ? total : min(total, h.first + h.per)) - h.first;
    __syncthreads();
    return h;
  }
  const int each = (R + T - 1) / T, r_lo = min(R, tid * each), r_hi = min(R, r_lo + each);
  struct Row {
    int b, p;
    bool valid;
  };
  auto row_at = [&](int r) {
    Row x{-1, -1, false};
    if (r < 0 || r >= R) return x;
    x.b = __ldg(a.rows.row_req + r);
    x.p = __ldg(a.rows.row_pos + r);
    x.valid = kv8_row_valid(a.rows, x.b, x.p);
    return x;
  };
  auto follows = [&](const Row& x, const Row& y) { return RG > 1 && x.valid && y.valid && x.b == y.b && x.p + 1 == y.p; };
  Row start = row_at(r_lo);
  bool inside = follows(row_at(r_lo - 1), start);
  // runs of rows that follow one another: the start of the one that reaches into this thread's rows
  int run = r_lo;
  if (RG > 1) {
    int last = -1;
    bool on = inside;
    Row x = start;
#pragma unroll 1
    for (int r = r_lo; r < r_hi; ++r) {
      if (!on) last = r;
      const Row y = row_at(r + 1);
      on = follows(x, y);
      x = y;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, last, o);
      if (lane >= o) last = max(last, y);
    }
    if (lane == 31) s.starts[warp] = last;
    __syncthreads();
    run = __shfl_up_sync(0xFFFFFFFFu, last, 1);
    if (lane == 0) run = -1;
#pragma unroll
    for (int w = 0; w < T / 32; ++w)
      if (w < warp) run = max(run, s.starts[w]);
  }
  // Groups begin every RG rows of a run, and a group's units count where it ends.  First their sum over this
  // thread's rows; then, in the one thread whose groups hold this share's first unit, the group that does.
  long long sum = 0, lo = 0, per = 0, units = 0, u = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int k = inside ? (r_lo - run) % RG : 0;      // rows of the group before this one
    Row x = start;
#pragma unroll 1
    for (int r = r_lo; r < r_hi; ++r) {
      const Row y = row_at(r + 1);
      const bool on = k + 1 < RG && follows(x, y);
      if (!on) {
        const long long n = group_units(a, group_tiles(a, x.b, x.p - k, k + 1));
        if (pass == 0) {
          sum += n;
        } else if (lo >= u + n) {
          u += n;
        } else {
          s.out.row = r - k;
          s.out.first = lo - u;
          break;
        }
      }
      k = on ? k + 1 : 0;
      x = y;
    }
    if (pass > 0) break;
    long long upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s.sums[warp] = upto;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) {
      if (w < warp) upto += s.sums[w];
      total += s.sums[w];
    }
    per = quotient(max(1ll, total - a.gap) + gridDim.x - 1, gridDim.x);   // nothing follows the last segment
    lo = min(total, (long long)blockIdx.x * per);
    units = (blockIdx.x + 1 == gridDim.x ? total : min(total, lo + per)) - lo;
    u = upto - sum;
    if (units == 0 || lo < u || lo >= upto) break;
  }
  __syncthreads();
  Share h = s.out;
  h.units = units;
  h.per = per;
  return h;
}

// ---- this CTA's tiles, segment by segment ------------------------------------------------
struct Walk {
  Group gr;
  int h, t0, t, t_end;                           // key head, the segment's tiles and the current one
  long long left;                                // units of the share from this segment's first one on
  __device__ __forceinline__ void enter(int head, int first) {
    h = head;
    t0 = t = first;
    t_end = (int)min((long long)gr.tiles, first + left);
  }
  __device__ __forceinline__ bool open(const Kv8AttnArgs& a, int RG, int row, long long first) {
    if (left <= 0) return false;
    gr = group_at(a, row, RG);
    const int one = gr.tiles + a.gap;
    const int head = (int)quotient(first, one);
    if (gr.tiles > 0) enter(head, (int)(first - (long long)head * one));
    else enter(0, 0);
    return true;
  }
  // the share's first segment; false when the share is empty
  __device__ __forceinline__ bool first(const Kv8AttnArgs& a, int RG, const Share& s) {
    left = s.units;
    return open(a, RG, s.row, s.first);
  }
  __device__ __forceinline__ bool next_segment(const Kv8AttnArgs& a, int RG) {
    left -= gr.tiles > 0 ? gr.tiles + a.gap - t0 : 1;
    if (gr.tiles == 0 || h + 1 == a.heads) return open(a, RG, gr.r0 + gr.g, 0);
    if (left <= 0) return false;
    enter(h + 1, 0);
    return true;
  }
  // the first tile at or after t; false at the share's end
  __device__ __forceinline__ bool settle(const Kv8AttnArgs& a, int RG) {
    while (t >= t_end)
      if (!next_segment(a, RG)) return false;
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && left >= gr.tiles; }
};

// ---- sums ----------------------------------------------------------------------------------
// Value scales of a segment are near one another up to this many powers of two beside its first tile's.  There the
// probabilities that the products take, y <= 2^15, serve the sum as well: the key that makes most of it has y >= 2^-26
// (two scales can be 32 apart, and the largest y is 2^6 at least), one that fp32 no longer holds, below 2^-126, is
// nothing beside it, and the units' power of two, which the sum's maximum takes up, costs that a bit or two.
constexpr float kKv8Near = 16.0f;
// A logit's difference to the maximum is one fused step, off by half a step of the maximum: 2^-4 of a power of two at this
// magnitude.  Beyond it that error would be the result, so the tile that moves the maximum rounds the logit first, as
// the maximum was, and its largest y is what it should be.
constexpr float kKv8Large = 1048576.0f;

// ---- pages ---------------------------------------------------------------------------------
// The pages of 16 tiles, one a lane: page number (INT_MAX: none) and pool page.
struct Pages {
  int j, page;
};
// A list of pages, 32 entries at a time by a whole warp.  An entry counts when it is one of the row's pages and above all
// that count before it; those that count follow one another without gaps, so a row has no more of them than pages.
// Which of entries i = 32 k + lane do: `above` is the largest that does before them, and becomes the largest so far;
// `listed`, whether the entry stands before the list's end.
__device__ __forceinline__ bool entry_counts(int e, bool listed, int last, int& above) {
  const int lane = lane_id();
  int top = listed && e <= last ? e : -1;         // the largest entry up to this lane
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, top, o);
    if (lane >= o) top = max(top, y);
  }
  int before = __shfl_up_sync(0xFFFFFFFFu, top, 1);
  before = lane == 0 ? above : max(above, before);
  above = max(above, __shfl_sync(0xFFFFFFFFu, top, 31));
  return listed && e <= last && e > before;
}
// Those of tiles 16 chunk .. 16 chunk + 15, whatever the list holds: it is read from its beginning, and to its end
// for the flag.
__device__ __noinline__ inline int any_entries(const int32_t* list, int n_blocks, int last, int chunk, uint32_t* status) {
  const int lane = lane_id();
  int n = 0, above = -1, j = INT_MAX;            // n: how many count so far
#pragma unroll 1
  for (int i = 0; i < n_blocks; i += 32) {
    const int e = i + lane < n_blocks ? __ldg(list + i + lane) : -1;
    const uint32_t stop = __ballot_sync(0xFFFFFFFFu, e < 0);
    const bool listed = lane < (stop ? __ffs(stop) - 1 : 32);
    const uint32_t counts = __ballot_sync(0xFFFFFFFFu, entry_counts(e, listed, last, above));
    if (listed && !((counts >> lane) & 1u)) raise_flag(status, CSA_FLAG_TOPK_OOB);
    if ((n & 31) == 0 && (counts & (counts + 1)) == 0) {     // as they are
      if (n == 32 * chunk && ((counts >> lane) & 1u)) j = e;
      n += __popc(counts);
    } else {
#pragma unroll 1
      for (uint32_t left = counts; left; left &= left - 1, ++n) {
        const int v = __shfl_sync(0xFFFFFFFFu, e, __ffs(left) - 1);
        if (n == 32 * chunk + lane) j = v;
      }
    }
    if (stop) break;
  }
  return j;
}
// The pages of tiles 16 chunk .. 16 chunk + 15.  kCarry: `above` and `ended` carry a list's rule from chunk to chunk, and of
// one with an entry that does not count nothing is above `above`; else a chunk is looked for by itself, which is less
// code beside loops that have no lists.
template <bool kCarry>
__device__ __forceinline__ Pages pages_of(const Kv8AttnArgs& a, const Group& gr, int h, int chunk, int& above,
                                          bool& ended) {
  const int lane = lane_id(), i = 32 * chunk + lane, last = (gr.p0 + gr.g - 1) >> 6;
  Pages x{INT_MAX, -1};
  if (a.blocks == nullptr) {
    if (i <= last) x.j = i;
  } else if (const int32_t* list = a.blocks + ((size_t)gr.r0 * a.heads + h) * a.n_blocks; !kCarry) {
    x.j = any_entries(list, a.n_blocks, last, chunk, a.status);
  } else {
    const int e = i < a.n_blocks && !ended ? __ldg(list + i) : -1;
    const uint32_t stop = __ballot_sync(0xFFFFFFFFu, e < 0);
    const bool listed = !ended && lane < (stop ? __ffs(stop) - 1 : 32);
    ended = ended || stop != 0;
    const bool counts = entry_counts(e, listed, last, above);
    if (counts) x.j = e;
    if (__any_sync(0xFFFFFFFFu, listed && !counts)) {
      x.j = any_entries(list, a.n_blocks, last, chunk, a.status);
      above = INT_MAX;
      ended = false;
    }
  }
  if (x.j != INT_MAX) {
    x.page = __ldg(a.page_table + (size_t)gr.b * a.rows.max_pages + x.j);
    if ((uint32_t)x.page >= (uint32_t)a.num_pages) {
      raise_flag(a.status, CSA_FLAG_PAGE_OOB);
      x = Pages{INT_MAX, -1};
    }
  }
  return x;
}
// Behind the segment's last tile: entries that no tile has are looked at, too (where kCarry, else they have been).
__device__ __forceinline__ void end_of_list(const Kv8AttnArgs& a, const Group& gr, int h, bool ended) {
  if (a.blocks == nullptr || ended || (gr.tiles + 15) / 16 * 32 >= a.n_blocks) return;
  (void)any_entries(a.blocks + ((size_t)gr.r0 * a.heads + h) * a.n_blocks, a.n_blocks, (gr.p0 + gr.g - 1) >> 6, 0, a.status);
}

// ---- launch ------------------------------------------------------------------------------------
constexpr size_t up256(size_t x) { return (x + 255) / 256 * 256; }
constexpr int kKv8WideCols = 256;                // columns of a wide group

// CTAs of a call: no more than units of work (gap 1), as far as the host's bounds tell.
inline int kv8_grid(int64_t rows, int64_t heads, int64_t pages, int limit) {
  const int64_t tiles = rows * heads * ((pages + 1) / 2 + 1);
  return (int)(tiles < 1 ? 1 : (tiles < limit ? tiles : limit));
}
inline int kv8_wide_grid(int64_t rows, int64_t heads, int64_t max_entries, int num_sms) {
  return kv8_grid(rows, heads, kv8_pages(max_entries), num_sms);
}
// The parts of cut segments in the workspace: records, (m, l), O / l.
inline size_t kv8_parts_bytes(size_t grid, size_t cols, size_t dim) {
  return up256(grid * sizeof(int4)) + up256(2 * grid * 2 * cols * sizeof(float)) + 2 * grid * cols * dim * sizeof(float);
}
inline void kv8_place_parts(Kv8AttnArgs& a, uint8_t* ws, size_t grid, size_t cols) {
  a.rec = reinterpret_cast<int4*>(ws);
  ws += up256(grid * sizeof(int4));
  a.part_ml = reinterpret_cast<float*>(ws);
  ws += up256(2 * grid * 2 * cols * sizeof(float));
  a.part = reinterpret_cast<float*>(ws);
}
// Joins the parts of the segments that `grid` CTAs cut (kv8_attn.cu).
cudaError_t launch_kv8_merge(const Kv8AttnArgs& a, int cols, int grid, cudaStream_t stream);
// Attention of groups of up to kKv8WideCols columns (kv8_wide.cu).
cudaError_t launch_kv8_wide(const Kv8AttnArgs& a, uint8_t* ws, int num_sms, cudaStream_t stream);

}  // namespace csa
