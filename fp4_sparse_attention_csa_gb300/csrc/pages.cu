// csa_pages_reserve / fork / free / compact: the page table, the pages' counts
// and, where a page is copied or moved, both pools, changed on the device.
//
// Mathematics.  Let used(p) = [refs[p] > 0] and before(p) = sum of used over ids
// below p.  The k-th lowest free page is the free p with p - before(p) = k, so
// one exclusive sum over the counts numbers every free page; the k-th highest
// used page is the used p with U - before(p) - 1 = k (U pages used), so the
// holes below U and the used pages past U pair up without a second pass over
// their number.  A reservation numbers its own needs by the same kind of sum,
// over (request, logical page) in list order.
//
// Both sums run in one launch of one 8-CTA cluster: each CTA counts its eighth,
// the counts are exchanged through distributed shared memory, and each CTA
// numbers its eighth.  What is bound by memory, the page copies, is a second
// launch over the whole GPU whose prologue overlaps the first.  Counts change
// by atomic adds of whole numbers, whose order cannot show in the result.
//
// Measured on the device, with the two small copies that reset the tables, us:
// forking 2 requests and reserving their next block 17; 64 x 3 children with a copied
// page each 34 (32 MB both ways: the plan and the launches are half of it);
// releasing 96 requests and reserving 96 prompts 23; compacting 1500 pages 14, 49999
// pages 112.  Of the last 90 are k_pages_move, 516 MB at 5.7 TB/s, 0.84 of a plain
// copy's rate, and 13 the plan: two passes over the counts and their exchange.
#include <cooperative_groups.h>

#include <algorithm>

#include "csa_device.cuh"
#include "csa_internal.h"

namespace cg = cooperative_groups;

namespace csa {

namespace {

constexpr int kPlanCtas = 8;                   // the portable cluster size
constexpr int kPlanThreads = 1024;
constexpr int kPerThread = 16;                 // counts a thread numbers per round
constexpr int kCopyThreads = 256;
constexpr int kCopyCtasPerSm = 8;
constexpr int kKvVec = KV_PAGE / 16, kPageVec = (KV_PAGE + IDX_PAGE) / 16;   // 1152, 1424

// Head of a planning workspace.
struct PlanHead {
  int32_t copies;                              // pages to copy
  int32_t pad[63];
};

__host__ __device__ constexpr size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// The whole list strictly increasing, below num_requests, padded at the end;
// the same answer in every thread of the block.
__device__ bool list_ok(const int32_t* req, int n, int num_requests) {
  bool ok = true;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int v = __ldg(req + i), prev = i > 0 ? __ldg(req + i - 1) : 0;
    if (v >= 0) ok &= v < num_requests && (i == 0 || (prev >= 0 && v > prev));
  }
  return __syncthreads_and(ok);
}

// Exclusive sum over the block's threads; total in every thread.
__device__ int block_exclusive(int v, int* s_warp, int& total) {
  const int lane = lane_id(), warp = warp_id(), warps = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                             // the previous round's readers are done
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < warps ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  total = s_warp[warps - 1];
  return x - v + (warp > 0 ? s_warp[warp - 1] : 0);
}

__device__ int block_sum(int v, int* s_warp) {
  int total;
  block_exclusive(v, s_warp, total);
  return total;
}

__device__ __forceinline__ int4 refs4(const int32_t* refs, int i, int n) {
  if (i + 4 <= n) return *reinterpret_cast<const int4*>(refs + i);
  int4 v = make_int4(0, 0, 0, 0);
  if (i < n) v.x = refs[i];
  if (i + 1 < n) v.y = refs[i + 1];
  if (i + 2 < n) v.z = refs[i + 2];
  return v;
}

// Elements per CTA of n spread over the cluster, a multiple of 4.
__device__ __forceinline__ int plan_share(int n) { return (int)((((int64_t)n + kPlanCtas - 1) / kPlanCtas + 3) & ~(int64_t)3); }

__device__ int count_used(const int32_t* refs, int lo, int hi, int n) {
  int c = 0;
#pragma unroll 4
  for (int i = lo + 4 * (int)threadIdx.x; i < hi; i += 4 * kPlanThreads) {
    const int4 v = refs4(refs, i, n);
    c += (v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0);
  }
  return c;
}

// emit(p, used, used pages below p) for every p in [lo, hi)
template <typename F>
__device__ void number_pages(const int32_t* refs, int lo, int hi, int n, int below, int* s_warp, F emit) {
  for (int base = lo; base < hi; base += kPerThread * kPlanThreads) {
    const int p0 = base + kPerThread * (int)threadIdx.x;
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < kPerThread; k += 4) {
      if (p0 + k < hi) {
        const int4 v = refs4(refs, p0 + k, n);
        bits |= (uint32_t)((v.x > 0) | (v.y > 0) << 1 | (v.z > 0) << 2 | (v.w > 0) << 3) << k;
      }
    }
    int total;
    int u = below + block_exclusive(__popc(bits), s_warp, total);
    for (int k = 0; k < kPerThread && p0 + k < hi; ++k) {
      const bool used = (bits >> k) & 1u;
      emit(p0 + k, used, u);
      u += used;
    }
    below += total;
  }
}

// The CTA copies page src to page dst in both pools.
__device__ __forceinline__ void copy_page(const PagesArgs& a, int src, int dst) {
  const uint4* kv = reinterpret_cast<const uint4*>(a.kv_pool + (size_t)src * KV_PAGE);
  const uint4* ix = reinterpret_cast<const uint4*>(a.idx_pool + (size_t)src * IDX_PAGE);
  uint4* kvd = reinterpret_cast<uint4*>(a.kv_pool + (size_t)dst * KV_PAGE);
  uint4* ixd = reinterpret_cast<uint4*>(a.idx_pool + (size_t)dst * IDX_PAGE);
  constexpr int kRounds = (kPageVec + kCopyThreads - 1) / kCopyThreads;
  uint4 v[kRounds];
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const int i = threadIdx.x + k * kCopyThreads;
    if (i < kPageVec) v[k] = __ldcs(i < kKvVec ? kv + i : ix + (i - kKvVec));
  }
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const int i = threadIdx.x + k * kCopyThreads;
    if (i < kPageVec) __stcs(i < kKvVec ? kvd + i : ixd + (i - kKvVec), v[k]);
  }
}

// ---- reserve ---------------------------------------------------------------------
struct ReserveWs {
  PlanHead* head;
  int32_t* plan;                               // [units] need's number * 2 + copied, -1: none
  int32_t* fresh;                              // [units] free pages, lowest first
  int32_t* src;                                // [units] pages to copy
  int32_t* dst;
};
__host__ __device__ inline ReserveWs reserve_ws(void* ws, int64_t units) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  const size_t step = up256((size_t)units * sizeof(int32_t));
  ReserveWs w;
  w.head = reinterpret_cast<PlanHead*>(p);
  p += sizeof(PlanHead);
  w.plan = reinterpret_cast<int32_t*>(p);
  w.fresh = reinterpret_cast<int32_t*>(p + step);
  w.src = reinterpret_cast<int32_t*>(p + 2 * step);
  w.dst = reinterpret_cast<int32_t*>(p + 3 * step);
  return w;
}

// One unit = one logical page of one request of the list.  The table slot of
// unit u, or -1 when the unit is not asked for; an impossible request adds its flag.
__device__ __forceinline__ int64_t unit_slot(const PagesArgs& a, int u, int upr, uint32_t& flags) {
  const int i = u / upr, b = __ldg(a.req + i);
  if (b < 0) return -1;
  const int64_t first = __ldg(a.arg0 + i), count = __ldg(a.arg1 + i);
  if (first < 0 || count < 0 || count > a.max_count ||
      (count > 0 && (first + count - 1) / PAGE >= a.max_pages)) {
    flags |= CSA_FLAG_ROW_INVALID;
    return -1;
  }
  const int64_t lp = first / PAGE + u % upr;
  if (count == 0 || lp > (first + count - 1) / PAGE) return -1;
  return (int64_t)b * a.max_pages + lp;
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
k_pages_reserve(PagesArgs a, int units, int upr) {
  __shared__ int s_warp[32];
  __shared__ int s_used, s_need;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  pdl_trigger();
  const ReserveWs w = reserve_ws(a.ws, units);
  if (!list_ok(a.req, a.n, a.num_requests)) {  // the same answer in all CTAs
    if (rank == 0 && threadIdx.x == 0) {
      raise_flag(a.status, CSA_FLAG_ROW_INVALID);
      w.head->copies = 0;
    }
    return;
  }
  const int N = a.num_pages;
  const int share = plan_share(N), lo = min(N, rank * share), hi = min(N, lo + share);
  const int ushare = (units + kPlanCtas - 1) / kPlanCtas;
  const int ulo = min(units, rank * ushare), uhi = min(units, ulo + ushare);
  // ---- count: used pages, and the needs (0 none, 2 a page, 3 a copy)
  const int used = block_sum(count_used(a.refs, lo, hi, N), s_warp);
  int need = 0;
  uint32_t flags = 0;
  for (int u = ulo + (int)threadIdx.x; u < uhi; u += kPlanThreads) {
    const int64_t at = unit_slot(a, u, upr, flags);
    int kind = 0;
    if (at >= 0) {
      const int p = a.page_table[at];
      if (p < 0) {
        kind = 2;
      } else {
        const int r = p < N ? a.refs[p] : 0;
        if (r <= 0) flags |= CSA_FLAG_PAGE_OOB;
        else if (r > 1) kind = 3;
      }
    }
    w.plan[u] = kind;
    need += kind != 0;
  }
  need = block_sum(need, s_warp);
  if (threadIdx.x == 0) {
    s_used = used;
    s_need = need;
    if (rank == 0) w.head->copies = 0;
  }
  cluster.sync();
  int used_below = 0, need_below = 0, needs = 0, all_used = 0;
#pragma unroll
  for (int c = 0; c < kPlanCtas; ++c) {
    const int uc = *cluster.map_shared_rank(&s_used, c), nc = *cluster.map_shared_rank(&s_need, c);
    if (c < rank) { used_below += uc; need_below += nc; }
    needs += nc;
    all_used += uc;
  }
  // ---- number: the free pages that are needed, and the needs
  if (needs > 0) {
    number_pages(a.refs, lo, hi, N, used_below, s_warp, [&](int p, bool is_used, int below) {
      if (!is_used && p - below < needs) w.fresh[p - below] = p;
    });
    for (int base = ulo; base < uhi; base += kPlanThreads) {
      const int u = base + (int)threadIdx.x;
      const int kind = u < uhi ? w.plan[u] : 0;
      int total;
      const int k = need_below + block_exclusive(kind != 0, s_warp, total);
      if (u < uhi) w.plan[u] = kind ? 2 * k + (kind & 1) : -1;
      need_below += total;
    }
  }
  cluster.sync();                              // fresh[] complete, every count read; remote reads done
  // ---- write: table, counts and the list of copies
  if (needs > 0) {
    const int free_pages = N - all_used;
    for (int u = ulo + (int)threadIdx.x; u < uhi; u += kPlanThreads) {
      const int v = w.plan[u];
      if (v < 0) continue;
      if ((v >> 1) >= free_pages) {
        flags |= CSA_FLAG_NO_PAGES;
        continue;
      }
      const int p = __ldcg(w.fresh + (v >> 1));
      uint32_t none = 0;
      const int64_t at = unit_slot(a, u, upr, none);
      if (v & 1) {
        const int old = a.page_table[at];
        atomicSub(a.refs + old, 1);
        const int c = atomicAdd(&w.head->copies, 1);
        w.src[c] = old;
        w.dst[c] = p;
      }
      a.refs[p] = 1;
      a.page_table[at] = p;
    }
  }
  if (flags) raise_flag(a.status, flags);
}

__global__ void __launch_bounds__(kCopyThreads) k_pages_copy(PagesArgs a, int units) {
  pdl_wait();
  const ReserveWs w = reserve_ws(a.ws, units);
  const int n = __ldcg(&w.head->copies);
  for (int k = blockIdx.x; k < n; k += gridDim.x) copy_page(a, __ldcg(w.src + k), __ldcg(w.dst + k));
}

// ---- fork ------------------------------------------------------------------------
// Whether `v` is in the (valid) list of children: a binary search, its padding
// sorting last.
__device__ bool in_list(const int32_t* req, int n, int v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    const int x = __ldg(req + mid);
    if (x >= 0 && x < v) lo = mid + 1; else hi = mid;
  }
  return lo < n && __ldg(req + lo) == v;
}

// Adds a count to page p; false when the page has none.  By compare and swap, so that
// nobody sees a count that is taken back.
__device__ __forceinline__ bool add_count(int32_t* refs, int p) {
  int seen = __ldcg(refs + p);
  while (seen > 0) {                             // ends: each failure is another thread's success
    const int was = atomicCAS(refs + p, seen, seen + 1);
    if (was == seen) return true;
    seen = was;
  }
  return false;
}
// Drops one count of page p; false when the page had none.
__device__ __forceinline__ bool drop_count(int32_t* refs, int p) {
  if (atomicSub(refs + p, 1) > 0) return true;
  atomicAdd(refs + p, 1);
  return false;
}

__global__ void __launch_bounds__(256) k_pages_fork(PagesArgs a) {
  bool ok = list_ok(a.req, a.n, a.num_requests);
  bool mine = true;
  for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
    if (__ldg(a.req + i) < 0) continue;
    const int p = __ldg(a.parent + i);
    mine &= p >= 0 && p < a.num_requests && !in_list(a.req, a.n, p);
  }
  ok = __syncthreads_and(mine) && ok;
  if (!ok) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) raise_flag(a.status, CSA_FLAG_ROW_INVALID);
    return;
  }
  const int i = blockIdx.x, child = __ldg(a.req + i);
  if (child < 0) return;
  const int parent = __ldg(a.parent + i), entries = __ldg(a.arg0 + i);
  const int shared = entries / PAGE + (entries % PAGE > 0);
  if (entries < 0 || shared > a.max_pages) {
    if (blockIdx.y == 0 && threadIdx.x == 0) raise_flag(a.status, CSA_FLAG_ROW_INVALID);
    return;
  }
  const int t = blockIdx.y * blockDim.x + threadIdx.x, step = gridDim.y * blockDim.x;
  // ---- the ring and the pending token
  if (a.win_codes) {
    const size_t vecs = (size_t)a.win_cap * (D / 16);
    const uint4* s = reinterpret_cast<const uint4*>(a.win_codes) + parent * vecs;
    uint4* d = reinterpret_cast<uint4*>(a.win_codes) + child * vecs;
    size_t k = t;
    for (; k + 3 * (size_t)step < vecs; k += 4 * (size_t)step) {
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = s[k + j * (size_t)step];
#pragma unroll
      for (int j = 0; j < 4; ++j) d[k + j * (size_t)step] = v[j];
    }
    for (; k < vecs; k += step) d[k] = s[k];
    const float* fs = a.win_scale + (size_t)parent * a.win_cap;
    float* fd = a.win_scale + (size_t)child * a.win_cap;
    for (int j = t; j < a.win_cap; j += step) fd[j] = fs[j];
  }
  if (a.pending) {
    constexpr int kVecs = (D + DI) * 2 / 16;
    const uint4* s = reinterpret_cast<const uint4*>(a.pending) + (size_t)parent * kVecs;
    uint4* d = reinterpret_cast<uint4*>(a.pending) + (size_t)child * kVecs;
    for (int k = t; k < kVecs; k += step) d[k] = s[k];
  }
  // ---- the table row and the counts
  const int32_t* ps = a.page_table + (size_t)parent * a.max_pages;
  int32_t* pd = a.page_table + (size_t)child * a.max_pages;
  uint32_t flags = 0;
  for (int j = t; j < a.max_pages; j += step) {
    const int old = pd[j];
    int p = j < shared ? ps[j] : -1;
    if (p >= a.num_pages) {
      flags |= CSA_FLAG_PAGE_OOB;
      p = -1;
    }
    p = max(p, -1);
    if (p >= 0 && !add_count(a.refs, p)) {
      flags |= CSA_FLAG_PAGE_OOB;
      p = -1;
    }
    if (old >= a.num_pages || (old >= 0 && !drop_count(a.refs, old))) flags |= CSA_FLAG_PAGE_OOB;
    if (old != p) pd[j] = p;
  }
  if (flags) raise_flag(a.status, flags);
}

// ---- free ------------------------------------------------------------------------
__global__ void __launch_bounds__(256) k_pages_free(PagesArgs a) {
  if (!list_ok(a.req, a.n, a.num_requests)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) raise_flag(a.status, CSA_FLAG_ROW_INVALID);
    return;
  }
  const int b = __ldg(a.req + blockIdx.x);
  if (b < 0) return;
  const int keep = a.arg0 ? __ldg(a.arg0 + blockIdx.x) : 0;
  if (keep < 0) {
    if (blockIdx.y == 0 && threadIdx.x == 0) raise_flag(a.status, CSA_FLAG_ROW_INVALID);
    return;
  }
  const int kept = keep / PAGE + (keep % PAGE > 0);
  int32_t* row = a.page_table + (size_t)b * a.max_pages;
  uint32_t flags = 0;
  for (int64_t j = (int64_t)kept + blockIdx.y * blockDim.x + threadIdx.x; j < a.max_pages; j += gridDim.y * blockDim.x) {
    const int p = row[j];
    if (p < 0) continue;
    row[j] = -1;
    if (p >= a.num_pages || !drop_count(a.refs, p)) flags |= CSA_FLAG_PAGE_OOB;
  }
  if (flags) raise_flag(a.status, flags);
}

// ---- compact ---------------------------------------------------------------------
struct CompactWs {
  PlanHead* head;
  int32_t* map;                                // [num_pages] new id, -1 free
  int32_t* hole;                               // [num_pages / 2 + 1]
  int32_t* mover;
};
__host__ __device__ inline CompactWs compact_ws(void* ws, int num_pages) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  const size_t half = up256(((size_t)num_pages / 2 + 1) * sizeof(int32_t));
  CompactWs w;
  w.head = reinterpret_cast<PlanHead*>(p);
  p += sizeof(PlanHead);
  w.map = reinterpret_cast<int32_t*>(p);
  p += up256((size_t)num_pages * sizeof(int32_t));
  w.hole = reinterpret_cast<int32_t*>(p);
  w.mover = reinterpret_cast<int32_t*>(p + half);
  return w;
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1) k_pages_compact(PagesArgs a) {
  __shared__ int s_warp[32];
  __shared__ int s_used;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  pdl_trigger();
  const CompactWs w = compact_ws(a.ws, a.num_pages);
  int32_t* map = a.new_id ? a.new_id : w.map;
  const int N = a.num_pages;
  const int share = plan_share(N), lo = min(N, rank * share), hi = min(N, lo + share);
  const int used = block_sum(count_used(a.refs, lo, hi, N), s_warp);
  if (threadIdx.x == 0) s_used = used;
  cluster.sync();
  int below = 0, U = 0;
#pragma unroll
  for (int c = 0; c < kPlanCtas; ++c) {
    const int uc = *cluster.map_shared_rank(&s_used, c);
    if (c < rank) below += uc;
    U += uc;
  }
  if (rank == 0 && threadIdx.x == 0) {
    if (a.num_used) *a.num_used = U;
    if (U == 0 || U == N) w.head->copies = 0;
  }
  // holes below U and used pages past U are equally many, at most N / 2
  number_pages(a.refs, lo, hi, N, below, s_warp, [&](int p, bool is_used, int before) {
    if (is_used && p >= U) {
      w.mover[U - before - 1] = p;             // its hole's number; map[p] follows below
    } else {
      if (p < U && !is_used) w.hole[p - before] = p;
      map[p] = is_used ? p : -1;
    }
    if (p == U - 1 && U < N) w.head->copies = U - (before + is_used);
  });
  cluster.sync();                              // hole[], mover[] and copies complete; remote reads done
  const int M = (U == 0 || U == N) ? 0 : __ldcg(&w.head->copies);
  for (int k = rank * kPlanThreads + (int)threadIdx.x; k < M; k += kPlanCtas * kPlanThreads)
    map[__ldcg(w.mover + k)] = __ldcg(w.hole + k);
}

__global__ void __launch_bounds__(kCopyThreads) k_pages_move(PagesArgs a) {
  pdl_wait();
  const CompactWs w = compact_ws(a.ws, a.num_pages);
  const int32_t* map = a.new_id ? a.new_id : w.map;
  const int M = __ldcg(&w.head->copies);
  // the table through the map
  const int64_t slots = (int64_t)a.num_requests * a.max_pages;
  uint32_t flags = 0;
  for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < slots; i += (int64_t)gridDim.x * kCopyThreads) {
    const int p = a.page_table[i];
    if (p < 0) continue;
    const int q = p < a.num_pages ? __ldcg(map + p) : -1;
    if (q < 0) flags |= CSA_FLAG_PAGE_OOB;
    if (q != p) a.page_table[i] = q;
  }
  if (flags) raise_flag(a.status, flags);
  for (int k = blockIdx.x; k < M; k += gridDim.x) {
    const int src = __ldcg(w.mover + k), dst = __ldcg(w.hole + k);
    copy_page(a, src, dst);
    if (threadIdx.x == 0) {
      a.refs[dst] = a.refs[src];
      a.refs[src] = 0;
    }
  }
}

}  // namespace

int64_t pages_reserve_units(int32_t n, int32_t max_count) {
  return (int64_t)n * ((int64_t)max_count / PAGE + 2);
}
size_t pages_reserve_ws_bytes(int32_t n, int32_t max_count) {
  return sizeof(PlanHead) + 4 * up256((size_t)pages_reserve_units(n, max_count) * sizeof(int32_t));
}
size_t pages_compact_ws_bytes(int32_t num_pages) {
  return sizeof(PlanHead) + up256((size_t)num_pages * sizeof(int32_t)) +
         2 * up256(((size_t)num_pages / 2 + 1) * sizeof(int32_t));
}

cudaError_t launch_pages_reserve(const PagesArgs& a, int num_sms, cudaStream_t stream) {
  const int upr = a.max_count / PAGE + 2;
  const int units = (int)pages_reserve_units(a.n, a.max_count);
  cudaError_t e = launch_kernel(Order::kStream, k_pages_reserve, dim3(kPlanCtas), dim3(kPlanThreads), 0, stream, a,
                                units, upr);
  if (e != cudaSuccess) return e;
  const int grid = std::min(units, std::max(1, num_sms) * kCopyCtasPerSm);
  return launch_kernel(Order::kChained, k_pages_copy, dim3(grid), dim3(kCopyThreads), 0, stream, a, units);
}

cudaError_t launch_pages_fork(const PagesArgs& a, cudaStream_t stream) {
  // 16 KB of ring, or 1024 table slots, per CTA
  const int64_t ring = a.win_codes ? ((int64_t)a.win_cap * D + 16383) / 16384 : 1;
  const int64_t slots = ((int64_t)a.max_pages + 1023) / 1024;
  const int parts = (int)std::min<int64_t>(64, std::max(ring, slots));
  return launch_kernel(Order::kStream, k_pages_fork, dim3(a.n, parts), dim3(256), 0, stream, a);
}

cudaError_t launch_pages_free(const PagesArgs& a, cudaStream_t stream) {
  const int parts = (int)std::min<int64_t>(64, ((int64_t)a.max_pages + 1023) / 1024);
  return launch_kernel(Order::kStream, k_pages_free, dim3(a.n, parts), dim3(256), 0, stream, a);
}

cudaError_t launch_pages_compact(const PagesArgs& a, int num_sms, cudaStream_t stream) {
  cudaError_t e =
      launch_kernel(Order::kStream, k_pages_compact, dim3(kPlanCtas), dim3(kPlanThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  const int64_t slots = (int64_t)a.num_requests * a.max_pages;
  const int64_t want = std::max<int64_t>(a.num_pages / 2 + 1, (slots + kCopyThreads - 1) / kCopyThreads);
  const int grid = (int)std::min<int64_t>(want, (int64_t)std::max(1, num_sms) * kCopyCtasPerSm);
  return launch_kernel(Order::kChained, k_pages_move, dim3(grid), dim3(kCopyThreads), 0, stream, a);
}

}  // namespace csa
