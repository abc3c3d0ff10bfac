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
#include <algorithm>

#include "attn_device.cuh"
#include "csa_internal.h"

namespace csa {

namespace {

constexpr int kThreads = 512;
constexpr int kTileKeys = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;             // the running max moves when exceeded by 2^8: p <= 2^8 in fp16

// ---- the list of work ----------------------------------------------------------------
struct Group {
  int r0, g, b, p0;                              // first row, rows, request, first position
  int W, wlo;                                    // window keys and the first one's position
  int keys, tiles;                               // tiles 0: the rows see nothing (or are invalid)
};

__device__ __forceinline__ bool row_valid(const DenseArgs& a, int b, int pos) {
  return b >= 0 && b < a.num_requests && pos >= 0 && (a.rope_cos == nullptr || pos < a.rope_rows) &&
         ((int64_t)pos + 1) / a.P <= (int64_t)a.max_pages * PAGE;
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
  q.keys = q.W + (int)(((int64_t)last + 1) / a.P);
  q.tiles = (q.keys + kTileKeys - 1) / kTileKeys;
  return q;
}
// A group of no tiles still takes one unit: its rows are written out empty.
__device__ __forceinline__ int group_units(const Group& q) { return max(1, q.tiles); }

struct Share {
  int64_t lo, hi, per;                           // this CTA's units and the units per CTA
  int row;                                       // the first group's row
  int64_t unit;                                  // its first unit
};

// This CTA's share of the list; every thread of the block takes part.
// s: scratch of 2 * kThreads int64.
__device__ Share find_share(const DenseArgs& a, int G, int64_t* s, Share* out) {
  const int tid = threadIdx.x, R = a.num_rows;
  const int each = (R + kThreads - 1) / kThreads;
  const int r_lo = min(R, tid * each), r_hi = min(R, r_lo + each);
  // the last run start at or before r_lo - 1
  int start = -1;
  for (int r = r_lo; r < r_hi; ++r)
    if (!row_continues(a, r)) start = r;
  int* st = reinterpret_cast<int*>(s);
  st[tid] = start;
  __syncthreads();
  for (int o = 1; o < kThreads; o <<= 1) {       // inclusive running maximum
    const int v = tid >= o ? st[tid - o] : -1;
    __syncthreads();
    st[tid] = max(st[tid], v);
    __syncthreads();
  }
  int run = tid > 0 ? st[tid - 1] : -1;          // start of the run that reaches into this thread's rows
  __syncthreads();
  const int run0 = run;
  int64_t sum = 0;
  for (int r = r_lo; r < r_hi; ++r) {
    if (G > 1 && row_continues(a, r)) {
      if ((r - run) % G != 0) continue;
    } else {
      run = r;
    }
    sum += group_units(group_at(a, r, G));
  }
  s[tid] = sum;
  __syncthreads();
  for (int o = 1; o < kThreads; o <<= 1) {
    const int64_t v = tid >= o ? s[tid - o] : 0;
    __syncthreads();
    s[tid] += v;
    __syncthreads();
  }
  const int64_t total = s[kThreads - 1];
  const int64_t per = (total + gridDim.x - 1) / gridDim.x;
  const int64_t lo = min(total, (int64_t)blockIdx.x * per), hi = min(total, lo + per);
  const int64_t before = s[tid] - sum;
  if (lo < hi && before <= lo && lo < s[tid]) {  // exactly one thread
    run = run0;
    int64_t u = before;
    for (int r = r_lo; r < r_hi; ++r) {
      if (G > 1 && row_continues(a, r)) {
        if ((r - run) % G != 0) continue;
      } else {
        run = r;
      }
      const int n = group_units(group_at(a, r, G));
      if (lo < u + n) {
        out->row = r;
        out->unit = u;
        break;
      }
      u += n;
    }
  }
  __syncthreads();
  Share h = *out;
  h.lo = lo;
  h.hi = hi;
  h.per = per;
  return h;
}

// ---- shared memory ---------------------------------------------------------------------
template <int COLS>
struct Smem {
  uint8_t k[kTileKeys * D * 2];                  // 64-dim atoms of 16 KB: (key/8)*1024 + (key%8)*128
  uint8_t q[COLS * D * 2];                       // 64-dim atoms of COLS * 128 B: (c/8)*1024 + (c%8)*128
  uint8_t q_lo[COLS * 128];                      // low parts of the rotated 64 dims, one such atom
  uint8_t p[kTileKeys * 128];                    // (key/8)*1024 + (key%8)*128, columns along the row
  float mu[kTileKeys];                           // factor of a key's logit and p; < 0: left out
  float factor[COLS];                            // of a column's logits (log2 units)
  float red_max[4][COLS], red_sum[4][COLS];
  float m_buf[2][COLS];
  float m_fin[COLS], l_fin[COLS];
  Share share;
  uint64_t s_bar, pv_bar;
  uint32_t tmem_base;
};

template <int COLS>
__global__ void __launch_bounds__(kThreads, 1) k_dense_attn(DenseArgs a) {
  constexpr int HH = COLS / 4;
  extern __shared__ uint8_t smem_raw[];
  using S = Smem<COLS>;
  S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = lane_id(), warp = warp_id();
  const int G = COLS / a.H;
  pdl_trigger();
  if (tid == 0) {
    mbar_init(&sm.s_bar, 1);
    mbar_init(&sm.pv_bar, 1);
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(&sm.tmem_base, 512);
  const Share sh = find_share(a, G, reinterpret_cast<int64_t*>(sm.p), &sm.share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const uint32_t tS = tmem, tO = tmem + 64;
  const int q4 = warp & 3, hsel = warp >> 2;
  const int mykey = 32 * q4 + lane;
  const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
  const int myc = hsel * HH + (lane < HH ? lane : 0);
  const int key = 8 * warp + (lane & 7), gq = lane >> 3;
  const uint64_t dK = smem_desc(smem_u32(sm.k), 16, 1024, kSwizzle128B);
  const uint64_t dQ = smem_desc(smem_u32(sm.q), 16, 1024, kSwizzle128B);
  const uint64_t dQl = smem_desc(smem_u32(sm.q_lo), 16, 1024, kSwizzle128B);
  const uint64_t dV = smem_desc(smem_u32(sm.k), 16384, 1024, kSwizzle128B);
  const uint64_t dP = smem_desc(smem_u32(sm.p), 8192, 1024, kSwizzle128B);
  bool ok = true;
  uint32_t phase = 0;
  bool cut = false;                              // the last group goes on in the next CTA
  int4 rec = make_int4(-1, 0, 0, 0);
  int64_t unit = sh.unit;
  int row = sh.row;
  for (int64_t u = sh.lo; u < sh.hi && ok;) {
    const Group gr = group_at(a, row, G);
    const int n_units = group_units(gr);
    const int t0 = (int)(u - unit), t1 = (int)min((int64_t)n_units, sh.hi - unit);
    const bool whole = t0 == 0 && t1 == n_units;
    const int tiles_end = min(t1, gr.tiles);
    if (gr.tiles == 0 && !row_valid(a, gr.b, gr.p0) && tid == 0) raise_flag(a.status, CSA_FLAG_ROW_INVALID);
    // ---- queries
    const int cols = gr.g * a.H;
    for (int c = warp; c < COLS; c += kThreads / 32) {
      float f[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = 0.0f;
      if (c < cols) {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + ((size_t)gr.r0 * a.H + c) * D) + 2 * lane;
        const uint4 x = __ldg(src), y = __ldg(src + 1);
        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[2 * i] = __uint_as_float(w[i] << 16);
          f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
        if (a.rope_cos && gr.tiles > 0) {
          float other[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) other[i] = __shfl_xor_sync(0xFFFFFFFFu, f[i], 2);
          if (lane >= 28) {
            const size_t at = (size_t)(gr.p0 + c / a.H) * 32 + 16 * (lane & 1);
            rotate16(f, other, lane < 30, a.rope_cos + at, a.rope_sin + at);
          }
        }
      }
      float big = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) big = fmaxf(big, fabsf(f[i]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
      // 2^-e puts the largest magnitude in [128, 256)
      const int e = (big > 0.0f && big < INFINITY) ? ilogbf(big) - 7 : 0;
      const int e1 = -e / 2, e2 = -e - e1;       // two factors: 2^-e may be past the fp32 range
      const float s1 = __uint_as_float((uint32_t)(e1 + 127) << 23), s2 = __uint_as_float((uint32_t)(e2 + 127) << 23);
      if (lane == 0) sm.factor[c] = ldexpf(a.softmax_scale * kLog2e, e);
      uint32_t o[8], lo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = f[2 * i] * s1 * s2, y = f[2 * i + 1] * s1 * s2;
        const __half2 h = __floats2half2_rn(x, y);
        const float2 hf = __half22float2(h);
        const __half2 r = __floats2half2_rn(x - hf.x, y - hf.y);
        o[i] = *reinterpret_cast<const uint32_t*>(&h);
        lo[i] = *reinterpret_cast<const uint32_t*>(&r);
      }
      if (a.rope_cos && lane >= 28) {
        uint8_t* dl = sm.q_lo + (c >> 3) * 1024;
        *reinterpret_cast<uint4*>(dl + swz128(c & 7, 2 * (lane & 3))) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4*>(dl + swz128(c & 7, 2 * (lane & 3) + 1)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
      }
      uint8_t* dst = sm.q + (lane >> 2) * (COLS * 128) + (c >> 3) * 1024;
      *reinterpret_cast<uint4*>(dst + swz128(c & 7, 2 * (lane & 3))) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(dst + swz128(c & 7, 2 * (lane & 3) + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
    if (tid < COLS) {
      sm.m_buf[0][tid] = -INFINITY;
      sm.m_buf[1][tid] = -INFINITY;
    }
    int mcur = 0;
    float lpart[HH];
#pragma unroll
    for (int i = 0; i < HH; ++i) lpart[i] = 0.0f;
    for (int t = t0; t < tiles_end && ok; ++t) {
      // ---- the tile's keys, dequantised
      {
        const int ki = t * kTileKeys + key;
        uint8_t* krow = sm.k + (key >> 3) * 1024;
        float mu = -1.0f;
        if (ki < gr.W) {
          const int p = gr.wlo + ki;
          const size_t slot = (size_t)gr.b * a.win_cap + (size_t)(p % a.win_cap);
          const float ws = __ldg(a.win_scale + slot);
          int e = -14;
          if (ws > 0.0f) e = min(7, max(-14, ilogbf(ws)));
          mu = ldexpf(ws, -e);
          const __half2 hp = __float2half2_rn(ldexpf(1.0f, e));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 dv = ldg_nc_v4(a.win_codes + slot * D + 16 * gq + 64 * i);
            const uint32_t w4[4] = {dv.x, dv.y, dv.z, dv.w};
            uint32_t o[8];
#pragma unroll
            for (int wd = 0; wd < 4; ++wd) {
              uint32_t f[2];
              e4m3x4_to_f16(w4[wd], f);
              o[2 * wd] = hmul2_u32(f[0], hp);
              o[2 * wd + 1] = hmul2_u32(f[1], hp);
            }
            if (i == 7 && a.rope_cos) {          // dims 448 + 16 gq: lanes gq, gq ^ 2 hold the halves
              // both halves are loaded here: a neighbouring lane may hold an entry
              const uint4 ov = ldg_nc_v4(a.win_codes + slot * D + 16 * (gq ^ 2) + 64 * i);
              const uint32_t v4[4] = {ov.x, ov.y, ov.z, ov.w};
              float mine[16], other[16];
              const float pw = ldexpf(1.0f, e);
#pragma unroll
              for (int wd = 0; wd < 4; ++wd) {
                uint32_t f[2], h[2];
                e4m3x4_to_f16(w4[wd], f);
                e4m3x4_to_f16(v4[wd], h);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f[k]));
                  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
                  mine[4 * wd + 2 * k] = x.x * pw;
                  mine[4 * wd + 2 * k + 1] = x.y * pw;
                  other[4 * wd + 2 * k] = y.x * pw;
                  other[4 * wd + 2 * k + 1] = y.y * pw;
                }
              }
              const size_t at = (size_t)p * 32 + 16 * (gq & 1);
              rotate16(mine, other, gq < 2, a.rope_cos + at, a.rope_sin + at);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const __half2 v = __floats2half2_rn(mine[2 * k], mine[2 * k + 1]);
                o[k] = *reinterpret_cast<const uint32_t*>(&v);
              }
            }
            const int c8 = 2 * (4 * i + gq);
            uint8_t* d = krow + (c8 >> 3) * 16384;
            *reinterpret_cast<uint4*>(d + swz128(key & 7, c8 & 7)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(d + swz128(key & 7, (c8 & 7) + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        } else {
          int pg = -1, slot = 0;
          if (ki < gr.keys) {
            const int e = ki - gr.W;
            pg = __ldg(a.page_table + (size_t)gr.b * a.max_pages + e / PAGE);
            slot = e % PAGE;
            if (pg < 0 || pg >= a.num_pages) {
              raise_flag(a.status, CSA_FLAG_PAGE_OOB);
              pg = -1;
            }
          }
          if (pg >= 0) mu = 1.0f;
          const uint8_t* src = a.kv_pool + (size_t)max(pg, 0) * KV_PAGE;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c16 = 4 * i + gq;
            uint4 dv = make_uint4(0u, 0u, 0u, 0u);
            uint16_t sc = 0;
            if (pg >= 0) {
              dv = ldg_nc_v4(src + slot * 256 + 16 * c16);
              sc = ldg_nc_u16(src + KV_SCALE_OFF + slot * 32 + 2 * c16);
            }
            const uint32_t w4[4] = {dv.x, dv.y, dv.z, dv.w};
            const uint32_t sp = e4m3x2_to_f16(sc);
            const __half2 hs0 = __low2half2(*reinterpret_cast<const __half2*>(&sp));
            const __half2 hs1 = __high2half2(*reinterpret_cast<const __half2*>(&sp));
            uint8_t* d = krow + (c16 >> 1) * 16384;
#pragma unroll
            for (int wd = 0; wd < 4; ++wd) {
              uint32_t f[4];
              e2m1x8_to_f16(w4[wd], f);
#pragma unroll
              for (int k = 0; k < 4; ++k) f[k] = hmul2_u32(f[k], wd < 2 ? hs0 : hs1);
              *reinterpret_cast<uint4*>(d + swz128(key & 7, (c16 & 1) * 4 + wd)) = make_uint4(f[0], f[1], f[2], f[3]);
            }
          }
        }
        if (gq == 0) sm.mu[key] = mu;
      }
      // ---- S^T
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
        constexpr uint32_t id = idesc_f16(128, COLS, 0, 0);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_f16(tS, dK + (uint64_t)((ks >> 2) * 1024 + (ks & 3) * 2),
                  dQ + (uint64_t)((ks >> 2) * (COLS * 8) + (ks & 3) * 2), id, ks > 0 ? 1u : 0u);
        if (a.rope_cos) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_f16(tS, dK + (uint64_t)(7 * 1024 + ks * 2), dQl + (uint64_t)(ks * 2), id, 1u);
        }
        tc_commit(&sm.s_bar);
      }
      __syncwarp();
      if (__syncthreads_or(!mbar_wait_for(&sm.s_bar, phase, a.wait_budget))) {
        ok = false;
        break;
      }
      tc_fence_after();
      // ---- softmax
      float lg[HH];
      tmem_ld_n<HH>(tS + lane_off + hsel * HH, lg);
      const float mu = sm.mu[mykey];
      // the group's rows that see this key
      int ilo = 0, ihi = -1;
      {
        const int ki = t * kTileKeys + mykey;
        if (mu >= 0.0f) {
          if (ki < gr.W) {
            ilo = max(0, gr.wlo + ki - gr.p0);
            ihi = min(gr.g - 1, gr.wlo + ki + (WIN - 1) - gr.p0);
          } else {
            ilo = (int)max((int64_t)0, (int64_t)a.P * (ki - gr.W + 1) - 1 - gr.p0);
            ihi = gr.g - 1;
          }
        }
      }
      const int clo = ilo * a.H - hsel * HH, chi = (ihi + 1) * a.H - hsel * HH;
#pragma unroll
      for (int i = 0; i < HH; ++i)
        lg[i] = (i >= clo && i < chi) ? lg[i] * (mu * sm.factor[hsel * HH + i]) : -INFINITY;
      const float* mr = sm.m_buf[mcur] + hsel * HH;
      bool need = false;
#pragma unroll
      for (int i = 0; i < HH; ++i) need |= lg[i] > mr[i] + kRescaleLog2;
      need = group_sync_or(1 + hsel, need);
      float mi[HH];
      if (need) {
        float tmp[HH];
#pragma unroll
        for (int i = 0; i < HH; ++i) tmp[i] = lg[i];
        constexpr int kShift = RedShift<HH>::v;
        const float mx = warp_reduce_many<HH, true>(tmp, lane);
        if ((lane & ((1 << kShift) - 1)) == 0) sm.red_max[q4][hsel * HH + (lane >> kShift)] = mx;
        group_sync(5 + hsel);
        const float tmax = fmaxf(fmaxf(sm.red_max[0][myc], sm.red_max[1][myc]),
                                 fmaxf(sm.red_max[2][myc], sm.red_max[3][myc]));
        const float mold = sm.m_buf[mcur][myc];
        const float mnew = (mold == -INFINITY || tmax > mold + kRescaleLog2) ? tmax : mold;
        const float alpha = mold == -INFINITY ? 0.0f : (mnew == mold ? 1.0f : exp2f(mold - mnew));
        if (q4 == 0 && lane < HH) sm.m_buf[mcur ^ 1][myc] = mnew;
        bool moved = false;
        float al[HH];
#pragma unroll
        for (int i = 0; i < HH; ++i) {
          mi[i] = __shfl_sync(0xFFFFFFFFu, mnew, i);
          al[i] = __shfl_sync(0xFFFFFFFFu, alpha, i);
          lpart[i] *= al[i];
          moved |= al[i] != 1.0f;
        }
        if (t > t0 && moved) {
#pragma unroll 1
          for (int dc = 0; dc < D / 128; ++dc) {
            float v[HH];
            const uint32_t ta = tO + lane_off + dc * 64 + hsel * HH;
            tmem_ld_n<HH>(ta, v);
#pragma unroll
            for (int i = 0; i < HH; ++i) v[i] *= al[i];
            tmem_st_n<HH>(ta, v);
          }
          tmem_st_wait();
        }
        mcur ^= 1;
      } else {
#pragma unroll
        for (int i = 0; i < HH; ++i) mi[i] = mr[i];
      }
      {
        const float fm = fmaxf(mu, 0.0f);
        uint32_t packed[HH / 2];
#pragma unroll
        for (int i = 0; i < HH; i += 2) {
          const float p0 = (lg[i] == -INFINITY) ? 0.0f : exp2f(lg[i] - mi[i]);
          const float p1 = (lg[i + 1] == -INFINITY) ? 0.0f : exp2f(lg[i + 1] - mi[i + 1]);
          lpart[i] += p0;
          lpart[i + 1] += p1;
          const __half2 hv = __floats2half2_rn(p0 * fm, p1 * fm);
          packed[i / 2] = *reinterpret_cast<const uint32_t*>(&hv);
        }
        uint8_t* prow = sm.p + (mykey >> 3) * 1024;
        const int chunk = (hsel * HH) / 8;
        if constexpr (HH >= 8) {
#pragma unroll
          for (int c = 0; c < HH / 8; ++c)
            *reinterpret_cast<uint4*>(prow + swz128(mykey & 7, chunk + c)) =
                make_uint4(packed[4 * c], packed[4 * c + 1], packed[4 * c + 2], packed[4 * c + 3]);
        } else {
          *reinterpret_cast<uint2*>(prow + swz128(mykey & 7, chunk) + 8 * (hsel & 1)) = make_uint2(packed[0], packed[1]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      // ---- O^T += V^T P^T
      if (tid == 0) {
        tc_fence_after();
        constexpr uint32_t id = idesc_f16(128, COLS, 1, 1);
#pragma unroll
        for (int dc = 0; dc < D / 128; ++dc)
#pragma unroll
          for (int ks = 0; ks < kTileKeys / 16; ++ks)
            mma_f16(tO + dc * 64, dV + (uint64_t)(dc * 2048 + ks * 128), dP + (uint64_t)(ks * 128), id,
                    (ks > 0 || t > t0) ? 1u : 0u);
        tc_commit(&sm.pv_bar);
      }
      __syncwarp();
      if (__syncthreads_or(!mbar_wait_for(&sm.pv_bar, phase, a.wait_budget))) ok = false;
      phase ^= 1;
    }
    if (!ok) break;
    // ---- the columns' sums
    {
      constexpr int kShift = RedShift<HH>::v;
      const float sum = warp_reduce_many<HH, false>(lpart, lane);
      if ((lane & ((1 << kShift) - 1)) == 0) sm.red_sum[q4][hsel * HH + (lane >> kShift)] = sum;
      group_sync(1 + hsel);
      if (q4 == 0 && lane < HH) {
        sm.l_fin[myc] = (sm.red_sum[0][myc] + sm.red_sum[1][myc]) + (sm.red_sum[2][myc] + sm.red_sum[3][myc]);
        sm.m_fin[myc] = sm.m_buf[mcur][myc];
      }
    }
    tc_fence_after();
    __syncthreads();
    // ---- out: thread = dim 128 * hsel + 32 * q4 + lane
    const int d = 128 * hsel + mykey;
    const bool have = tiles_end > t0;
    const int slot = t0 > 0 ? 2 * blockIdx.x : 2 * blockIdx.x + 1;
    for (int c0 = 0; c0 < cols; c0 += 16) {
      uint32_t v[16];
      if (have) {
        tmem_ld16(tO + lane_off + hsel * 64 + c0, v);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0u;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (whole) {
          const float l = sm.l_fin[c0 + i];
          const float o = l == 0.0f ? 0.0f : __uint_as_float(v[i]) / l;
          const __nv_bfloat16 ob = __float2bfloat16_rn(o);
          a.out[((size_t)gr.r0 * a.H + c0 + i) * D + d] = *reinterpret_cast<const uint16_t*>(&ob);
        } else {
          __stcg(a.part + ((size_t)slot * COLS + c0 + i) * D + d, __uint_as_float(v[i]));
        }
      }
    }
    if (tid < cols) {
      const float l = sm.l_fin[tid], m = sm.m_fin[tid];
      if (whole) {
        if (a.lse) a.lse[(size_t)gr.r0 * a.H + tid] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
      } else {
        a.part_ml[(size_t)slot * 2 * COLS + tid] = m;
        a.part_ml[(size_t)slot * 2 * COLS + COLS + tid] = l;
      }
    }
    if (!whole && t0 == 0) {
      cut = true;
      rec = make_int4(gr.r0, gr.g, blockIdx.x, (int)((unit + n_units - 1) / sh.per));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    u = unit + t1;
    unit += n_units;
    row += gr.g;
  }
  if (tid == 0) {
    if (!ok) raise_flag(a.status, CSA_FLAG_TIMEOUT);
    a.rec[blockIdx.x] = cut && ok ? rec : make_int4(-1, 0, 0, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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
  float M = -INFINITY;
  for (int q = 0; q < n; ++q) M = fmaxf(M, __ldcg(a.part_ml + (size_t)slot(q) * 2 * cols_max + c));
  float L = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int q = 0; q < n; ++q) {
    const float* ml = a.part_ml + (size_t)slot(q) * 2 * cols_max + c;
    const float m = __ldcg(ml), l = __ldcg(ml + cols_max);
    const float w = m == -INFINITY ? 0.0f : exp2f(m - M);
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
  const size_t smem = sizeof(Smem<COLS>) + 1024;
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
