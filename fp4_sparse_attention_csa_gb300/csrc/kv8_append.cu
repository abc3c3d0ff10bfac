// csa_kv8_append: new tokens' keys and values into the 8-bit paged cache.
//
// Mathematics.  Of a page's tokens x (keys k' = bf16(rotation of k), values v; the page's
// earlier tokens from the bf16 tail): s = amax / 448, code = E4M3(x * (448 / amax)); the
// summary is the mean m of the 64 slots' keys (a binary tree of fp32 sums of k' / 64), its
// codes rint(m * (127 / max|m|)).  A page is quantised whole at every append, so its bytes are
// a function of its tokens.
//
// One CTA per touched page and head, 2 D threads.  A thread holds 8 dims of 4 consecutive
// slots, keys and values (8 loads of 16 bytes, all asked for at once), so the amax is one
// exchange between the warps, the first two levels of the summary's tree are the thread's
// own and the next are its warp's, and four slots of a dim are one word of the transposed
// values.  Codes go through shared memory, padded so that neither side conflicts, and out
// in 16-byte pieces.
//
// What bounds it.  A small call: one dependent chain (offsets, page, tokens, amax, codes) in
// each CTA, 4.7 us for a token of 8 heads of 128.  128 requests' single tokens take 13.8 us, 2.5
// TB/s of the bytes that they must move: the chain again, in 1024 CTAs of which 608 run at once (a
// warp for the search alone took 19.9 us).  A prompt's 4 x 4001 tokens with half of each key rotated
// take 39 us, 2.7 TB/s: a warp issues 1360 instructions a page for rotation, amax, sums and codes, in
// 59 % of the issue slots.
//
// The tail is read and written by one call: a page's CTA reads the slots of its earlier
// tokens, and new tokens land in slots p % 128.  Only the first page of a request has
// earlier tokens, and slots of pages an even distance apart coincide; so the first page's
// CTA writes the later pages of its parity as well, after its own reads.
#include <algorithm>

#include "kv8_device.cuh"

namespace csa {

namespace {

struct Unit {
  int b, j;                                      // request and page
  int pos0, n, off;                              // its tokens: first position, how many, first input row
};

// A request's new tokens, n = 0 when there are none or they do not fit.
__device__ __forceinline__ Unit tokens_of(const Kv8AppendArgs& a, int b, bool* bad) {
  Unit u;
  u.b = b;
  u.pos0 = __ldg(a.pos0 + b);
  u.off = __ldg(a.tok_off + b);
  const int64_t end = __ldg(a.tok_off + b + 1), n = end - u.off;
  const int64_t last = (int64_t)u.pos0 + n;
  *bad = n < 0 || u.off < 0 || end > a.total_tokens ||
         (n > 0 && (u.pos0 < 0 || last > (int64_t)a.max_pages * PAGE || last > kKv8MaxPos ||
                    (a.rope.cos != nullptr && last > a.rope.rows)));
  u.n = *bad ? 0 : (int)n;
  u.j = u.n > 0 ? u.pos0 >> 6 : 0;
  return u;
}
__device__ __forceinline__ int pages_of(const Unit& u) {
  return u.n > 0 ? ((u.pos0 + u.n - 1) >> 6) - (u.pos0 >> 6) + 1 : 0;
}

// The at-th touched page over all requests, to s_unit and its pool page to s_page; false past the
// last.  Every thread takes part, one request each at a time.
template <int T>
__device__ __forceinline__ bool find_unit(const Kv8AppendArgs& a, int at, int* s_sums, Unit* s_unit, int* s_page) {
  const int tid = threadIdx.x, lane = lane_id(), warp = warp_id();
  int before = 0;
#pragma unroll 1
  for (int base = 0; base < a.num_requests; base += T) {
    Unit mine{};
    bool bad;
    if (base + tid < a.num_requests) mine = tokens_of(a, base + tid, &bad);
    const int count = pages_of(mine);
    int upto = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s_sums[warp] = upto;
    __syncthreads();
    int total = before;
    upto += before;
#pragma unroll
    for (int w = 0; w < T / 32; w += 4) {
      const int4 s = *reinterpret_cast<const int4*>(s_sums + w);
      const int each[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (w + k < warp) upto += each[k];
        total += each[k];
      }
    }
    if (at >= upto - count && at < upto) {
      mine.j += at - (upto - count);
      *s_unit = mine;
      *s_page = __ldg(a.page_table + (size_t)mine.b * a.max_pages + mine.j);
    }
    __syncthreads();
    if (at < total) return true;
    before = total;
  }
  return false;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// Pair k of eight bf16.
__device__ __forceinline__ float2 pair_of(uint4 v, int k) {
  const uint32_t w = k == 0 ? v.x : (k == 1 ? v.y : (k == 2 ? v.z : v.w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <int D>
struct AppendSmem {
  static constexpr int kKeyStride = D / 16 * 144;          // 8 slots: 16-byte pieces of 8 rows, 144 apart
  static constexpr int kValueStride = 528;                 // 8 dims: 4 x 128 bytes
  uint8_t k[8 * kKeyStride];
  uint8_t v[D / 8 * kValueStride];
  float sum[2 * D / 32][D];
  float top[2][2 * D / 32];                      // 16-byte pieces
  int sums[2 * D / 32];
  Unit unit;
  int page;
};

template <int D>
__global__ void __launch_bounds__(2 * D, 1024 / (2 * D)) k_kv8_append(Kv8AppendArgs a) {
  constexpr int T = 2 * D, kPieces = D / 8, kWarps = T / 32;
  __shared__ __align__(16) AppendSmem<D> sm;
  const int tid = threadIdx.x, lane = lane_id(), warp = warp_id(), h = blockIdx.y, H = a.heads;
  const int i0 = 8 * (tid % kPieces), t0 = 4 * (tid / kPieces);   // the thread's dims and slots
  if (blockIdx.x == 0 && h == 0) {               // requests that are left out
    bool any = tid == 0 && (__ldg(a.tok_off) != 0 || __ldg(a.tok_off + a.num_requests) != a.total_tokens);
    for (int b = tid; b < a.num_requests; b += T) {
      bool bad;
      (void)tokens_of(a, b, &bad);
      any |= bad;
    }
    if (any) raise_flag(a.status, CSA_FLAG_APPEND);
  }
  for (int at = blockIdx.x;; at += gridDim.x) {
    if (!find_unit<T>(a, at, sm.sums, &sm.unit, &sm.page)) return;
    const Unit u = sm.unit;
    const int last = u.pos0 + u.n - 1, j0 = u.pos0 >> 6;
    uint16_t* tail = a.tail + ((size_t)u.b * H + h) * 2 * kKv8Tail * D;   // keys, then values
    const int page = sm.page;
    // ---- the thread's dims of its slots: new, earlier, or none; all asked for before any is used.  A warp
    // whose slots lie behind the last token has zeros and nothing to do for them.
    uint4 raw[2][4];
    uint32_t is_new = 0, nan = 0;
    const bool some = u.j * PAGE + 4 * (32 * warp / kPieces) <= last;
    float top[2] = {0.0f, 0.0f}, sum[8] = {};
    if (some) {
      const size_t step = (size_t)H * D;
      const int p0 = u.j * PAGE + t0;
      const size_t row = ((int64_t)u.off + (p0 - u.pos0)) * (int64_t)step + (size_t)h * D + i0;
      const uint16_t* old = tail + (size_t)(p0 & (kKv8Tail - 1)) * D + i0;     // 4 slots do not wrap
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bool is_old = p0 + s < u.pos0;
        raw[0][s] = raw[1][s] = make_uint4(0u, 0u, 0u, 0u);
        if (p0 + s <= last) {
          if (!is_old) is_new |= 1u << s;
          raw[0][s] = *reinterpret_cast<const uint4*>(is_old ? old + s * D : a.k_in + row + s * step);
          raw[1][s] = *reinterpret_cast<const uint4*>(is_old ? old + (kKv8Tail + s) * D : a.v_in + row + s * step);
        }
      }
      if (a.rope.cos != nullptr) {               // a pair's other half is another lane's of the same row
        Kv8Turn turn{i0, 0, false};
        const bool turns = turn_of(a.rope, i0, turn);
        const int from = lane + (turn.other - i0) / 8;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint4 other = of_lane(raw[0][s], from);
          if (turns && ((is_new >> s) & 1u)) raw[0][s] = turn8(raw[0][s], other, a.rope, turn, p0 + s);
        }
      }
      // ---- new tokens to the tail: slots of this page that no one reads
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int p = u.j * PAGE + t0 + t;
        if (((is_new >> t) & 1u) && p > last - kKv8Tail && (u.j == j0 || ((u.j - j0) & 1))) {
          uint16_t* dst = tail + (size_t)(p & (kKv8Tail - 1)) * D + i0;
          *reinterpret_cast<uint4*>(dst) = raw[0][t];
          *reinterpret_cast<uint4*>(dst + kKv8Tail * D) = raw[1][t];
        }
      }
      // ---- amax of both sides; tokens that are not all numbers count as zeros from here on
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float k = __low2float(bf16x8_top(raw[0][t])), v = __low2float(bf16x8_top(raw[1][t]));
        const uint32_t row = ((1u << kPieces) - 1u) << (lane / kPieces * kPieces);
        const bool bad = !(k <= 3.4028234663852886e38f) || !(v <= 3.4028234663852886e38f);
        if (__ballot_sync(0xFFFFFFFFu, bad) & row) {
          nan |= 1u << t;
          raw[0][t] = raw[1][t] = make_uint4(0u, 0u, 0u, 0u);
        } else {
          top[0] = fmaxf(top[0], k);
          top[1] = fmaxf(top[1], v);
        }
      }
      // ---- the keys' sums: slots 4 at a time, then the warp's; each over 64 before the sums, which could overflow
      constexpr float f = 1.0f / PAGE;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f2 = make_float2(f, f);
        const float2 s = add2(fma2(pair_of(raw[0][1], k), f2, mul2(pair_of(raw[0][0], k), f2)),
                              fma2(pair_of(raw[0][3], k), f2, mul2(pair_of(raw[0][2], k), f2)));
        sum[2 * k] = s.x;
        sum[2 * k + 1] = s.y;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int o = kPieces; o < 32; o <<= 1) sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], o);
    }
    if (lane < kPieces) {
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<float4*>(&sm.sum[warp][i0 + i]) = make_float4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float t = warp_top(top[k]);
      if (lane == 0) sm.top[k][warp] = t;
    }
    __syncthreads();                             // the tail has been read, too
    float amax[2], inv[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      amax[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; w += 4) {
        const float4 t = *reinterpret_cast<const float4*>(&sm.top[k][w]);
        amax[k] = fmaxf(amax[k], fmaxf(fmaxf(t.x, t.y), fmaxf(t.z, t.w)));
      }
      if (!(amax[k] >= kKv8Least)) amax[k] = 0.0f;
      inv[k] = amax[k] > 0.0f ? __fdiv_rn(448.0f, amax[k]) : 0.0f;
    }
    // ---- and later pages' to the slots that this page's earlier tokens had
    if (u.j == j0) {
      const int from = max(last - kKv8Tail + 1, (j0 + 2) * PAGE);
      for (int p = from + tid / kPieces; p <= last; p += T / kPieces) {
        if (((p >> 6) - j0) & 1) continue;
        const size_t row = ((size_t)(u.off + (p - u.pos0)) * H + h) * D;
        uint16_t* dst = tail + (size_t)(p & (kKv8Tail - 1)) * D + i0;
        *reinterpret_cast<uint4*>(dst) = rotated8(a.k_in + row, i0, a.rope, p);
        *reinterpret_cast<uint4*>(dst + kKv8Tail * D) = __ldg(reinterpret_cast<const uint4*>(a.v_in + row + i0));
      }
    }
    const bool in_pool = (uint32_t)page < (uint32_t)a.num_pages;
    if (!in_pool) {
      if (tid == 0) raise_flag(a.status, CSA_FLAG_PAGE_OOB);
      __syncthreads();
      continue;
    }
    // ---- codes
    if (some) {
      uint32_t vc[4][4];                         // [slot][pair of dims]
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t kc[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 k = mul2(pair_of(raw[0][s], i), make_float2(inv[0], inv[0]));
          const float2 v = mul2(pair_of(raw[1][s], i), make_float2(inv[1], inv[1]));
          const uint32_t c = e4m3x2_of(k.x, k.y);
          kc[i >> 1] = (i & 1) ? kc[i >> 1] | (c << 16) : c;
          vc[s][i] = e4m3x2_of(v.x, v.y);
        }
        if ((nan >> s) & 1u) kc[0] = kc[1] = 0x7F7F7F7Fu;
        const int t = t0 + s;
        *reinterpret_cast<uint2*>(sm.k + (t >> 3) * AppendSmem<D>::kKeyStride + (i0 >> 4) * 144 + (t & 7) * 16 +
                                  (i0 & 15)) = make_uint2(kc[0], kc[1]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {                // two dims: four slots each
        const uint32_t lo = __byte_perm(vc[0][i], vc[1][i], 0x5140), hi = __byte_perm(vc[2][i], vc[3][i], 0x5140);
        uint8_t* dst = sm.v + (i0 >> 3) * AppendSmem<D>::kValueStride + (t0 >> 4) * 128 + 2 * i * 16 + (t0 & 15);
        *reinterpret_cast<uint32_t*>(dst) = __byte_perm(lo, hi, 0x5410);
        *reinterpret_cast<uint32_t*>(dst + 16) = __byte_perm(lo, hi, 0x7632);
      }
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int t = t0 + s;
        *reinterpret_cast<uint2*>(sm.k + (t >> 3) * AppendSmem<D>::kKeyStride + (i0 >> 4) * 144 + (t & 7) * 16 +
                                  (i0 & 15)) = make_uint2(0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint32_t*>(sm.v + (i0 >> 3) * AppendSmem<D>::kValueStride + (t0 >> 4) * 128 + i * 16 +
                                     (t0 & 15)) = 0u;
    }
    __syncthreads();
    uint8_t* rec = a.pool + kv8_record<D>(page, H, h);
#pragma unroll
    for (int i = tid; i < 4 * D; i += T) {       // 16-byte pieces of the keys, then of the values
      const int g = i / (D / 2), rest = i % (D / 2);       // a group of 8 slots: D / 16 blocks of 8 pieces
      *reinterpret_cast<uint4*>(rec + 16 * i) = *reinterpret_cast<const uint4*>(
          sm.k + g * AppendSmem<D>::kKeyStride + (rest >> 3) * 144 + (rest & 7) * 16);
      *reinterpret_cast<uint4*>(rec + 64 * D + 16 * i) =
          *reinterpret_cast<const uint4*>(sm.v + (i >> 5) * AppendSmem<D>::kValueStride + (i & 31) * 16);
    }
    if (tid < 32)
      reinterpret_cast<float*>(rec + 128 * D)[tid] = tid < 2 ? __fdiv_rn(tid == 0 ? amax[0] : amax[1], 448.0f) : 0.0f;
    // ---- summary, by the last warp
    if (a.sum_codes != nullptr && warp == kWarps - 1) {
      constexpr int N = D / 32;
      float m[N], big = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float w[kWarps];
#pragma unroll
        for (int k = 0; k < kWarps; ++k) w[k] = sm.sum[k][N * lane + i];
#pragma unroll
        for (int o = 1; o < kWarps; o <<= 1)
#pragma unroll
          for (int k = 0; k < kWarps; k += 2 * o) w[k] = w[k] + w[k + o];
        m[i] = w[0];
        big = fmaxf(big, fabsf(m[i]));
      }
      big = warp_top(big);
      const bool some = big >= kKv8Least;
      const float f = some ? __fdiv_rn(127.0f, big) : 0.0f;
      uint32_t packed = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = max(-127, min(127, __float2int_rn(m[i] * f)));
        packed |= (uint32_t)(c & 255) << (8 * i);
      }
      int8_t* dst = a.sum_codes + ((size_t)page * H + h) * D + N * lane;
      if constexpr (N == 4) *reinterpret_cast<uint32_t*>(dst) = packed;
      else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)packed;
      if (lane == 0) a.sum_scale[(size_t)page * H + h] = some ? __fdiv_rn(big, 127.0f) : 0.0f;
    }
    __syncthreads();                             // shared memory is the next page's
  }
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t stream) {
  // touched pages: at most one per token, and n tokens touch at most n / 64 + 2
  const int64_t T = a.total_tokens, B = std::min<int64_t>(a.num_requests, T);
  const int64_t units = std::min(T, T / PAGE + 2 * B);
  const dim3 grid((unsigned)std::min<int64_t>(units, 1 << 16), (unsigned)a.heads);
  if (a.dim == 64) return launch_kernel(Order::kStream, k_kv8_append<64>, grid, dim3(128), 0, stream, a);
  return launch_kernel(Order::kStream, k_kv8_append<128>, grid, dim3(256), 0, stream, a);
}

}  // namespace csa
