// Paged key/value cache: its plan, writing it and reading it back.
//
// The plan (one CTA, no host synchronisation) checks a call's sequences and lists the attention's
// work: the steps' key tiles and the chunk items, each with the running sum of its key tiles, so
// that a kernel can deal the key tiles out evenly whatever the sequences are.
//
// Writing quantizes each (token, head) row by itself, the per-token form of the operand quantizer:
// a later token changes no earlier one's code.  e = least integer with amax <= 448 2^e.
// Both directions move every byte once and are bound by memory: a warp takes a token's rows (of
// all heads, K and V), 16 bytes a lane and load, four loads in flight.
#include <type_traits>

#include "cache.cuh"

namespace flamia {

namespace {

constexpr int kPlanThreads = 1024;

// Block-wide exclusive scan of one value per thread; the block's total in *total.
__device__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const int64_t before = (warp > 0 ? warp_sums[warp - 1] : 0) + x - v;
  *total = warp_sums[31];
  __syncthreads();
  return before;
}

__global__ void __launch_bounds__(kPlanThreads)
    cache_plan_kernel(const int32_t* __restrict__ cu, const int32_t* __restrict__ kv, int N, int T, int hq, int hkv,
                      int max_chunk, int64_t max_kv, int left, void* plan) {
  __shared__ int64_t warp_sums[32];
  __shared__ int s_bad;
  const CachePlanView pv = cache_plan_view(plan, T, N, hq, hkv);
  const int group = hq / hkv, limit = step_rows(group, max_chunk);
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  for (int n = threadIdx.x; n < N; n += kPlanThreads) {
    const int a = cu[n], b = cu[n + 1];
    int bad = 0;
    if (b < a || (n == 0 && a != 0) || (n == N - 1 && b > T)) bad |= FLAMIA_DEV_BAD_CU_SEQLENS;
    else if (b - a > max_chunk) bad |= FLAMIA_DEV_CAPACITY;
    else if (b > a && (kv[n] < b - a || kv[n] > max_kv)) bad |= FLAMIA_DEV_BAD_KV_LENS;
    if (bad) atomicOr(&s_bad, bad);
  }
  __syncthreads();
  const int bad = s_bad;
  if (threadIdx.x == 0) {
    int* h = pv.hdr;
    h[kCpStatus] = bad;
    h[kCpNumSeqs] = N;
    h[kCpTotal] = T;
    h[kCpHkv] = hkv;
    h[kCpHq] = hq;
    h[kCpMaxChunk] = max_chunk;
    h[kCpLeft] = left;
    h[kCpValid] = bad || N == 0 ? 0 : cu[N];
    *reinterpret_cast<int64_t*>(h + kCpStepPlaces) = *reinterpret_cast<int64_t*>(h + kCpChunkPlaces) = 0;
    h[kCpStepCtas] = h[kCpChunkCtas] = 0;
  }
  for (int i = threadIdx.x; i < kDone; i += kPlanThreads) pv.done[i] = 0;
  if (bad || N == 0) return;
  // sequences; steps with their places; chunk items before each sequence
  int64_t step_places = 0, steps = 0, items = 0;
  for (int base = 0; base < N; base += kPlanThreads) {
    const int n = base + threadIdx.x;
    int4 r = make_int4(0, 0, 0, 0);
    int64_t st = 0, it = 0;
    int tile = 0, row_tiles = 0;
    if (n < N) {
      r.x = cu[n];
      r.y = cu[n + 1] - r.x;
      if (r.y > 0) {
        r.z = kv[n];
        r.w = left < 0 ? 0 : max(0, r.z - r.y - left);
        const int64_t rows = (int64_t)r.y * group;
        tile = r.w / kStepTile;
        if (rows <= limit) {
          st = (r.z + kStepTile - 1) / kStepTile - tile + kStepExtra;
          row_tiles = (int)(rows + kStepRows - 1) / kStepRows;
        } else it = (rows + kChunkRows - 1) / kChunkRows;
      }
      pv.seq[n] = r;
    }
    int64_t tot;
    const int64_t places = step_places + block_scan(st * row_tiles, warp_sums, &tot);
    step_places += tot;
    const int64_t number = steps + block_scan(row_tiles, warp_sums, &tot);
    steps += tot;
    for (int t = 0; t < row_tiles; ++t) {
      pv.items[1][number + t] = CacheItem{n, t * kStepRows, tile, (int)st - kStepExtra};
      pv.prefix[1][number + t] = places + t * st;
    }
    const int64_t b = block_scan(it, warp_sums, &tot);
    if (n < N) pv.base[n] = items + b;
    items += tot;
  }
  if (threadIdx.x == 0) {
    pv.prefix[1][steps] = step_places;
    pv.base[N] = items;
  }
  __syncthreads();
  int64_t chunk_places = 0;
  for (int64_t base = 0; base < items; base += kPlanThreads) {
    const int64_t i = base + threadIdx.x;
    int cost = 0;
    if (i < items) {
      int lo = 0, hi = N;          // base[lo] <= i < base[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pv.base[mid] <= i) lo = mid; else hi = mid;
      }
      const int4 r = pv.seq[lo];
      CacheItem x;
      x.seq = lo;
      x.row = (int)(i - pv.base[lo]) * kChunkRows;
      const int64_t rows = (int64_t)r.y * group;
      const int last = (int)(min((int64_t)x.row + kChunkRows, rows) - 1) / group;
      const int first = r.z - r.y + x.row / group;
      x.tile = (left < 0 ? 0 : max(0, first - left)) / kTile;
      x.tiles = (r.z - r.y + last) / kTile - x.tile + 1;
      cost = x.tiles + kChunkExtra;
      pv.items[0][i] = x;
    }
    int64_t tot;
    const int64_t a = block_scan(cost, warp_sums, &tot);
    if (i < items) pv.prefix[0][i] = chunk_places + a;
    chunk_places += tot;
  }
  if (threadIdx.x == 0) pv.prefix[0][items] = chunk_places;
  __syncthreads();
  // shares: the CTAs that get one, and the unit that each begins in
  auto shares = [&](auto STEP, int64_t total, int64_t n_items, int least, int ctas, int c) {
    constexpr int kStep = decltype(STEP)::value;
    Shares sh;
    sh.total = total;
    sh.n = (int)min((int64_t)ctas, (total + least - 1) / least);
    if (c == 0) {
      *reinterpret_cast<int64_t*>(pv.hdr + (kStep ? kCpStepPlaces : kCpChunkPlaces)) = total;
      pv.hdr[kStep ? kCpStepCtas : kCpChunkCtas] = sh.n;
    }
    if (c >= sh.n) return;
    const int64_t f = sh.begin(c);
    int64_t lo = 0, hi = n_items;          // prefix[lo] hkv <= f < prefix[hi] hkv
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (pv.prefix[kStep][mid] * hkv <= f) lo = mid; else hi = mid;
    }
    CachedUnit u = cached_item<kStep != 0>(pv, (int)lo, hq, hkv);
    const int len = u.tiles + (kStep ? kStepExtra : kChunkExtra);
    u.h = (int)((f - u.begin) / len);
    u.begin += (int64_t)u.h * len;
    pv.first[kStep][c] = u;
  };
  // A CTA takes some places at least: fewer would cost more in joining than they save.
  if (threadIdx.x < kStepCtas)
    shares(std::integral_constant<int, 1>{}, step_places * hkv, steps, 4 + kStepExtra, kStepCtas, threadIdx.x);
  else if (threadIdx.x < kStepCtas + kChunkCtas)
    shares(std::integral_constant<int, 0>{}, chunk_places * hkv, items, 2 + kChunkExtra, kChunkCtas, threadIdx.x - kStepCtas);
}

// ---------------------------------------------------------------- write, read
constexpr int kWarps = 8;
constexpr int kRowsPerWarp = 16;      // of a token's 2 hkv rows

// A warp's token and where its rows live: false where there is nothing to do.
struct TokenPlace {
  int token, first;      // first of its rows
  bool tail;             // behind the last sequence, or its page is none
  int64_t base;          // row of kv head 0 in the pools
};
__device__ __forceinline__ bool place_token(const CacheParams& p, TokenPlace& t) {
  const int parts = (2 * p.hkv + kRowsPerWarp - 1) / kRowsPerWarp;
  const int64_t job = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (job >= (int64_t)p.T * parts) return false;
  t.token = (int)(job / parts);
  t.first = (int)(job % parts) * kRowsPerWarp;
  t.tail = t.token >= cache_valid_rows(p);
  t.base = 0;
  if (t.tail) return true;
  const int4* seq = reinterpret_cast<const int4*>(p.plan + kCpHeaderWords);
  const int n = warp_upper(p.N, t.token, [&](int i) { return seq[i].x; });
  const int4 r = seq[n];
  const int pos = r.z - r.y + t.token - r.x;
  const int page = cache_page(p, n, pos >> p.page_shift);
  t.tail = page < 0;
  t.base = ((int64_t)page * p.hkv << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
  return true;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) cache_write_kernel(const CacheParams p, const uint4* __restrict__ k,
                                                                  const uint4* __restrict__ v) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;      // lanes a row, rows a load
  TokenPlace t;
  if (!place_token(p, t) || t.tail) return;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, seg = lane % kLanes;
  const int rows = min(2 * p.hkv, t.first + kRowsPerWarp);
  constexpr int kUnroll = 4;
  for (int r0 = t.first; r0 < rows; r0 += kUnroll * kPer) {
    uint4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kPer + sub, h = r < p.hkv ? r : r - p.hkv;
      x[u] = r < rows ? ((r < p.hkv ? k : v)[((int64_t)t.token * p.hkv + h) * kLanes + seg]) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kPer + sub, h = r < p.hkv ? r : r - p.hkv;
      const int64_t at = t.base + ((int64_t)h << p.page_shift);
      uint8_t* pool = r < p.hkv ? p.k : p.v;
      if constexpr (E4M3) {
        // the largest magnitude by its bits: a NaN's are above infinity's
        const uint32_t m7 = 0x7fff7fffu;
        uint32_t m = __vmaxu2(__vmaxu2(x[u].x & m7, x[u].y & m7), __vmaxu2(x[u].z & m7, x[u].w & m7));
        m = max(m & 0xffffu, m >> 16);
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool nan = m > 0x7f80u;
        const int e = nan ? 128 : roundup_exp(__uint_as_float(m << 16));
        const float inv = nan ? 0.f : exp2i(-e);
        uint32_t c[4];
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = __uint_as_float(w[i] << 16) * inv, b = __uint_as_float(w[i] & 0xffff0000u) * inv;
          c[i] = nan ? 0u : e4m3x2(a, b);
        }
        if (r < rows) {
          *reinterpret_cast<uint2*>(pool + at * D + seg * 8) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
          if (seg == 0) (r < p.hkv ? p.k_scales : p.v_scales)[at] = (uint8_t)(e + 127);
        }
      } else if (r < rows) {
        *reinterpret_cast<uint4*>(pool + (at * D + seg * 8) * 2) = x[u];
      }
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) cache_read_kernel(const CacheParams p, uint4* __restrict__ k,
                                                                 uint4* __restrict__ v) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;
  TokenPlace t;
  if (!place_token(p, t)) return;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, seg = lane % kLanes;
  const int rows = min(2 * p.hkv, t.first + kRowsPerWarp);
  constexpr int kUnroll = 4;
  for (int r0 = t.first; r0 < rows; r0 += kUnroll * kPer) {
    uint4 x[kUnroll];
    float f[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kPer + sub, h = r < p.hkv ? r : r - p.hkv;
      const int64_t at = t.base + ((int64_t)h << p.page_shift);
      const uint8_t* pool = r < p.hkv ? p.k : p.v;
      x[u] = make_uint4(0, 0, 0, 0);
      f[u] = 0.f;
      if (r < rows && !t.tail) {
        if constexpr (E4M3) {
          const uint2 c = *reinterpret_cast<const uint2*>(pool + at * D + seg * 8);
          x[u].x = c.x;
          x[u].y = c.y;
          f[u] = cache_scale((r < p.hkv ? p.k_scales : p.v_scales)[at]);
        } else {
          x[u] = *reinterpret_cast<const uint4*>(pool + (at * D + seg * 8) * 2);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kPer + sub, h = r < p.hkv ? r : r - p.hkv;
      if constexpr (E4M3) {
        uint32_t y[4];
        const uint32_t w[2] = {x[u].x, x[u].y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
          const float2 ab = __half22float2(__half2(hr));
          y[i] = bf16x2_bits(ab.x * f[u], ab.y * f[u]);
        }
        x[u] = make_uint4(y[0], y[1], y[2], y[3]);
      }
      if (r < rows) (r < p.hkv ? k : v)[((int64_t)t.token * p.hkv + h) * kLanes + seg] = x[u];
    }
  }
}

inline int64_t token_blocks(const CacheParams& p) {
  const int64_t parts = (2 * p.hkv + kRowsPerWarp - 1) / kRowsPerWarp;
  return ((int64_t)p.T * parts + kWarps - 1) / kWarps;
}

}  // namespace

cudaError_t launch_cache_plan(const int32_t* cu, const int32_t* kv, int N, int T, int hq, int hkv, int max_chunk,
                              int64_t max_kv, int left, void* plan, cudaStream_t s) {
  cache_plan_kernel<<<1, kPlanThreads, 0, s>>>(cu, kv, N, T, hq, hkv, max_chunk, max_kv, left, plan);
  return cudaGetLastError();
}

cudaError_t launch_cache_write(int D, bool e4m3, const CacheParams& p, const void* k, const void* v, cudaStream_t s) {
  const int64_t blocks = token_blocks(p);
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const auto f = D == 128 ? (e4m3 ? cache_write_kernel<128, true> : cache_write_kernel<128, false>)
                          : (e4m3 ? cache_write_kernel<64, true> : cache_write_kernel<64, false>);
  f<<<(unsigned)blocks, kWarps * 32, 0, s>>>(p, static_cast<const uint4*>(k), static_cast<const uint4*>(v));
  return cudaGetLastError();
}

cudaError_t launch_cache_read(int D, bool e4m3, const CacheParams& p, void* k, void* v, cudaStream_t s) {
  const int64_t blocks = token_blocks(p);
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const auto f = D == 128 ? (e4m3 ? cache_read_kernel<128, true> : cache_read_kernel<128, false>)
                          : (e4m3 ? cache_read_kernel<64, true> : cache_read_kernel<64, false>);
  f<<<(unsigned)blocks, kWarps * 32, 0, s>>>(p, static_cast<uint4*>(k), static_cast<uint4*>(v));
  return cudaGetLastError();
}

}  // namespace flamia
