// Paged key/value cache: its plan, writing it and reading it back.
//
// The plan (one CTA, no host synchronisation) checks a call's sequences and lists the attention's
// work: the steps' key tiles and the chunk items, each with the running sum of its key tiles, so
// that a kernel can deal the key tiles out evenly whatever the sequences are.
//
// Writing quantizes each (token, head) row by itself, the per-token form of the operand quantizer: a later token changes
// no earlier one's code.  Both directions move every byte once.
#include <algorithm>
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
  __shared__ int s_bad, s_largest[2];      // places of the largest unit
  const CachePlanView pv = cache_plan_view(plan, T, N, hq, hkv);
  const int group = hq / hkv, limit = step_rows(group, max_chunk);
  if (threadIdx.x == 0) s_bad = s_largest[0] = s_largest[1] = 0;
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
          atomicMax(&s_largest[1], (int)st);
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
      atomicMax(&s_largest[0], cost);
      pv.items[0][i] = x;
    }
    int64_t tot;
    const int64_t a = block_scan(cost, warp_sums, &tot);
    if (i < items) pv.prefix[0][i] = chunk_places + a;
    chunk_places += tot;
  }
  if (threadIdx.x == 0) pv.prefix[0][items] = chunk_places;
  __syncthreads();
  // shares: the CTAs that get one, and where each begins and ends.  whole: that many whole units a CTA; 0: equal shares
  auto shares = [&](auto STEP, int64_t total, int64_t n_items, int n, int whole, int c) {
    constexpr int kStep = decltype(STEP)::value;
    Shares sh;
    sh.total = total;
    sh.n = n;
    if (c == 0) {
      *reinterpret_cast<int64_t*>(pv.hdr + (kStep ? kCpStepPlaces : kCpChunkPlaces)) = total;
      pv.hdr[kStep ? kCpStepCtas : kCpChunkCtas] = sh.n;
    }
    if (c >= sh.n) return;
    const int64_t* prefix = pv.prefix[kStep];
    auto unit_begin = [&](int64_t unit) {
      const int64_t i = unit / hkv;
      return i < n_items ? prefix[i] * hkv + unit % hkv * (prefix[i + 1] - prefix[i]) : total;
    };
    ShareStart x;
    x.from = whole ? unit_begin((int64_t)c * whole) : sh.begin(c);
    x.to = whole ? unit_begin((int64_t)(c + 1) * whole) : sh.begin(c + 1);
    int64_t lo = 0, hi = n_items;          // prefix[lo] hkv <= from < prefix[hi] hkv
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (prefix[mid] * hkv <= x.from) lo = mid; else hi = mid;
    }
    x.u = cached_item<kStep != 0>(pv, (int)lo, hq, hkv);
    const int len = x.u.tiles + (kStep ? kStepExtra : kChunkExtra);
    x.u.h = (int)((x.from - x.u.begin) / len);
    x.u.begin += (int64_t)x.u.h * len;
    pv.first[kStep][c] = x;
  };
  // A CTA takes some places at least: fewer would cost more in joining than they save.  Where steps are the lesser part
  // beside chunks they get a CTA a SM on as many SMs as their part is (a place of theirs takes about a third of a
  // chunk's), and the chunks the others: a chunk's CTA does not fit beside a step's, and the ones that had to wait
  // came last (ragged chunks and two steps: 62 instead of 54 us).
  const int64_t steps_all = step_places * hkv, chunks_all = chunk_places * hkv;
  int64_t step_most = kStepCtas, chunk_most = kChunkCtas;
  if (steps_all > 0 && chunks_all > 0 && steps_all < 3 * chunks_all) {
    step_most = kChunkCtas * steps_all / (steps_all + 3 * chunks_all) + 1;
    chunk_most = kChunkCtas - min(step_most, (steps_all + 3 + kStepExtra) / (4 + kStepExtra));
  }
  // Whole units, as many a CTA, where that takes little longer than equal shares, whose ends have to be joined: 16 sequences
  // of 26 rows of 4 heads over some 300 keys 17 instead of 30 us, steps of 4 of some 100 keys 7.4 instead of 11.5.
  auto deal = [&](int64_t all, int64_t units, int64_t largest, int64_t most, int least, int join, int& n) {
    n = (int)min(most, (all + least - 1) / least);
    if (n == 0) return 0;
    const int64_t whole = (units + most - 1) / most;
    if (whole * largest > all / n + join) return 0;
    n = (int)((units + whole - 1) / whole);
    return (int)whole;
  };
  const bool step = threadIdx.x < kStepCtas;
  int n;
  const int whole = step ? deal(steps_all, steps * hkv, s_largest[1], step_most, 4 + kStepExtra, kStepJoin, n)
                         : deal(chunks_all, items * hkv, s_largest[0], chunk_most, 2 + kChunkExtra, kChunkJoin, n);
  if (step) shares(std::integral_constant<int, 1>{}, steps_all, steps, n, whole, threadIdx.x);
  else if (threadIdx.x < kStepCtas + kChunkCtas)
    shares(std::integral_constant<int, 0>{}, chunks_all, items, n, whole, threadIdx.x - kStepCtas);
}

// The sequence and the position of each row.
__global__ void __launch_bounds__(256) cache_rows_kernel(int N, int T, int hq, int hkv, void* plan) {
  const CachePlanView pv = cache_plan_view(plan, T, N, hq, hkv);
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= pv.hdr[kCpValid]) return;
  int lo = 0, hi = N;          // the last sequence that begins at t or before
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pv.seq[mid].x <= t) lo = mid; else hi = mid;
  }
  const int4 r = pv.seq[lo];
  pv.row[t] = make_int2(lo, r.z - r.y + t - r.x);
}

// ---------------------------------------------------------------- write, read
// A warp takes the rows (of all heads) of some tokens, of K or of V: a stream on the packed side.  16 elements a lane, so that
// what a row needs once (its largest value, its scale, its place) is shared by few lanes: with 8 the
// instructions bound it (write of 16384 tokens, 16 heads, d 128: 48 instead of 38 us, 70% of the issue slots).
// 32 rows a warp: 34.3 us, 5.9 TB/s (87% of a copy's rate), and 37 for the read of 4 x 8192 of 8 heads; with 64 or 128 rows
// 38 and 36, 38 and 44.  With loads that are marked as streaming the write takes 36.8 in a row of calls.
// Where the tokens live it looks up once, a lane a token.
constexpr int kWarps = 8;
constexpr int kRowsPerWarp = 32;

struct TokenGroup {
  int token, n;      // first token, tokens
  bool v;            // V's rows, not K's
};
__device__ __forceinline__ TokenGroup token_group(const CacheParams& p, int per) {
  const int64_t job = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), at = (job >> 1) * per;
  TokenGroup g;
  g.v = job & 1;
  g.token = (int)min(at, (int64_t)p.T);
  g.n = min(per, p.T - g.token);
  return g;
}
// The lane's token's place (row of kv head 0 in the pools), -1 where it has none: behind the last sequence, or no page.
__device__ __forceinline__ int64_t token_place(const CacheParams& p, const TokenGroup& g, int lane, int valid) {
  if (lane >= g.n || g.token + lane >= valid) return -1;
  const int2 r = reinterpret_cast<const int2*>(p.plan + kCpRowWords)[g.token + lane];
  const int page = cache_page(p, r.x, r.y >> p.page_shift);
  return page < 0 ? -1 : ((int64_t)page * p.hkv << p.page_shift) + (r.y & ((1 << p.page_shift) - 1));
}
// A row's lanes: 16-byte words seg and seg + kLanes of it; kPer rows a load.
template <int D>
struct RowLanes {
  static constexpr int kLanes = D / 16, kPer = 32 / kLanes, kUnroll = 2;
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) cache_write_kernel(const CacheParams p, const uint4* __restrict__ k,
                                                                  const uint4* __restrict__ v, const int per,
                                                                  const uint32_t inv_hkv) {
  using R = RowLanes<D>;
  const TokenGroup g = token_group(p, per);
  if (g.n <= 0) return;
  const int lane = threadIdx.x & 31, sub = lane / R::kLanes, seg = lane % R::kLanes, rows = g.n * p.hkv;
  const uint4* src = (g.v ? v : k) + (int64_t)g.token * p.hkv * (D / 8) + seg;
  uint8_t* pool = g.v ? p.v : p.k;
  uint8_t* scales = g.v ? p.v_scales : p.k_scales;
  int64_t places = -2;
  for (int r0 = 0; r0 < rows; r0 += R::kUnroll * R::kPer) {
    uint4 x[R::kUnroll][2];
#pragma unroll
    for (int u = 0; u < R::kUnroll; ++u)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = r0 + u * R::kPer + sub;
        x[u][j] = r < rows ? src[r * (D / 8) + j * R::kLanes] : make_uint4(0, 0, 0, 0);
      }
    if (places == -2) places = token_place(p, g, lane, cache_valid_rows(p));     // (while the first loads fly)
#pragma unroll
    for (int u = 0; u < R::kUnroll; ++u) {
      const int r = r0 + u * R::kPer + sub, i = p.hkv == 1 ? r : (int)__umulhi((uint32_t)r, inv_hkv);     // token r / hkv
      const int64_t base = __shfl_sync(0xffffffffu, places, i & 31);
      const int64_t at = base + ((int64_t)(r - i * p.hkv) << p.page_shift);
      const bool use = r < rows && base >= 0;
      if constexpr (E4M3) {
        // the largest magnitude by its bits (a NaN's are above infinity's): e = least integer with amax <= 448 2^e is
        // the exponent less 8, and one more above 1.75; byte e + 127
        const uint32_t m7 = 0x7fff7fffu;
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[u][j].x & m7, x[u][j].y & m7), __vmaxu2(x[u][j].z & m7, x[u][j].w & m7)));
#pragma unroll
        for (int o = R::kLanes / 2; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = max(m & 0xffffu, m >> 16);
        const bool nan = m > 0x7f80u;
        const uint32_t byte = nan ? 255u : m == 0 ? 127u : max((m + 31) >> 7, 8u) - 8;
        const float f = nan ? 0.f : __uint_as_float((254 - byte) << 23);      // 2^-e
        const float2 f2 = make_float2(f, f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t c[4];
          const uint32_t w[4] = {x[u][j].x, x[u][j].y, x[u][j].z, x[u][j].w};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const float2 y = fmul2(make_float2(__uint_as_float(w[t] << 16), __uint_as_float(w[t] & 0xffff0000u)), f2);
            c[t] = e4m3x2(y.x, y.y);
          }
          if (use)
            *reinterpret_cast<uint2*>(pool + at * D + (j * R::kLanes + seg) * 8) =
                nan ? make_uint2(0, 0) : make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
        }
        if (use && seg == 0) scales[at] = (uint8_t)byte;
      } else if (use) {
#pragma unroll
        for (int j = 0; j < 2; ++j) *reinterpret_cast<uint4*>(pool + (at * D + (j * R::kLanes + seg) * 8) * 2) = x[u][j];
      }
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2_bits(float2 a) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a.x, a.y);
  return *reinterpret_cast<const uint32_t*>(&x);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) cache_read_kernel(const CacheParams p, uint4* __restrict__ k,
                                                                 uint4* __restrict__ v, const int per,
                                                                 const uint32_t inv_hkv) {
  using R = RowLanes<D>;
  const TokenGroup g = token_group(p, per);
  if (g.n <= 0) return;
  const int lane = threadIdx.x & 31, sub = lane / R::kLanes, seg = lane % R::kLanes, rows = g.n * p.hkv;
  uint4* dst = (g.v ? v : k) + (int64_t)g.token * p.hkv * (D / 8) + seg;
  const uint8_t* pool = g.v ? p.v : p.k;
  const uint8_t* scales = g.v ? p.v_scales : p.k_scales;
  const int64_t places = token_place(p, g, lane, cache_valid_rows(p));
  for (int r0 = 0; r0 < rows; r0 += R::kUnroll * R::kPer) {
    uint4 x[R::kUnroll][2];
    uint32_t b[R::kUnroll];
#pragma unroll
    for (int u = 0; u < R::kUnroll; ++u) {
      const int r = r0 + u * R::kPer + sub, i = p.hkv == 1 ? r : (int)__umulhi((uint32_t)r, inv_hkv);
      const int64_t base = __shfl_sync(0xffffffffu, places, i & 31);
      const int64_t at = base + ((int64_t)(r - i * p.hkv) << p.page_shift);
      const bool use = r < rows && base >= 0;
      b[u] = E4M3 && use ? scales[at] : 127;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x[u][j] = make_uint4(0, 0, 0, 0);
        if constexpr (E4M3) {
          const uint2 c = use ? *reinterpret_cast<const uint2*>(pool + at * D + (j * R::kLanes + seg) * 8) : make_uint2(0, 0);
          x[u][j].x = c.x;
          x[u][j].y = c.y;
        } else if (use) {
          x[u][j] = *reinterpret_cast<const uint4*>(pool + (at * D + (j * R::kLanes + seg) * 8) * 2);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < R::kUnroll; ++u) {
      const int r = r0 + u * R::kPer + sub;
      const float f = cache_scale(b[u]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (E4M3) {
          uint32_t y[4];
          const uint32_t w[2] = {x[u][j].x, x[u][j].y};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[t / 2] >> (16 * (t & 1))), __NV_E4M3);
            y[t] = bf16x2_bits(fmul2(__half22float2(__half2(hr)), make_float2(f, f)));
          }
          x[u][j] = make_uint4(y[0], y[1], y[2], y[3]);
        }
        if (r < rows) dst[r * (D / 8) + j * R::kLanes] = x[u][j];
      }
    }
  }
}

// Tokens a warp: kRowsPerWarp rows where that leaves the GPU's warps busy.
struct TokenGrid {
  int per;
  int64_t blocks;
  uint32_t inv_hkv;      // ceil(2^32 / hkv): r / hkv by a multiplication, exact for r below 2^32 / hkv
};
inline TokenGrid token_grid(const CacheParams& p) {
  TokenGrid g;
  const int64_t most = std::min<int64_t>(32, (kRowsPerWarp + p.hkv - 1) / p.hkv);
  g.per = (int)std::min<int64_t>(std::max<int64_t>((int64_t)p.T * 2 / (152 * 32), 1), most);
  g.blocks = (((int64_t)p.T + g.per - 1) / g.per * 2 + kWarps - 1) / kWarps;
  g.inv_hkv = (uint32_t)((((uint64_t)1 << 32) + p.hkv - 1) / p.hkv);
  return g;
}

}  // namespace

cudaError_t launch_cache_plan(const int32_t* cu, const int32_t* kv, int N, int T, int hq, int hkv, int max_chunk,
                              int64_t max_kv, int left, void* plan, cudaStream_t s) {
  cache_plan_kernel<<<1, kPlanThreads, 0, s>>>(cu, kv, N, T, hq, hkv, max_chunk, max_kv, left, plan);
  if (T > 0) cache_rows_kernel<<<(T + 255) / 256, 256, 0, s>>>(N, T, hq, hkv, plan);
  return cudaGetLastError();
}

cudaError_t launch_cache_write(int D, bool e4m3, const CacheParams& p, const void* k, const void* v, cudaStream_t s) {
  const TokenGrid g = token_grid(p);
  if (g.blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const auto f = D == 128 ? (e4m3 ? cache_write_kernel<128, true> : cache_write_kernel<128, false>)
                          : (e4m3 ? cache_write_kernel<64, true> : cache_write_kernel<64, false>);
  f<<<(unsigned)g.blocks, kWarps * 32, 0, s>>>(p, static_cast<const uint4*>(k), static_cast<const uint4*>(v), g.per, g.inv_hkv);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(int D, bool e4m3, const CacheParams& p, void* k, void* v, cudaStream_t s) {
  const TokenGrid g = token_grid(p);
  if (g.blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const auto f = D == 128 ? (e4m3 ? cache_read_kernel<128, true> : cache_read_kernel<128, false>)
                          : (e4m3 ? cache_read_kernel<64, true> : cache_read_kernel<64, false>);
  f<<<(unsigned)g.blocks, kWarps * 32, 0, s>>>(p, static_cast<uint4*>(k), static_cast<uint4*>(v), g.per, g.inv_hkv);
  return cudaGetLastError();
}

}  // namespace flamia
