// Paged key/value cache: what its kernels and the ABI share (the plan's layout, page look-up,
// the attention's parameters and workspace).
#pragma once
#include "common.cuh"
#include "scored.cuh"

namespace flamia {

// Rows of a kv head in a sequence: its new tokens times the query heads that share the head, token by token.
constexpr int kStepRows = 16;      // up to so many a sequence may be a step: one tile of rows, keys streamed past it
constexpr int kChunkRows = 2 * kTile;   // rows of a unit otherwise
constexpr int kStepTile = 64;      // keys a tile of a step
// Rows up to which a call's sequences are steps.  In a call that has chunks too, 8 where a token's rows fit in: its steps
// then cost half of what 16 rows do, and the few sequences between the two go with the chunks.
__host__ __device__ inline int step_rows(int group, int64_t max_chunk) {
  return max_chunk * group > kStepRows && group <= 8 ? 8 : kStepRows;
}
// What a unit costs besides its key tiles, in key tiles, when the work is dealt out: its queries, its end.
constexpr int kStepExtra = 3, kChunkExtra = 1;

// ---------------------------------------------------------------- plan
enum CachePlanWord : int {
  kCpStatus = 0,
  kCpNumSeqs = 1,
  kCpTotal = 2,
  kCpHkv = 3,
  kCpHq = 4,
  kCpMaxChunk = 5,
  kCpLeft = 6,
  kCpValid = 7,        // rows of the sequences (0: the plan is bad)
  kCpItems = 8,        // chunk items
  kCpHeaderWords = 16,
};
// A chunk item: up to kChunkRows rows of a sequence, the same for every kv head.
struct CacheItem {
  int seq, row, tile, tiles;     // first row; first key tile (kTile keys) and their number
};
struct CachePlanView {
  int* hdr;
  int4* seq;               // [N] {first token, new tokens, keys with them, first key that the first new one sees}
  int64_t* step_prefix;    // [N + 1] key tiles of the steps before, kStepExtra more for each
  int64_t* item_base;      // [N + 1] chunk items before
  CacheItem* items;        // [cap]
  int64_t* item_prefix;    // [cap + 1] key tiles of the items before, kChunkExtra more for each
};
__host__ __device__ inline int64_t cache_item_capacity(int64_t T, int N, int hq, int hkv) {
  return T * (hq / hkv) / kChunkRows + N;
}
__host__ __device__ inline size_t cache_plan_bytes(int64_t T, int N, int hq, int hkv) {
  const int64_t cap = cache_item_capacity(T, N, hq, hkv);
  return (size_t)kCpHeaderWords * 4 + (size_t)N * 16 + (size_t)(N + 1) * 16 + (size_t)cap * 24 + 16;
}
// The sequences come first: writing and reading the cache need no more of the layout.
__host__ __device__ inline CachePlanView cache_plan_view(const void* plan, int64_t T, int N, int hq, int hkv) {
  CachePlanView v;
  v.hdr = (int*)plan;
  v.seq = (int4*)(v.hdr + kCpHeaderWords);
  v.items = (CacheItem*)(v.seq + N);
  v.step_prefix = (int64_t*)(v.items + cache_item_capacity(T, N, hq, hkv));
  v.item_base = v.step_prefix + (N + 1);
  v.item_prefix = v.item_base + (N + 1);
  return v;
}

struct CacheParams {
  uint8_t *k, *v;                  // [pages][hkv][P][d] E4M3 or bf16
  uint8_t *k_scales, *v_scales;    // [pages][hkv][P] UE8M0 (E4M3)
  const int32_t* table;            // [N][max_pages]
  int num_pages, max_pages, page_shift, hkv;
  int* plan;
  int N, T;
};
// Rows that the plan says lie in sequences; 0 where it was built for another call.
__device__ __forceinline__ int cache_valid_rows(const CacheParams& p) {
  const int* h = p.plan;
  if (h[kCpNumSeqs] == p.N && h[kCpTotal] == p.T && h[kCpHkv] == p.hkv) return h[kCpValid];
  atomicOr(p.plan + kCpStatus, FLAMIA_DEV_PLAN_MISMATCH);
  return 0;
}
// Page of index i of sequence n, or -1 (and the status bit) where the table has none.
__device__ __forceinline__ int cache_page(const CacheParams& p, int n, int i) {
  const int page = i < p.max_pages ? p.table[(int64_t)n * p.max_pages + i] : -1;
  if ((unsigned)page < (unsigned)p.num_pages) return page;
  atomicOr(p.plan + kCpStatus, FLAMIA_DEV_BAD_PAGE);
  return -1;
}
// Largest n in [0, N) with at(n) <= x, at non-decreasing and at(0) <= x: 32 probes a round by a whole warp.
template <class At, class X>
__device__ __forceinline__ int warp_upper(int N, X x, At at) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = N;
  while (n > 1) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const int below = __popc(__ballot_sync(0xffffffffu, lane * step < n && at(i) <= x)) - 1;
    lo += below * step;
    n = min(step, n - below * step);
  }
  return lo;
}
// 2^(b - 127), NaN for 255.
__device__ __forceinline__ float cache_scale(uint32_t b) { return b == 255 ? __uint_as_float(0x7fc00000u) : ue8m0_to_f32(b); }

// ---------------------------------------------------------------- attention
struct CachedParams {
  CacheParams c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  int hq, left, max_chunk;
  double scale;              // softmax scale
  float scale2;              // softmax scale log2 e
  float cap;                 // 0: none
  CapForm capf;
  float* part;               // workspace
};
// A CTA leaves at most two unfinished pieces of units behind (the unit that its first key tile lies inside of, and the
// one that its last lies inside of): a row's weighted values, its sum and its reference each.
constexpr int kStepCtas = 304, kChunkCtas = 152;
inline size_t cached_workspace_bytes(int hq, int hkv, int d, int max_chunk) {
  const size_t row = (size_t)(d + 2) * 4;
  return 2 * row * ((size_t)kStepCtas * kStepRows + ((int64_t)max_chunk * (hq / hkv) > step_rows(hq / hkv, max_chunk) ? (size_t)kChunkCtas * kChunkRows : 0));
}
__device__ __forceinline__ int cached_valid_rows(const CachedParams& p) {
  const int* h = p.c.plan;
  if (h[kCpHq] == p.hq && h[kCpLeft] == p.left && h[kCpMaxChunk] == p.max_chunk) return cache_valid_rows(p.c);
  atomicOr(p.c.plan + kCpStatus, FLAMIA_DEV_PLAN_MISMATCH);
  return 0;
}


// ---------------------------------------------------------------- units and shares
// A unit is a tile of a sequence's rows (a step: all of them) and a kv head, over the key tiles that its rows see.
// The places of all units, unit after unit, are dealt out to the CTAs in equal shares, so that every CTA has the same
// to do whatever the sequences' lengths are: a unit has kExtra places, then one for each key tile.  A unit whose key
// tiles lie in several shares is joined after.
struct CachedUnit {
  int seq, h, row, rows, tile, tiles;     // first row, rows, first key tile, key tiles
  int start, count, keys, lo;             // of the sequence (CachePlanView::seq)
  int64_t begin;                          // its first place
};
template <bool STEP>
__device__ __forceinline__ int64_t cached_places(const CachedParams& p, const CachePlanView& pv) {
  return (STEP ? pv.step_prefix[p.c.N] : pv.item_prefix[pv.hdr[kCpItems]]) * p.c.hkv;
}
// The unit of place f (found by a whole warp).
template <bool STEP>
__device__ __forceinline__ CachedUnit cached_unit(const CachedParams& p, const CachePlanView& pv, int64_t f) {
  constexpr int kExtra = STEP ? kStepExtra : kChunkExtra;
  CachedUnit u;
  const int64_t* prefix = STEP ? pv.step_prefix : pv.item_prefix;
  const int hkv = p.c.hkv;
  const int i = warp_upper(STEP ? p.c.N : pv.hdr[kCpItems], f, [&](int x) { return prefix[x] * hkv; });
  const int64_t first = prefix[i] * hkv;
  CacheItem item{i, 0, 0, 0};
  if (!STEP) item = pv.items[i];
  const int4 r = pv.seq[item.seq];
  u.seq = item.seq;
  u.start = r.x;
  u.count = r.y;
  u.keys = r.z;
  u.lo = r.w;
  const int rows = r.y * (p.hq / hkv);
  u.row = item.row;
  u.rows = STEP ? rows : min(rows - u.row, kChunkRows);
  u.tile = STEP ? r.w / kStepTile : item.tile;
  u.tiles = STEP ? (int)(prefix[i + 1] - prefix[i]) - kExtra : item.tiles;
  u.h = (int)((f - first) / (u.tiles + kExtra));
  u.begin = first + (int64_t)u.h * (u.tiles + kExtra);
  return u;
}
// A share's part of a unit: key tiles [t0, t1), none where the share ends before the first; f moves behind it.
template <bool STEP>
__device__ __forceinline__ int2 cached_piece(const CachedUnit& u, int64_t& f, int64_t end) {
  constexpr int kExtra = STEP ? kStepExtra : kChunkExtra;
  const int64_t to = min(u.begin + kExtra + u.tiles, end);
  const int2 t = make_int2(max((int)(f - u.begin) - kExtra, 0), max((int)(to - u.begin) - kExtra, 0));
  f = to;
  return t;
}
struct Shares {
  int64_t total;
  int n;              // CTAs with a share
  __device__ __forceinline__ int64_t begin(int c) const { return total * c / n; }
  __device__ __forceinline__ int of(int64_t f) const { return (int)(((f + 1) * n - 1) / total); }   // the last c with begin(c) <= f
};
// A CTA takes kLeast places at least: fewer would cost more in joining than they save.
template <bool STEP>
__device__ __forceinline__ Shares cached_shares(const CachedParams& p, const CachePlanView& pv) {
  constexpr int kCtas = STEP ? kStepCtas : kChunkCtas, kLeast = STEP ? 4 + kStepExtra : 2 + kChunkExtra;
  Shares s;
  s.total = cached_places<STEP>(p, pv);
  s.n = (int)min((int64_t)kCtas, (s.total + kLeast - 1) / kLeast);
  return s;
}
// The unit that begins in CTA c's share and ends behind it, whose pieces in c .. c + n - 1 are to be joined; n = 0: none.
template <bool STEP>
__device__ __forceinline__ int cached_split(const CachedParams& p, const CachePlanView& pv, const Shares& sh, int c,
                                            CachedUnit& u) {
  if (c + 1 >= sh.n) return 0;
  u = cached_unit<STEP>(p, pv, sh.begin(c + 1) - 1);
  const int64_t first = u.begin + (STEP ? kStepExtra : kChunkExtra), last = first + u.tiles - 1;
  if (first < sh.begin(c) || first >= sh.begin(c + 1) || last < sh.begin(c + 1)) return 0;
  return sh.of(last) - c + 1;
}
// Unfinished pieces: the one that a CTA's share begins in the middle of (0), and the one that it ends in the middle of and
// has the beginning of (1).  [rows][D] weighted values, [rows] references (base 2), [rows] sums.
template <bool STEP, int D>
__device__ __forceinline__ float* cached_part(const CachedParams& p, int cta, int slot) {
  constexpr int kRows = STEP ? kStepRows : kChunkRows;
  float* base = p.part + (STEP ? 0 : (size_t)2 * kStepCtas * kStepRows * (D + 2));
  return base + (size_t)(2 * cta + slot) * kRows * (D + 2);
}
// Where row r of a unit is: token and query head.
__device__ __forceinline__ int2 cached_row(const CachedParams& p, const CachedUnit& u, int r) {
  const int group = p.hq / p.c.hkv, x = u.row + r;
  return make_int2(u.start + x / group, u.h * group + x % group);
}

}  // namespace flamia
