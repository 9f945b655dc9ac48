// Paged key/value cache: what its kernels and the ABI share (the plan's layout, page look-up,
// the attention's parameters and workspace).
#pragma once
#include "common.cuh"
#include "scored.cuh"

namespace flamia {

// Rows of a kv head in a sequence: its new tokens times the query heads that share the head, token by token.
constexpr int kStepRows = 16;      // rows of a step's unit, past which its keys are streamed
constexpr int kStepTiles = 2;      // row tiles that a step has at most
constexpr int kChunkRows = 2 * kTile;   // rows of a unit otherwise
constexpr int kStepTile = 64;      // keys a tile of a step
// Rows up to which a call's sequences are steps, each row tile a stream of its own.  Steps against chunks, us: 16 sequences
// of 32 rows over some 3200 keys 40 / 43 (E4M3), 42 / 43 (bf16), d 64 31 / 40, one over 30000 35 / 57; with 48 rows 53 / 44.
// In a call that has chunks too, 8 where a token's rows fit in: its steps then cost half of what 16 rows do, and the
// few sequences between the two go with the chunks.
__host__ __device__ inline int step_rows(int group, int64_t max_chunk) {
  return max_chunk * group > kStepTiles * kStepRows && group <= 8 ? 8 : kStepTiles * kStepRows;
}
// What a unit costs besides its key tiles, in key tiles, when the work is dealt out: its queries, its start, its end.
constexpr int kStepExtra = 3, kChunkExtra = 3;
// What it costs to join pieces, in key tiles (chunks gained up to 9; steps of 5 sequences of 100 to 900 keys took 14.8
// instead of 12.6 us whole, with 12).
constexpr int kStepJoin = 9, kChunkJoin = 9;

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
  kCpStepPlaces = 8,   // two words each, as the next: places of all steps, of all chunk units
  kCpChunkPlaces = 10,
  kCpStepCtas = 12,    // CTAs that they are dealt out to
  kCpChunkCtas = 13,
  kCpHeaderWords = 16,
};
// An item: the units of a row tile, the same for every kv head.
struct alignas(16) CacheItem {
  int seq, row, tile, tiles;     // first row; first key tile and their number
};
// A unit is an item for a kv head: a tile of a sequence's rows over the key tiles that they see.  The places of all
// units, unit after unit, are dealt out to the CTAs in equal shares, so that every CTA has the same to do whatever
// the sequences' lengths are (in whole units where that takes little longer): a unit has some places for what it costs
// besides (kStepExtra, kChunkExtra), then one for each key tile.  A unit whose key tiles lie in several shares is joined
// after.
struct CachedUnit {
  int seq, h, row, rows, tile, tiles;     // first row, rows, first key tile, key tiles
  int start, count, keys, lo;             // of the sequence (CachePlanView::seq)
  int item, pad;
  int64_t begin;                          // its first place
};
struct ShareStart {
  CachedUnit u;                           // the unit that the share begins in
  int64_t from, to;                       // its places
};
static_assert(sizeof(ShareStart) == 72, "");
constexpr int kStepCtas = 304, kChunkCtas = 152, kDone = kStepCtas + 8 * kChunkCtas;
// Words before the rows' places, the same in every plan: so a kernel may read its share before it knows whose plan it has.
constexpr int kCpRowWords = kCpHeaderWords + (kChunkCtas + kStepCtas) * (int)(sizeof(ShareStart) / 4);
static_assert(kCpRowWords % 4 == 0, "");
struct CachePlanView {
  int* hdr;
  int2* row;                  // [T] {sequence, position} of the sequences' rows
  int4* seq;                  // [N] {first token, new tokens, keys with them, first key that the first new one sees}
  CacheItem* items[2];        // [cap] chunk items, [kStepTiles N] steps
  int64_t* prefix[2];         // [items + 1] places of the items before, for one kv head
  int64_t* base;              // [N + 1] chunk items before
  ShareStart* first[2];       // [CTAs] where a CTA's share begins and ends
  int* done;                  // [kStepCtas + 8 kChunkCtas] finished pieces of a split unit (of a chunk's 32 rows each), by
                              // the CTA that has its beginning; 0 between calls
};
__host__ __device__ inline int64_t cache_item_capacity(int64_t T, int N, int hq, int hkv) {
  return T * (hq / hkv) / kChunkRows + N;
}
// The shares and the rows come first: writing and reading the cache need no more of the layout.
__host__ __device__ inline CachePlanView cache_plan_view(const void* plan, int64_t T, int N, int hq, int hkv, size_t* bytes = nullptr) {
  const int64_t cap = cache_item_capacity(T, N, hq, hkv);
  CachePlanView v;
  v.hdr = (int*)plan;
  v.first[0] = (ShareStart*)(v.hdr + kCpHeaderWords);
  v.first[1] = v.first[0] + kChunkCtas;
  v.row = (int2*)(v.hdr + kCpRowWords);
  v.seq = (int4*)(v.row + ((T + 1) & ~(int64_t)1));
  v.items[0] = (CacheItem*)(v.seq + N);
  v.items[1] = v.items[0] + cap;
  v.prefix[0] = (int64_t*)(v.items[1] + (int64_t)kStepTiles * N);
  v.prefix[1] = v.prefix[0] + (cap + 1);
  v.base = v.prefix[1] + ((int64_t)kStepTiles * N + 1);
  v.done = (int*)(v.base + (N + 1));
  if (bytes) *bytes = (size_t)((const uint8_t*)(v.done + kDone) - (const uint8_t*)plan);
  return v;
}
inline size_t cache_plan_bytes(int64_t T, int N, int hq, int hkv) {
  size_t n;
  cache_plan_view(nullptr, T, N, hq, hkv, &n);
  return n;
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
  uint32_t inv_group;        // 2^16 / (hq / hkv) and a bit more: a division of a step's rows
  float* part;               // workspace
};
// A CTA leaves at most two unfinished pieces of units behind (the unit that its first key tile lies inside of, and the
// one that its last lies inside of): a row's weighted values, its sum and its reference each.
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
// O = 0, LSE = +inf behind the last sequence.
template <int D>
__device__ __forceinline__ void clear_rows(const CachedParams& p, int valid, int threads) {
  for (int row = valid + blockIdx.x; row < p.c.T; row += gridDim.x) {
    uint4* dst = reinterpret_cast<uint4*>(p.out + (int64_t)row * p.hq * D);
#pragma unroll 1
    for (int i = threadIdx.x; i < p.hq * (D / 8); i += threads) dst[i] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (int h = threadIdx.x; h < p.hq; h += threads) p.lse[(int64_t)h * p.c.T + row] = INFINITY;
  }
}

// ---------------------------------------------------------------- units and shares
struct Shares {
  int64_t total;      // places
  int n;              // CTAs with a share
  __device__ __forceinline__ int64_t begin(int c) const { return total * c / n; }
  __device__ __forceinline__ int of(int64_t f) const { return (int)(((f + 1) * n - 1) / total); }   // the last c with begin(c) <= f
};
template <bool STEP>
__device__ __forceinline__ Shares cached_shares(const int* hdr) {
  Shares s;
  s.total = *reinterpret_cast<const int64_t*>(hdr + (STEP ? kCpStepPlaces : kCpChunkPlaces));
  s.n = hdr[STEP ? kCpStepCtas : kCpChunkCtas];
  return s;
}
// The first unit of item i.
template <bool STEP>
__device__ __forceinline__ CachedUnit cached_item(const CachePlanView& pv, int i, int hq, int hkv) {
  const CacheItem x = pv.items[STEP][i];
  const int4 r = pv.seq[x.seq];
  CachedUnit u;
  u.seq = x.seq;
  u.h = 0;
  u.row = x.row;
  u.rows = min(r.y * (hq / hkv) - x.row, STEP ? kStepRows : kChunkRows);
  u.tile = x.tile;
  u.tiles = x.tiles;
  u.start = r.x;
  u.count = r.y;
  u.keys = r.z;
  u.lo = r.w;
  u.item = i;
  u.pad = 0;
  u.begin = pv.prefix[STEP][i] * hkv;
  return u;
}
// The unit after u.
template <bool STEP>
__device__ __forceinline__ void cached_next(const CachePlanView& pv, CachedUnit& u, int hq, int hkv) {
  if (u.h + 1 < hkv) {
    ++u.h;
    u.begin += u.tiles + (STEP ? kStepExtra : kChunkExtra);
  } else {
    u = cached_item<STEP>(pv, u.item + 1, hq, hkv);
  }
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
// The CTAs whose pieces of u are to be joined, of which the caller has key tiles [t0, t1): the first one, and their number.
template <bool STEP>
__device__ __forceinline__ int2 cached_owners(const CachedUnit& u, const Shares& sh, int t0, int t1) {
  const int64_t first = u.begin + (STEP ? kStepExtra : kChunkExtra);
  int2 c = make_int2(blockIdx.x, blockIdx.x);
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {        // (mostly one division, of 64 bits)
    if (i ? t1 == u.tiles : t0 == 0) continue;
    const int y = sh.of(i ? first + u.tiles - 1 : first);
    if (i) c.y = y;
    else c.x = y;
  }
  return make_int2(c.x, c.y - c.x + 1);
}
// Unfinished pieces: the one that a CTA's share begins in the middle of (0), and the one that it ends in the middle of and
// has the beginning of (1).  [rows][D] weighted values, [rows] references (base 2), [rows] sums.
template <bool STEP, int D>
__device__ __forceinline__ float* cached_part(const CachedParams& p, int cta, int slot) {
  constexpr int kRows = STEP ? kStepRows : kChunkRows;
  float* base = p.part + (STEP ? 0 : (size_t)2 * kStepCtas * kStepRows * (D + 2));
  return base + (size_t)(2 * cta + slot) * kRows * (D + 2);
}
// One more piece of a split unit is finished (the caller's writes and those of the threads it has met since are
// visible to whoever sees the count): true for the last of n, who joins them, in the order of the keys whoever it is.
__device__ __forceinline__ bool cached_last(int* done, int n) {
  __threadfence();
  const bool last = atomicAdd(done, 1) == n - 1;
  if (last) *done = 0;
  __threadfence();
  return last;
}

}  // namespace flamia
