// Attention over the paged cache for steps: a sequence's few new tokens, in tiles of up to 16 rows of a kv head.
//
//   x = scale log2 e q.k (capped), m = running maximum, l += 2^(x - m), O += 2^(x - m) v
//
// Bound by memory: every key and value is read once, for 4 d flops a row.  A CTA streams its share of
// the key tiles (64 keys, K and V) through shared memory: one warp issues TMA copies page by page, two compute
// warps take every other tile each, 32 keys a warp with a softmax of its own, and meet only where a unit ends.
// Two CTAs an SM, so that one streams while the other meets, with some 128 KB in flight between them.
// Measured, 32 heads on 8, d 128, E4M3: a token each over 2 x 131972 keys 91 us, 6.0 TB/s (88% of a copy's rate); over 64
// sequences of 251670 keys in pages of 16 99 us (a page is a TMA copy of 2 KB, whose rate bounds it; 91 with pages of 64).
// bf16, 16 heads, a window of 2048 of 32 sequences: 89 us, 5.7 TB/s.  With two row tiles (16 drafts of 4 tokens, 32 heads on 4,
// 52000 keys: 36 us) the products and the softmax bound it, 0.85 us a key tile.
//
// The products run as 16 x 8 x 16 MMAs from registers, keys (then head dimensions) as the 16 and query rows as the 8:
// what is to be fast here is the stream, not the products, and a step's rows rarely fill more (tcgen05 would
// want 64 at least and the codes unpacked into shared memory; rows as the 16 cost twice the softmax and twice
// the accumulators: 98 instead of 91 us on two sequences of 131972).  Which of the head dimensions a lane's operand
// words stand for is free as long as both operands agree, so a lane takes whole 16-byte words of a key's row,
// and for V of one head-dim run in four keys' rows, whose bytes are paired by permutes; with the copies' swizzle
// both are free of bank conflicts.  The weights change from scores' to operands' places by a transpose
// of 8 x 8 within the warp.
//
// E4M3: a code is exact in fp16, two are converted at a time, and the products run in fp16.  Queries are
// scaled by a power of two a row, its largest value to [2^14, 2^15).  The key's scale multiplies the
// score.  The value's scale 2^e enters the weight: w = 2^(x - m + e - M + 13) with a running maximum M of x - m + e
// of its own (against m, so that scores of any size leave the exponents their digits): the largest w is in
// [2^13, 2^15] whatever the scales are, and what falls below fp16's range is 2^-38 of it.  Rounding w
// to fp16 costs 2^-12 of it at most.  An infinity is a code whose scale takes it past fp32's range, which neither product
// sees: tiles with scales that large (some 2^120) add their infinities besides, to the scores and to O.  The others
// pay for that code's registers: 33.4 -> 34.1 us with two row tiles (the drafts below, in a graph), 89.0 -> 89.4 with one.
// bf16: the products run in bf16, and so do the weights (2^-9 at most).
#include <type_traits>

#include "cache.cuh"
#include "ptx.cuh"
#include "tmap.h"

namespace flamia {

cudaError_t launch_cached_chunk(int D, bool e4m3, const CachedParams& p, bool tail, cudaStream_t s);

namespace {

constexpr int kComputeWarps = 4, kThreads = (kComputeWarps + 1) * 32;
constexpr float kBoost = 13.f, kSlack = 2.f;
constexpr int kScaleCopies = 2 * kStepTile / 16;     // of 16 bytes: a TMA copy that small takes as long as a page's
constexpr int kUnits = 2;         // described and their queries fetched ahead

// A unit's piece as the compute warps need it.
struct alignas(16) StepPiece {
  int t0, t1, tiles, tile;        // key tiles [t0, t1) of the unit's; its first tile's number in the sequence.  t1 0: no more
  int h, row, rows, start;        // first row, rows; first token of the sequence
  int pos0, keys, lo;             // its position
  int owner, pieces, last, pad[2];      // of a split unit: the CTA that has its beginning, the CTAs that have pieces
};
static_assert(sizeof(StepPiece) == 64, "");

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two E4M3 codes (the low 16 bits) -> two fp16 values.
__device__ __forceinline__ uint32_t codes_f16(uint32_t c) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t codes_f16_hi(uint32_t c) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(c));
  return r;
}
// A code times its scale 2^(b - 127) is past fp32's (and bf16's) range from 2^(255 - b) on: an infinity, as reading the cache and
// the chunks have it.  The products have the code alone and cannot see that.  The least such code's magnitude; none for
// b < 247 (448 2^119 is finite) and 255 (a NaN's row).
constexpr uint32_t kNoInfinity = 128;
__device__ __forceinline__ uint32_t infinite_from(uint32_t b) { return b < 247 || b == 255 ? kNoInfinity : (262 - b) << 3; }
__device__ __forceinline__ float signed_infinity(uint32_t code) { return __uint_as_float(0x7f800000u | (code & 128) << 24); }
// Products of the infinities of a row of codes with a lane's queries of two row tiles (four of each of D / 16 steps, as they
// are kept in shared memory).  A function that is called: inlined it has the rest spill more (drafts 34.7 instead of 34.1 us).
template <int D>
__device__ __noinline__ float2 infinite_products(const uint8_t* codes, const uint8_t* queries, uint32_t from) {
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int s = 0; s < D / 16; ++s) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(codes) ^ (4 * s & 16)) + (4 * s & 15));
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      const uint32_t c = w >> 8 * j & 255;
      if ((c & 127) < from) continue;
      const __half* y = reinterpret_cast<const __half*>(queries + s * 512) + j;
      sum.x += signed_infinity(c) * __half2float(y[0]);
      sum.y += signed_infinity(c) * __half2float(y[4]);
    }
  }
  return sum;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
__device__ __forceinline__ float cap_one(float x, const CapForm& F) {
  const float z = x * F.zscale, w = z * z;
  float t = fmaf(w, kTanh5e, kTanh5d);
  t = fmaf(w, t, kTanh5c);
  t = fmaf(w, t, kTanh5b);
  t = fmaf(w, t, kTanh5a);
  return fabsf(z) <= kTanh5To ? fmaf(x, w * t, x) : F.inv * tanh_any(z);
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int D, bool E4M3, int NT>
struct StepSmem {
  static constexpr int kRowBytes = E4M3 ? D : 2 * D;
  static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kBoxes = kRowBytes / kBoxBytes;
  static constexpr int kTileBytes = kStepTile * kRowBytes;                    // of K, or of V
  static constexpr int kScales = 2 * kTileBytes;                              // in a stage: K's and V's scale bytes
  static constexpr int kStage = kScales + (E4M3 ? 1024 : 0);           // (stages stay on 1024 bytes)
  // (an even number: a pair of warps takes every other tile, so that a stage is always the same pair's, which sees each
  // phase of its barrier; with an odd number a pair could not tell a phase from the last but one)
  static constexpr int kStages = E4M3 ? (D == 128 ? 4 : 6) : (D == 128 ? 2 : 4);
  static_assert(kStages % 2 == 0, "see above");
  static constexpr int kRows = 8 * NT;
  static constexpr int kRed = kStages * kStage;                               // [4 warps][kRows][D] floats
  static constexpr int kStat = kRed + kComputeWarps * kRows * D * 4;          // [4 warps][m, l][kRows]
  static constexpr int kQ = kStat + kComputeWarps * 2 * kRows * 4;            // [2 units in turn][kRows] queries
  static constexpr int kUnit = kQ + kUnits * kRows * D * 2;
  static constexpr int kSplits = kUnit + kUnits * 64;        // the share's split units, by slot
  static constexpr int kBar = kSplits + 2 * 64;
  static constexpr int kBytes = kBar + (2 * kStages + 2 * kUnits) * 8;
  static constexpr int kAlloc = kBytes + 1024;
};
static_assert(2 * (StepSmem<128, false, 2>::kAlloc + 1024) <= 233472 && 2 * (StepSmem<128, true, 2>::kAlloc + 1024) <= 233472,
              "two CTAs an SM");

// A split unit's rows warp, warp + 4, ... at once (so that their loads fly together); its pieces may be hundreds: a lane a
// piece for their weights.
template <int D, int ROWS>
__device__ __forceinline__ void join_rows(const CachedParams& p, const StepPiece& u, int warp, int lane) {
  constexpr int kPer = D / 32, kMine = (ROWS + kComputeWarps - 1) / kComputeWarps;
  using Vec = std::conditional_t<kPer == 2, float2, float4>;
  constexpr int kAhead = 4;        // pieces whose values are fetched with the references
  constexpr int kPieceFloats = kStepRows * (D + 2);
  const float* base = cached_part<true, D>(p, u.owner, 0);
  auto piece = [&](int i) { return (2 * i + (i == 0 ? 1 : 0)) * kPieceFloats; };
  int row[kMine];
  float top[kMine], neg[kMine], l[kMine], ref[kMine], sum[kMine];
  Vec y[kAhead][kMine];
  {
    const float* mine = base + piece(min(lane, u.pieces - 1)) + kStepRows * D;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      row[k] = min(warp + kComputeWarps * k, u.rows - 1);
      ref[k] = top[k] = __ldcg(mine + row[k]);
      sum[k] = __ldcg(mine + kStepRows + row[k]);
    }
  }
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const float* from = base + piece(min(j, u.pieces - 1)) + lane * kPer;
#pragma unroll
    for (int k = 0; k < kMine; ++k) y[j][k] = __ldcg(reinterpret_cast<const Vec*>(from + row[k] * D));
  }
#pragma unroll 1
  for (int i = lane + 32; i < u.pieces; i += 32)
#pragma unroll
    for (int k = 0; k < kMine; ++k) top[k] = fmaxf(top[k], __ldcg(base + piece(i) + kStepRows * D + row[k]));
  float o[kMine][kPer] = {};
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
#pragma unroll
    for (int w = 16; w; w >>= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], w));
    neg[k] = top[k] == -INFINITY ? 0.f : -top[k];
    l[k] = 0.f;
  }
  auto add = [&](const Vec& x, float w, float (&acc)[kPer]) {
    acc[0] = fmaf(w, x.x, acc[0]);
    acc[1] = fmaf(w, x.y, acc[1]);
    if constexpr (kPer == 4) {
      acc[2] = fmaf(w, x.z, acc[2]);
      acc[3] = fmaf(w, x.w, acc[3]);
    }
  };
#pragma unroll 1
  for (int b = 0; b < u.pieces; b += 32) {
    const int i = b + lane;
    float wt[kMine] = {};
    if (i < u.pieces)
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        if (b) {
          ref[k] = __ldcg(base + piece(i) + kStepRows * D + row[k]);
          sum[k] = __ldcg(base + piece(i) + kStepRows * (D + 1) + row[k]);
        }
        wt[k] = fast_exp2(ref[k] + neg[k]);
        l[k] += wt[k] * sum[k];
      }
    const int here = min(32, u.pieces - b);
    // four pieces' values at a time, the next four on their way
#pragma unroll 1
    for (int j = 0; j < here; j += kAhead) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const float* from = base + piece(min(b + j + a + kAhead, u.pieces - 1)) + lane * kPer;
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          const float w = __shfl_sync(0xffffffffu, wt[k], (j + a) & 31);
          if (j + a < here) add(y[a][k], w, o[k]);
          y[a][k] = __ldcg(reinterpret_cast<const Vec*>(from + row[k] * D));
        }
      }
    }
  }
  // a lane a row finishes its row's sums
  const int group = p.hq / p.c.hkv;
  float mine_l = 1.f, mine_top = 0.f;
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
#pragma unroll
    for (int w = 16; w; w >>= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], w);
    if (lane == k) mine_l = l[k], mine_top = top[k];
  }
  const int r = warp + kComputeWarps * lane, x = u.row + min(r, u.rows - 1), t = (int)(x * p.inv_group >> 16);
  const int h = u.h * group + x - t * group;
  const int64_t tok = u.start + t, at = (tok * p.hq + h) * D;
  const float inv = 1.f / mine_l;
  if (lane < kMine && r < u.rows) p.lse[(int64_t)h * p.c.T + tok] = (mine_top + log2f(mine_l)) * kLn2;
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const float f = __shfl_sync(0xffffffffu, inv, k);
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + __shfl_sync(0xffffffffu, at, k) + lane * kPer);
    if (warp + kComputeWarps * k >= u.rows) continue;
#pragma unroll
    for (int j = 0; j < kPer / 2; ++j) dst[j] = pack2<false>(o[k][2 * j] * f, o[k][2 * j + 1] * f);
  }
}

// NT: tiles of 8 query rows.
template <int D, bool E4M3, bool CAP, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    cached_step_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const CachedParams p) {
  using L = StepSmem<D, E4M3, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + L::kStages;
  uint64_t* unit_full = empty + L::kStages;
  uint64_t* unit_done = unit_full + kUnits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_let_next();
  const CachePlanView pv = cache_plan_view(p.c.plan, p.c.T, p.c.N, p.hq, p.c.hkv);
  ShareStart share;
  if (warp == kComputeWarps) share = pv.first[1][blockIdx.x];      // (beside the header; of use if there is a share)
  const int valid = cached_valid_rows(p);
  clear_rows<D>(p, valid, kThreads);
  if (valid == 0) return;
  const Shares sh = cached_shares<true>(pv.hdr);
  if ((int)blockIdx.x >= sh.n) return;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&full[i], E4M3 ? 1 + kScaleCopies : 1);
      mbar_init(&empty[i], kComputeWarps / 2);
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&unit_full[i], 33);            // the producer's lanes as their copies land, and the description
      mbar_init(&unit_done[i], kComputeWarps);
    }
    for (int i = 0; i < 2; ++i) reinterpret_cast<StepPiece*>(smem + L::kSplits)[i].tiles = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  __syncthreads();
  int* status = p.c.plan + kCpStatus;
  const int group = p.hq / p.c.hkv;
  auto token_of = [&](int row) { return (int)(row * p.inv_group >> 16); };       // row / group
  bool ok = true;
  uint32_t ring = 0;

  if (warp == kComputeWarps) {
    // ------------------------------------------------------------ producer
    const int P = 1 << p.c.page_shift, rows = min(P, kStepTile), per = kStepTile / rows;      // pages a tile
    const uint32_t page_bytes = 2 * rows * L::kRowBytes;
    const int64_t f1 = share.to;
    CachedUnit u = share.u;
    int64_t f = share.from;
    for (int n = 0; ok;) {
      int2 piece = make_int2(0, 0);
      if (f < f1) {
        if (n > 0) cached_next<true>(pv, u, p.hq, p.c.hkv);
        piece = cached_piece<true>(u, f, f1);
        if (piece.y == 0) continue;            // (only the share's end)
      }
      if (n >= kUnits && !(ok = warp_wait(&unit_done[n % kUnits], (n / kUnits - 1) & 1, status))) break;
      const int t0 = piece.x, t1 = piece.y;
      StepPiece x{};
      if (lane == 0) {
        x.t0 = t0;
        x.t1 = t1;
        x.tiles = u.tiles;
        x.tile = u.tile;
        x.h = u.h;
        x.row = u.row;
        x.rows = u.rows;
        x.start = u.start;
        x.pos0 = u.keys - u.count;
        x.keys = u.keys;
        x.lo = u.lo;
        *reinterpret_cast<StepPiece*>(smem + L::kUnit + (n % kUnits) * sizeof(StepPiece)) = x;
      }
      // page (or half page) i of the unit's tiles: where its keys are, or -1
      const int first = (u.tile + t0) * per, end = (u.tile + t1) * per;
      auto page_of = [&](int i) {
        const int pos = i * rows;
        if (i >= end || pos >= u.keys || pos + rows <= u.lo) return -1;
        const int page = cache_page(p.c, u.seq, pos >> p.c.page_shift);
        return page < 0 ? -1 : page * p.c.hkv + u.h;
      };
      int batch = first, now = page_of(first + lane), next = page_of(first + 32 + lane);
      // queries: 16 bytes a lane and copy, rows behind the unit's are zeros.  A row's token and head by a lane a row
      const int my_row = u.row + (lane < u.rows ? lane : 0), my_t = token_of(my_row);
      const int64_t my_at = ((int64_t)u.start + my_t) * p.hq + u.h * group + my_row - my_t * group;
      constexpr int kLanes = D / 8, kPer = 32 / kLanes;
#pragma unroll
      for (int i = 0; i < L::kRows / kPer; ++i) {
        const int r = i * kPer + lane / kLanes, c = lane % kLanes;
        const bool in = t1 > 0 && r < u.rows;
        const int64_t at = __shfl_sync(0xffffffffu, my_at, r);
        const __nv_bfloat16* src = p.q + (in ? at * D + 8 * c : 0);
        const uint32_t dst = smem_u32(smem + L::kQ + ((n % kUnits) * L::kRows + r) * D * 2 + 16 * c);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
      }
      cp_async_arrive(&unit_full[n % kUnits]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&unit_full[n % kUnits]);
      ++n;
      if (t1 == 0) break;
      for (int t = t0; t < t1 && ok; ++t, ++ring) {
        const int i = (u.tile + t) * per;
        if (i >= batch + 32) {
          batch += 32;
          now = next;
          next = page_of(batch + 32 + lane);
        }
        const int page = __shfl_sync(0xffffffffu, now, (i - batch + (lane < per ? lane : 0)) & 31);
        const bool load = lane < per && page >= 0;
        const uint32_t st = ring % L::kStages;
        if (ring >= L::kStages && !(ok = warp_wait(&empty[st], (ring / L::kStages - 1) & 1, status))) break;
        const int pages = __popc(__ballot_sync(0xffffffffu, load));
        if (lane == 0) {
          if (pages) mbar_arrive_expect_tx(&full[st], pages * page_bytes);
          else mbar_arrive(&full[st]);
        }
        __syncwarp();
        if (load) {
          const int slot = (i + lane) * rows & (P - 1);
          uint8_t* dst = smem + st * L::kStage + lane * rows * L::kBoxBytes;
#pragma unroll
          for (int b = 0; b < L::kBoxes; ++b) {
            tma_load_3d(dst + b * kStepTile * 128, &tm_k, &full[st], 128 * b, page, slot);
            tma_load_3d(dst + L::kTileBytes + b * kStepTile * 128, &tm_v, &full[st], 128 * b, page, slot);
          }
        }
        if constexpr (E4M3) {                  // a lane 16 keys' scales, K's then V's
          const int key = lane % (kScaleCopies / 2) * 16;
          const int at_page = __shfl_sync(0xffffffffu, now, (i - batch + key / rows) & 31);
          if (lane < kScaleCopies) {
            const bool v = lane >= kScaleCopies / 2;
            if (at_page >= 0)
              cp_async16(smem + st * L::kStage + L::kScales + (v ? kStepTile : 0) + key,
                         (v ? p.c.v_scales : p.c.k_scales) + ((int64_t)at_page << p.c.page_shift) + ((i * rows + key) & (P - 1)));
            cp_async_arrive(&full[st]);
          }
        }
        __syncwarp();
      }
      // (read by the compute warps from the next unit's start on)
      if (lane == 0 && t1 - t0 < u.tiles) {
        const int2 c = cached_owners<true>(u, sh, t0, t1);
        x.owner = c.x;
        x.pieces = c.y;
        reinterpret_cast<StepPiece*>(smem + L::kSplits)[t0 == 0 ? 1 : 0] = x;
      }
    }
    // nothing may land after the CTA has left (reached early only when a wait ran out)
    for (uint32_t x = ring > L::kStages ? ring - L::kStages : 0; x < ring; ++x)
      mbar_wait(&full[x % L::kStages], (x / L::kStages) & 1, status);
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  // -------------------------------------------------------------- compute
  constexpr int kSteps = D / 16;
  constexpr int kWords = L::kRowBytes / 8 / 4;       // a lane's words of a value row
  constexpr int kOut = D / 16;                       // tiles of 16 head dimensions
  const int g = lane >> 2, q = lane & 3, pair = warp >> 1;
  float* red = reinterpret_cast<float*>(smem + L::kRed);
  float* stat = reinterpret_cast<float*>(smem + L::kStat);
  // this lane's places in a stage: words of key row g and of value rows 2 q and 2 q + 1 of the warp's first 8 keys
  constexpr int kLoads = E4M3 ? D / 64 : 2;
  const int key0 = 32 * (warp & 1);
  int at_k[kLoads], at_v[2];
#pragma unroll
  for (int j = 0; j < kLoads; ++j)
    at_k[j] = key0 * L::kBoxBytes + (E4M3 ? swz_offset(g, (D / 4) * q + 16 * j, L::kBoxBytes) : swz_offset(g, (2 * q + j) * 16, 128));
#pragma unroll
  for (int k = 0; k < 2; ++k)
    at_v[k] = L::kTileBytes + key0 * L::kBoxBytes + swz_offset(2 * q + k, kWords >= 4 ? 16 * g : 8 * g, L::kBoxBytes);
  // (g's words lie 64 bytes apart with D = 128 codes, 32 otherwise)
  auto turn = [](int row) { return E4M3 && D == 128 ? row >> 1 & 3 : (row >> 1 & 1) | (row >> 2 & 1) << 2; };
  StepPiece* splits = reinterpret_cast<StepPiece*>(smem + L::kSplits);
  int pending = -1;
  for (int n = 0; ok; ++n) {
    // (the warps meet here too: the last unit's sums have been read, and where a wait ran out all of them leave)
    ok = named_bar_and(1, kComputeWarps * 32, warp_wait(&unit_full[n % kUnits], (n / kUnits) & 1, status));
    if (!ok) break;
    // a split unit's piece is counted here and not where it ended: by now its stores have landed
    if (pending >= 0 && threadIdx.x == 0) splits[pending].last = cached_last(pv.done + splits[pending].owner, splits[pending].pieces);
    pending = -1;
    const StepPiece u = *reinterpret_cast<const StepPiece*>(smem + L::kUnit + (n % kUnits) * sizeof(StepPiece));
    if (u.t1 == 0) break;
    // queries as the products' second operand: row 8 t + g, four head dimensions a step of 16.  Scores and
    // weights then are of rows 8 t + 2 q and + 1.  Two row tiles' operands are kept in shared memory, in the
    // queries' place, a 16-byte word a lane and step: in registers they spill (179 instead of 111 us on two
    // sequences of 131972, 16 rows)
    constexpr bool kShared = NT == 2;
    uint8_t* frag = smem + L::kQ + (n % kUnits) * L::kRows * D * 2 + lane * 16;
    uint32_t b[kSteps][NT][2];
    float2 rowf[NT];
    int pos[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint8_t* src = smem + L::kQ + ((n % kUnits) * L::kRows + 8 * t + g) * D * 2;
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int d0 = E4M3 ? (D / 4) * q + 4 * s : (s >> 2) * 64 + (2 * q + ((s >> 1) & 1)) * 8 + (s & 1) * 4;
        const uint2 w = *reinterpret_cast<const uint2*>(src + d0 * 2);
        b[s][t][0] = w.x;
        b[s][t][1] = w.y;
        if constexpr (E4M3) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            top = fmax3(top, fabsf(__uint_as_float(b[s][t][k] << 16)), fabsf(__uint_as_float(b[s][t][k] & 0xffff0000u)));
        }
      }
      const float f = CAP ? 1.f : p.scale2;
      rowf[t] = make_float2(f, f);
      if constexpr (E4M3) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int shift = min(14 + 127 - (int)(__float_as_uint(top) >> 23), 126);     // (a row of zeros: any)
        const float up = exp2i(shift), down = f * exp2i(-shift);
        rowf[t] = make_float2(__shfl_sync(0xffffffffu, down, 8 * q), __shfl_sync(0xffffffffu, down, 8 * q + 4));
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            b[s][t][k] = pack2<true>(__uint_as_float(b[s][t][k] << 16) * up, __uint_as_float(b[s][t][k] & 0xffff0000u) * up);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 8 * t + 2 * q + r;
        pos[t][r] = u.pos0 + token_of(u.row + (row < u.rows ? row : 0));
      }
    }
    if constexpr (kShared) {
      named_bar_sync(1, kComputeWarps * 32);           // every warp has read the queries
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        if (s / (kSteps / kComputeWarps) == warp)
          *reinterpret_cast<uint4*>(frag + s * 512) = make_uint4(b[s][0][0], b[s][0][1], b[s][NT - 1][0], b[s][NT - 1][1]);
      named_bar_sync(1, kComputeWarps * 32);
    } else {
      __syncwarp();
      if (lane == 0) mbar_arrive(&unit_done[n % kUnits]);
    }
    auto operand = [&](int s, uint32_t (&y)[NT][2]) {
      if constexpr (kShared) {
        const uint4 f = *reinterpret_cast<const uint4*>(frag + s * 512);
        y[0][0] = f.x;
        y[0][1] = f.y;
        y[NT - 1][0] = f.z;
        y[NT - 1][1] = f.w;
      } else {
#pragma unroll
        for (int t = 0; t < NT; ++t) y[t][0] = b[s][t][0], y[t][1] = b[s][t][1];
      }
    };
    float o[kOut][NT][4] = {};
    float m[NT][2], M[NT][2];
    float2 l[NT], neg[NT], Neg[NT];      // neg, Neg: -m and 13 - M, 0 while they are infinite
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = M[t][0] = M[t][1] = -INFINITY;
      l[t] = neg[t] = Neg[t] = make_float2(0.f, 0.f);
    }
    auto scale_rows = [&](int t, float f0, float f1) {
#pragma unroll
      for (int d = 0; d < kOut; ++d) {
        o[d][t][0] *= f0;
        o[d][t][1] *= f1;
        o[d][t][2] *= f0;
        o[d][t][3] *= f1;
      }
    };
    const int all_see = u.pos0 + token_of(u.row) + 1 - kStepTile;          // tiles up to this key hide none behind a row's position
    const int window = p.left < 0 ? -1 : u.pos0 + token_of(u.row + u.rows - 1) - p.left;    // tiles from this key on none before one
    for (int tile = u.t0; tile < u.t1; ++tile, ++ring) {
      if ((ring & 1) != (uint32_t)pair) continue;
      const uint32_t st = ring % L::kStages;
      if (ok) ok = warp_wait(&full[st], (ring / L::kStages) & 1, status);
      if (!ok) continue;
      const uint8_t* stage = smem + st * L::kStage;
      const int c0 = (u.tile + tile) * kStepTile;
      const bool edge = c0 + kStepTile > u.keys || c0 < u.lo;       // what is no key of the sequence may be anything
      // scores of keys c0 + key0 + 16 i + 8 h + g, in four chains of products
      constexpr int kChains = NT == 1 ? 2 : 1;
      float2 x[2][2][NT];        // [i][h][t]
      {
        float s[2][kChains][NT][4] = {};
        if constexpr (E4M3) {
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            uint4 w[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h) w[i][h] = *reinterpret_cast<const uint4*>(stage + at_k[j] + (16 * i + 8 * h) * L::kBoxBytes);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t y[NT][2];
              operand(4 * j + k, y);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t w0 = (&w[i][0].x)[k], w1 = (&w[i][1].x)[k];
                const uint32_t a[4] = {codes_f16(w0), codes_f16(w1), codes_f16_hi(w0), codes_f16_hi(w1)};
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816<true>(s[i][k % kChains][t], a, y[t][0], y[t][1]);
              }
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            uint32_t y0[NT][2], y1[NT][2];
            operand(2 * j, y0);
            operand(2 * j + 1, y1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint4 w[2];
#pragma unroll
              for (int h = 0; h < 2; ++h)
                w[h] = *reinterpret_cast<const uint4*>(stage + at_k[j & 1] + (j >> 1) * kStepTile * 128 + (16 * i + 8 * h) * 128);
              const uint32_t a0[4] = {w[0].x, w[1].x, w[0].y, w[1].y}, a1[4] = {w[0].z, w[1].z, w[0].w, w[1].w};
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                mma16816<false>(s[i][0][t], a0, y0[t][0], y0[t][1]);
                mma16816<false>(s[i][kChains - 1][t], a1, y1[t][0], y1[t][1]);
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              x[i][h][t] = make_float2(s[i][0][t][2 * h], s[i][0][t][2 * h + 1]);
              if constexpr (kChains == 2) x[i][h][t] = fadd2(x[i][h][t], make_float2(s[i][1][t][2 * h], s[i][1][t][2 * h + 1]));
              if constexpr (!E4M3) x[i][h][t] = fmul2(x[i][h][t], rowf[t]);
            }
      }
      float e[2][2];           // exponents of the values' scales
      if constexpr (E4M3) {
        float k[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t* sc = stage + L::kScales + key0 + 16 * i + 8 * h + g;
            k[i][h] = __uint_as_float(max((uint32_t)sc[0] << 23, 0x00400000u));       // 2^(byte - 127)
            e[i][h] = __uint_as_float(0x4b000000u | sc[kStepTile]) - 8388735.f;       // (2^23 + byte by its bits) - 2^23 - 127
            if (edge) {
              const int key = c0 + key0 + 16 * i + 8 * h + g;
              if (key >= u.keys || key < u.lo) k[i][h] = 1.f, e[i][h] = 0.f;
            }
          }
        // byte 255: infinite, and 128; infinities have 247 or more
        if (__any_sync(0xffffffffu, fmaxf(fmax3(k[0][0], k[0][1], k[1][0]), k[1][1]) >= 0x1p120f ||
                                        fmaxf(fmax3(e[0][0], e[0][1], e[1][0]), e[1][1]) > 119.5f)) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (k[i][h] == INFINITY) k[i][h] = NAN;
              if (e[i][h] > 127.5f) e[i][h] = NAN;
            }
          // Infinities, a row of the cache at a time.  A row of values that is nothing but them and zeros then needs no weight: its
          // scale must not cost the others theirs
          uint32_t pure = 0;
#pragma unroll 1
          for (int n = 0; n < 32; ++n) {
            const int key = c0 + key0 + n;
            const uint32_t from_k = infinite_from(stage[L::kScales + key0 + n]), from_v = infinite_from(stage[L::kScales + kStepTile + key0 + n]);
            if ((from_k & from_v) == kNoInfinity || key >= u.keys || key < u.lo) continue;
            if (from_k != kNoInfinity) {        // products of row 8 t + g, then on top of the scores of rows 8 t + 2 q and + 1
              float sum[NT] = {};
              if constexpr (kShared) {
                const float2 y = infinite_products<D>(stage + key0 * L::kBoxBytes + swz_offset(n, (D / 4) * q, L::kBoxBytes), frag, from_k);
                sum[0] = y.x;
                sum[NT - 1] = y.y;
              } else {
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                  const uint32_t w = *reinterpret_cast<const uint32_t*>(stage + key0 * L::kBoxBytes + swz_offset(n, (D / 4) * q + 4 * s, L::kBoxBytes));
                  uint32_t y[NT][2];
                  operand(s, y);
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const uint32_t c = w >> 8 * j & 255;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                      if ((c & 127) >= from_k) sum[t] += signed_infinity(c) * __half2float(__ushort_as_half((unsigned short)(y[t][j >> 1] >> 16 * (j & 1))));
                  }
                }
              }
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                sum[t] += __shfl_xor_sync(0xffffffffu, sum[t], 1);
                sum[t] += __shfl_xor_sync(0xffffffffu, sum[t], 2);
                const float s0 = __shfl_sync(0xffffffffu, sum[t], 8 * q), s1 = __shfl_sync(0xffffffffu, sum[t], 8 * q + 4);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    if (n == 16 * i + 8 * h + g) x[i][h][t] = make_float2(x[i][h][t].x + s0, x[i][h][t].y + s1);
              }
            }
            if (from_v == kNoInfinity) continue;
            const uint8_t* row = stage + L::kTileBytes + key0 * L::kBoxBytes + swz_offset(n, 4 * kWords * g, L::kBoxBytes);
            bool sees[NT][2], finite = false;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int r = 0; r < 2; ++r) sees[t][r] = key <= pos[t][r] && !(p.left >= 0 && key < pos[t][r] - p.left);
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
              const uint32_t c = row[d];
              const bool infinite = (c & 127) >= from_v;
              finite = finite || (!infinite && (c & 127));
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                  if (infinite && sees[t][r]) o[d / 2][t][2 * (d & 1) + r] += signed_infinity(c);
            }
            if (!__any_sync(0xffffffffu, finite) && (n & 7) == g) pure |= 1u << (n >> 3);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (pure >> (2 * i + h) & 1) e[i][h] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t)           // (the scales first: with either alone a product may leave fp32's range)
              x[i][h][t] = fmul2(x[i][h][t], fmul2(rowf[t], make_float2(k[i][h], k[i][h])));
      }
      if constexpr (CAP) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t)
              x[i][h][t] = make_float2(cap_one(x[i][h][t].x, p.capf) * p.scale2, cap_one(x[i][h][t].y, p.capf) * p.scale2);
      }
      if (c0 > all_see || c0 < window) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = c0 + key0 + 16 * i + 8 * h + g;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if (key > pos[t][0] || (p.left >= 0 && key < pos[t][0] - p.left)) x[i][h][t].x = -INFINITY;
              if (key > pos[t][1] || (p.left >= 0 && key < pos[t][1] - p.left)) x[i][h][t].y = -INFINITY;
            }
          }
      }
      float mx[NT][2];
      auto maxima = [&]() {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mx[t][0] = fmaxf(fmax3(x[0][0][t].x, x[0][1][t].x, x[1][0][t].x), x[1][1][t].x);
          mx[t][1] = fmaxf(fmax3(x[0][0][t].y, x[0][1][t].y, x[1][0][t].y), x[1][1][t].y);
        }
      };
      auto over = [&](const float (&top)[NT][2]) {
        bool any = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) any = any || mx[t][0] > top[t][0] + kSlack || mx[t][1] > top[t][1] + kSlack;
        return __any_sync(0xffffffffu, any);
      };
      auto reduce = [&](float y) {        // over the keys
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
        return fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
      };
      maxima();
      if (over(m)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float f[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float m1 = fmaxf(m[t][r], reduce(mx[t][r])), down = m1 == m[t][r] ? 0.f : m[t][r] - m1;
            f[r] = fast_exp2(down);
            m[t][r] = m1;
            if constexpr (E4M3) M[t][r] += down;
          }
          neg[t] = make_float2(m[t][0] == -INFINITY ? 0.f : -m[t][0], m[t][1] == -INFINITY ? 0.f : -m[t][1]);
          l[t] = fmul2(l[t], make_float2(f[0], f[1]));
          if constexpr (E4M3)
            Neg[t] = make_float2(M[t][0] == -INFINITY ? 0.f : kBoost - M[t][0], M[t][1] == -INFINITY ? 0.f : kBoost - M[t][1]);
          else
            scale_rows(t, f[0], f[1]);
        }
      }
      uint32_t w[2][2][NT];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            x[i][h][t] = fadd2(x[i][h][t], neg[t]);
            const float2 y = make_float2(fast_exp2(x[i][h][t].x), fast_exp2(x[i][h][t].y));
            l[t] = fadd2(l[t], y);
            if constexpr (E4M3) x[i][h][t] = fadd2(x[i][h][t], make_float2(e[i][h], e[i][h]));
            else w[i][h][t] = pack2<false>(y.x, y.y);
          }
      if constexpr (E4M3) {
        maxima();
        if (over(M)) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float f[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float M1 = fmaxf(M[t][r], reduce(mx[t][r]));
              f[r] = fast_exp2(M1 == M[t][r] || M[t][r] == -INFINITY ? 0.f : M[t][r] - M1);      // (so far zeros, or infinities)
              M[t][r] = M1;
            }
            Neg[t] = make_float2(M[t][0] == -INFINITY ? 0.f : kBoost - M[t][0], M[t][1] == -INFINITY ? 0.f : kBoost - M[t][1]);
            scale_rows(t, f[0], f[1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const float2 y = fadd2(x[i][h][t], Neg[t]);
              w[i][h][t] = pack2<true>(fast_exp2(y.x), fast_exp2(y.y));
            }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int t = 0; t < NT; ++t) w[i][h][t] = transpose8(w[i][h][t]);
        // values of keys 16 i + 2 q, + 1, + 8, + 9
        uint32_t v[4][kWords];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint8_t* src = stage + at_v[k & 1] + (16 * i + 8 * (k >> 1)) * L::kBoxBytes;
          if constexpr (kWords >= 4) {
#pragma unroll
            for (int j = 0; j < kWords / 4; ++j) {
              const uint4 y = *reinterpret_cast<const uint4*>(src + j * kStepTile * 128);
              v[k][4 * j] = y.x;
              v[k][4 * j + 1] = y.y;
              v[k][4 * j + 2] = y.z;
              v[k][4 * j + 3] = y.w;
            }
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(src);
            v[k][0] = y.x;
            v[k][1] = y.y;
          }
          if (edge) {                              // weight 0 does not silence an infinity
            const int key = c0 + key0 + 16 * i + 8 * (k >> 1) + 2 * q + (k & 1);
            if (key >= u.keys || key < u.lo) {
#pragma unroll
              for (int j = 0; j < kWords; ++j) v[k][j] = 0;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          if constexpr (E4M3) {
            const uint32_t x0 = __byte_perm(v[0][j], v[1][j], 0x5140), x1 = __byte_perm(v[0][j], v[1][j], 0x7362);
            const uint32_t y0 = __byte_perm(v[2][j], v[3][j], 0x5140), y1 = __byte_perm(v[2][j], v[3][j], 0x7362);
            const uint32_t a0[4] = {codes_f16(x0), codes_f16_hi(x0), codes_f16(y0), codes_f16_hi(y0)};
            const uint32_t a1[4] = {codes_f16(x1), codes_f16_hi(x1), codes_f16(y1), codes_f16_hi(y1)};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              mma16816<true>(o[2 * j][t], a0, w[i][0][t], w[i][1][t]);
              mma16816<true>(o[2 * j + 1][t], a1, w[i][0][t], w[i][1][t]);
            }
          } else {
            const uint32_t a[4] = {__byte_perm(v[0][j], v[1][j], 0x5410), __byte_perm(v[0][j], v[1][j], 0x7632),
                                   __byte_perm(v[2][j], v[3][j], 0x5410), __byte_perm(v[2][j], v[3][j], 0x7632)};
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816<false>(o[j][t], a, w[i][0][t], w[i][1][t]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    // the unit's, or its piece's, end: the warps meet
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = r ? l[t].y : l[t].x;
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        if (g == 0) {
          float* y = stat + warp * 2 * L::kRows + 8 * t + 2 * q + r;
          y[0] = m[t][r];
          y[L::kRows] = sum;
        }
      }
    if (kShared) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&unit_done[n % kUnits]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 8 * t + 2 * q + r;
        if (row >= u.rows) continue;
        // values in units of 2^(M - 13) against m, M from some -130 to 130: in two factors that both stay within fp32's range
        // (fast_exp2 gives 0 below 2^-126), the first one far from where the values would leave it
        const float toward = M[t][r] < -64.f ? 64.f : M[t][r] > 64.f ? -64.f : 0.f;
        const float to = !E4M3 || M[t][r] == -INFINITY ? 1.f : fast_exp2(M[t][r] + toward), by = E4M3 ? exp2i(-(int)(kBoost + toward)) : 1.f;
        // head dimensions (D / 8) g + 2 d and + 1 of product tile d; bf16: of each half of the row's 8 g + 2 (d mod 4).
        // In words of 16 bytes whose places turn with the row, so that eight lanes (two g, four q) take all banks
        float* dst = red + (warp * L::kRows + row) * D;
#pragma unroll
        for (int d = 0; d < kOut; d += 2)
          *reinterpret_cast<float4*>(dst + 4 * (((E4M3 ? (D / 8) * g + 2 * d : (d >> 2) * 64 + 8 * g + 2 * (d & 3)) >> 2) ^ turn(row))) =
              make_float4(o[d][t][r] * by * to, o[d][t][2 + r] * by * to, o[d + 1][t][r] * by * to, o[d + 1][t][2 + r] * by * to);
      }
    ok = named_bar_and(1, kComputeWarps * 32, ok);
    if (!ok) break;
    const bool whole = u.t0 == 0 && u.t1 == u.tiles;
    if (!whole) pending = u.t0 == 0 ? 1 : 0;
    float* part = cached_part<true, D>(p, blockIdx.x, u.t0 == 0 ? 1 : 0);
    constexpr int kQuads = D / 4;
    for (int y = threadIdx.x; y < u.rows * kQuads; y += kComputeWarps * 32) {
      const int r = y / kQuads, c = y % kQuads;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float top = -INFINITY, tot = 0.f;
#pragma unroll
      for (int w = 0; w < kComputeWarps; ++w) top = fmaxf(top, stat[w * 2 * L::kRows + r]);
#pragma unroll
      for (int w = 0; w < kComputeWarps; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(red + (w * L::kRows + r) * D + 4 * (c ^ turn(r)));
        const float mw = stat[w * 2 * L::kRows + r], f = mw == top ? 1.f : fast_exp2(mw - top);     // (a warp that saw nothing: 0)
        sum = make_float4(fmaf(z.x, f, sum.x), fmaf(z.y, f, sum.y), fmaf(z.z, f, sum.z), fmaf(z.w, f, sum.w));
        tot = fmaf(stat[w * 2 * L::kRows + L::kRows + r], f, tot);
      }
      if (whole) {
        const int t = token_of(u.row + r), h = u.h * group + u.row + r - t * group;
        const int64_t tok = u.start + t;
        const float inv = 1.f / tot;
        *reinterpret_cast<uint2*>(p.out + (tok * p.hq + h) * D + 4 * c) =
            make_uint2(pack2<false>(sum.x * inv, sum.y * inv), pack2<false>(sum.z * inv, sum.w * inv));
        if (c == 0) p.lse[(int64_t)h * p.c.T + tok] = (top + log2f(tot)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(part + r * D + 4 * c) = sum;
        if (c == 0) {
          part[kStepRows * D + r] = top;
          part[kStepRows * (D + 1) + r] = tot;
        }
      }
    }
  }
  // Split units: the last of their pieces to be finished joins them, at its share's end.
  if (!ok) return;
  named_bar_sync(1, kComputeWarps * 32);
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const StepPiece u = splits[i];
    if (u.tiles && u.last) join_rows<D, L::kRows>(p, u, warp, lane);
  }
}

template <int D, bool E4M3, bool CAP, int NT>
cudaError_t launch(const CachedParams& p, cudaStream_t stream) {
  using L = StepSmem<D, E4M3, NT>;
  CUtensorMap tk, tv;
  const uint64_t P = (uint64_t)1 << p.c.page_shift, pages = (uint64_t)p.c.num_pages * p.c.hkv;
  const uint32_t rows = P < kStepTile ? (uint32_t)P : kStepTile;
  if (!make_tmap_u8_3d(&tk, p.c.k, L::kRowBytes, pages, P, P * L::kRowBytes, L::kRowBytes, L::kBoxBytes, rows) ||
      !make_tmap_u8_3d(&tv, p.c.v, L::kRowBytes, pages, P, P * L::kRowBytes, L::kRowBytes, L::kBoxBytes, rows))
    return cudaErrorInvalidValue;
  cudaError_t e = prepare_kernel<cached_step_kernel<D, E4M3, CAP, NT>>(L::kAlloc);
  if (e != cudaSuccess) return e;
  cached_step_kernel<D, E4M3, CAP, NT><<<kStepCtas, kThreads, L::kAlloc, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

template <int D, int NT>
cudaError_t launch_d(bool e4m3, const CachedParams& p, cudaStream_t s) {
  if (e4m3) return p.cap > 0.f ? launch<D, true, true, NT>(p, s) : launch<D, true, false, NT>(p, s);
  return p.cap > 0.f ? launch<D, false, true, NT>(p, s) : launch<D, false, false, NT>(p, s);
}

template <int D>
cudaError_t launch_all(bool e4m3, const CachedParams& p, cudaStream_t s) {
  const int group = p.hq / p.c.hkv;
  const int64_t most = (int64_t)p.max_chunk * group;
  const int limit = step_rows(group, p.max_chunk);
  const bool steps = group <= limit, chunks = most > limit;
  cudaError_t e = cudaSuccess;
  if (steps) e = (most < limit ? most : limit) <= 8 ? launch_d<D, 1>(e4m3, p, s) : launch_d<D, 2>(e4m3, p, s);
  if (e == cudaSuccess && chunks) e = launch_cached_chunk(D, e4m3, p, !steps, s);
  return e;
}

}  // namespace

cudaError_t launch_cached_fwd(int D, bool e4m3, const CachedParams& p, cudaStream_t s) {
  return D == 128 ? launch_all<128>(e4m3, p, s) : launch_all<64>(e4m3, p, s);
}

}  // namespace flamia
