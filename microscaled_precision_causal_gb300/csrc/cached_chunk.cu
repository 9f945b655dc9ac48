// Attention over the paged cache for chunks: more rows of a kv head than a step takes.
//
// The scored forward's scheme (bf16 tcgen05 MMAs, two tiles of 128 rows in turn, P in tensor memory over the
// scores it came from, a reference m near the row's maximum) with three differences:
//   - A tile's rows are a kv head's: the new tokens' query heads that share it, token by token.  With
//     grouped heads a key tile thus serves all of them, and short chunks still fill a tile.
//   - Key tiles come from pages, a TMA copy a page.  E4M3 codes go to a raw ring, from which four
//     warps write the bf16 tiles that the products read: code times scale is exact in bf16.
//     A thread unpacks a key's row, so the scale is one register; both sides are free of bank
//     conflicts by the copies' and the products' swizzles.
//   - All units' key tiles are dealt out in equal shares (cache.cuh): one chunk over a long context
//     keeps every SM busy, and the pieces are joined after.  Both warpgroups on the key tiles of a unit of one row tile, in
//     turn, gained little (16 sequences of 26 rows of 4 heads 16.7 -> 15.3 us, 11 of 86 17.4 -> 19.1) and cost the
//     others (4 x 1024 with a window 74.5 -> 77.8).
// Keys behind the sequence or before every row's window are zeros to the products, whatever the page holds.
//
// Roles (512 threads):
//   warp 0        producer: K and V tiles, page by page
//   warp 1        MMA issuer (at D = 64 of the first row tile; warp 3 of the second)
//   warp 2        TMEM allocator; finds the units ahead and loads their queries
//   warps 4-11    softmax, a warpgroup per row tile, thread = row; they write the unit's O too
//   warps 12-15   E4M3: unpack (eight warps, four each for K and V, at 136 registers for the softmax: 475 instead of 419
//                 us for a chunk of 2048 behind 14336)
// TMEM columns as in the scored forward.
//
// Bound by the chain of scores, softmax and values of two row tiles in turn, the tensor cores busy half the time, and at d 64
// by the softmax's arithmetic.  Measured: a chunk of 2048 behind 14336, 32 heads on 8, d 128, E4M3 415 us, 1240 TFLOP/s (65% of
// cuBLAS's bf16; bf16 pages 376); 4 chunks of 1024 with a window of 2048, 16 heads, d 64 76 us.
#include <type_traits>

#include "cache.cuh"
#include "ptx.cuh"
#include "tmap.h"

namespace flamia {

namespace {

constexpr int kThreads = 512;
constexpr float kRescaleAbove = 8.f, kLoose = 64.f;
constexpr int kLaunchRegs = (65536 / kThreads) & ~7;
constexpr int kRegCtl = 64, kRegUnpack = 80, kRegSoftmax = 184;
static_assert(kRegCtl * 128 + kRegUnpack * 128 + kRegSoftmax * 256 <= kLaunchRegs * kThreads, "register split");

// x - m is one multiply-add while m was rounded: from |m| = 2^28 on both are shrunk (as in the scored forward).
__device__ __forceinline__ float shrink_for(float m) {
  const uint32_t e = (__float_as_uint(m) >> 23) & 255;
  return e >= 127 + 28 && e < 255 ? __uint_as_float((2 * 127 + 28 - e) << 23) : 1.f;
}

// A unit's piece as the roles need it.  Key tiles last, last - 1, ..., last - tiles + 1: a causal row's
// largest scores tend to be near.
struct alignas(16) Piece {
  int tiles, last;                 // 0 tiles: no more
  int h, row, rows, ntq;
  int start, pos0, keys, lo;       // first token of the sequence, and its position; keys; first key seen by any row
  int seq, slot;                   // slot of the workspace, or -1: a whole unit
  int owner, pieces;               // of a split unit: the CTA that has its beginning, the CTAs that have pieces
  uint8_t ended[8];                // whether this CTA's piece was finished last, by the rows' warps
};
static_assert(sizeof(Piece) == 64, "read as four 16-byte words");
constexpr int kUnits = 4;
constexpr int kScaleCopies = kTile / 16;     // of 16 bytes, a tile

__device__ __forceinline__ Piece read_piece(const uint8_t* units, uint64_t* full, uint64_t* done, int n, bool whole_warp, bool& ok,
                                            int* status) {
  ok = mbar_wait(&full[n % kUnits], (n / kUnits) & 1, status);
  if (whole_warp) ok = __all_sync(0xffffffffu, ok);
  union {
    Piece p;
    int4 w[4];
  } x;
  const int4* src = reinterpret_cast<const int4*>(units + (n % kUnits) * sizeof(Piece));
#pragma unroll
  for (int i = 0; i < 4; ++i) x.w[i] = src[i];
  if (whole_warp) __syncwarp();
  if (!whole_warp || (threadIdx.x & 31) == 0) mbar_arrive(&done[n % kUnits]);
  if (!ok) x.p.tiles = 0;
  return x.p;
}

// Four products x -> a + b / (1 + 2^(z2 x)): with b = -2 a the tanh cap, in whatever units a is.  Reciprocals are a quarter
// as fast as exponentials, so the four share one, of their product (each at most 1 + 2^30: beyond, 1 - 2^-29).
__device__ __forceinline__ void tanh4(float2& x, float2& y, float z2, float a, float b) {
  x = fmul2(x, make_float2(z2, z2));
  y = fmul2(y, make_float2(z2, z2));
  const float2 one = make_float2(1.f, 1.f);
  // (a NaN stays one)
  x = fadd2(make_float2(fast_exp2(x.x > 30.f ? 30.f : x.x), fast_exp2(x.y > 30.f ? 30.f : x.y)), one);
  y = fadd2(make_float2(fast_exp2(y.x > 30.f ? 30.f : y.x), fast_exp2(y.y > 30.f ? 30.f : y.y)), one);
  const float2 xy = fmul2(make_float2(x.x, y.x), make_float2(x.y, y.y));
  const float r = fast_rcp(xy.x * xy.y) * b;
  const float2 rr = fmul2(make_float2(r, r), make_float2(xy.y, xy.x));
  x = ffma2(make_float2(x.y, x.x), make_float2(rr.x, rr.x), make_float2(a, a));
  y = ffma2(make_float2(y.y, y.x), make_float2(rr.y, rr.y), make_float2(a, a));
}
// 32 products of a row capped, in their own units: by a polynomial where every product of the warp's rows allows it, else
// by tanh4, whose error beside 0 is some 2^-22 of the cap: only columns with scores near the cap get it.
__device__ __forceinline__ void cap_columns(uint32_t (&v)[32], const CapForm& F, bool counts) {
  float m[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 32; j += 4)
#pragma unroll
    for (int g = 0; g < 2; ++g) m[g] = fmax3(m[g], fabsf(__uint_as_float(v[j + 2 * g])), fabsf(__uint_as_float(v[j + 2 * g + 1])));
  if (!__any_sync(0xffffffffu, counts && !(fmaxf(m[0], m[1]) <= F.t5))) {
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 x = pair_of(v, j), w = fmul2(x, x);
      float2 t = ffma2(w, F.k5[4], F.k5[3]);
      t = ffma2(w, t, F.k5[2]);
      t = ffma2(w, t, F.k5[1]);
      t = ffma2(w, t, F.k5[0]);
      put_pair(v, j, ffma2(x, fmul2(w, t), x));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      float2 x = pair_of(v, j), y = pair_of(v, j + 2);
      tanh4(x, y, F.zscale * (2.f * kLog2e), F.inv, -2.f * F.inv);
      put_pair(v, j, x);
      put_pair(v, j + 2, y);
    }
  }
}
// Largest product of a row's 128, or largest magnitude.
template <bool ABS>
__device__ __forceinline__ float columns_max(uint32_t s_addr) {
  uint32_t v[4][32];
  float m[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if constexpr (ABS) tmem_ld32_absmax(s_addr + 32 * g, v[g], m[g]);
    else tmem_ld32_max(s_addr + 32 * g, v[g], m[g]);
  }
  tmem_ld_wait();
  return fmaxf(fmax3(m[0], m[1], m[2]), m[3]);
}

template <int D, bool E4M3>
struct ChunkSmem {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kSlots = D == 128 ? 4 : 8;           // K and V tiles in turn
  static constexpr int kRaw = E4M3 ? (D == 128 ? 2 : 4) : 0;
  static constexpr int kRawBytes = kTile * D;
  static constexpr int kQ = 0;                              // [2]
  static constexpr int kKV = 2 * kTileBytes;
  static constexpr int kCodes = kKV + kSlots * kTileBytes;
  static constexpr int kScales = kCodes + kRaw * kRawBytes; // [kRaw][128]
  static constexpr int kUnit = kScales + kRaw * kTile;
  static constexpr int kSplits = kUnit + kUnits * (int)sizeof(Piece);   // the share's split units, by slot
  static constexpr int kBar = kSplits + 2 * (int)sizeof(Piece);
  static constexpr int kBytes = kBar + 512;
  static constexpr int kAlloc = kBytes + 1024;
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&x);
}
// Two codes of a word (the pair that SEL picks, each extended by its sign to a half word) times 2^-120 as bf16: exponent
// and mantissa bits four places up, the sign's other copies masked.  Subnormal codes become subnormal values of
// the same meaning.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
  uint32_t x;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(x) : "r"(w), "n"(SEL));
  return (x << 4) & 0x87f087f0u;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a));
  return x;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Row r of a tile of codes -> bf16 values times their scale 2^(b - 127).  One factor 2^(b - 7) up to b = 134; above,
// 2^120 first, then 2^(b - 127) (NaN for 255).
template <int D, bool BIG>
__device__ __forceinline__ void unpack_row(uint32_t raw, uint32_t tile, int r, uint32_t b) {
  const uint32_t f1 = BIG ? 0x7b807b80u : (b + 120) * 0x00800080u, f2 = b == 255 ? 0x7fc07fc0u : b * 0x00800080u;
  const uint32_t src = raw + swz_offset(r, 0, D), dst = tile + swz_offset(r, 0, 128);
  // (all loads first: one warp a scheduler unpacks, so what it waits for is its own latencies)
  uint4 c[D / 16];
#pragma unroll
  for (int j = 0; j < D / 16; ++j) c[j] = lds128(src ^ (16 * j));
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    const uint32_t w[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = mul_bf16x2(codes_bf16<0x9180>(w[i]), f1);
      y[2 * i + 1] = mul_bf16x2(codes_bf16<0xb3a2>(w[i]), f1);
    }
    if constexpr (BIG) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = mul_bf16x2(y[i], f2);
    }
    // (the tiles are aligned to their swizzle's period, so a column is an exclusive or)
    const uint32_t to = (dst ^ (32 * j & 127)) + (32 * j >> 7) * kTile * 128;
    sts128(to, y[0], y[1], y[2], y[3]);
    sts128(to ^ 16, y[4], y[5], y[6], y[7]);
  }
}

// The rows of a warp of row tile w from all pieces: references and sums with a lane a row, then values with eight
// lanes a row, of some rows and four pieces at a time: it is a matter of loads in flight.
template <int D>
__device__ __forceinline__ void join_rows(const CachedParams& p, const Piece& U, int w, int quarter, int lane) {
  constexpr int kPer = D / 32, kGroups = D == 64 ? 4 : 2, kPieces = 4;       // 16-byte words a lane, groups of four rows
  const int base = w * kTile + quarter * 32, sub = lane >> 3, seg = lane & 7, group = p.hq / p.c.hkv;
  const int rows = min(32, U.rows - base);
  auto piece = [&](int i) { return cached_part<false, D>(p, U.owner + i, i == 0 ? 1 : 0); };
  float top = -INFINITY, l = 0.f;
  const int mine = base + min(lane, rows - 1);
#pragma unroll 4
  for (int i = 0; i < U.pieces; ++i) top = fmaxf(top, __ldcg(piece(i) + kChunkRows * D + mine));
  const float neg = top == -INFINITY ? 0.f : -top;
#pragma unroll 4
  for (int i = 0; i < U.pieces; ++i)
    l += fast_exp2(__ldcg(piece(i) + kChunkRows * D + mine) + neg) * __ldcg(piece(i) + kChunkRows * (D + 1) + mine);
  if (lane < rows) {
    const int x = U.row + mine;
    p.lse[(int64_t)(U.h * group + x % group) * p.c.T + U.start + x / group] = (top + log2f(l)) * kLn2;
  }
  const float inv = 1.f / l;
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += 4 * kGroups) {
    float4 o[kGroups][kPer] = {};
#pragma unroll 1
    for (int b = 0; b < U.pieces; b += kPieces) {
      float4 y[kPieces][kGroups][kPer];
      float m[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const float* src = piece(min(b + i, U.pieces - 1));
        m[i] = b + i < U.pieces ? __ldcg(src + kChunkRows * D + mine) : -INFINITY;
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
          const int r = min(r0 + 4 * q + sub, rows - 1);
#pragma unroll
          for (int k = 0; k < kPer; ++k)
            y[i][q][k] = b + i < U.pieces ? __ldcg(reinterpret_cast<const float4*>(src + (size_t)(base + r) * D + k * 32 + 4 * seg))
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const float wm = b + i < U.pieces ? fast_exp2(m[i] + neg) * inv : 0.f;
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
          const float wt = __shfl_sync(0xffffffffu, wm, min(r0 + 4 * q + sub, rows - 1));
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            o[q][k].x = fmaf(wt, y[i][q][k].x, o[q][k].x);
            o[q][k].y = fmaf(wt, y[i][q][k].y, o[q][k].y);
            o[q][k].z = fmaf(wt, y[i][q][k].z, o[q][k].z);
            o[q][k].w = fmaf(wt, y[i][q][k].w, o[q][k].w);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const int r = r0 + 4 * q + sub;
      if (r >= rows) continue;
      const int x = U.row + base + r, h = U.h * group + x % group;
      __nv_bfloat16* dst = p.out + (((int64_t)U.start + x / group) * p.hq + h) * D + 4 * seg;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(o[q][k].x, o[q][k].y), b = __floats2bfloat162_rn(o[q][k].z, o[q][k].w);
        *reinterpret_cast<uint2*>(dst + 32 * k) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      }
    }
    __syncwarp();
  }
}

template <int D, bool E4M3, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    cached_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const CachedParams p, const bool tail) {
  using L = ChunkSmem<D, E4M3>;
  constexpr int kSlots = L::kSlots;
  constexpr bool kSplit = D == 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_full = bars;                  // [2 row tiles], as the next six
  uint64_t* q_empty = bars + 2;
  uint64_t* s_full = bars + 4;
  uint64_t* s_free = bars + 6;              // (split) scores read
  uint64_t* pv_done = bars + 8;             // (split) P read
  uint64_t* o_full = bars + 10;             // the unit's O is whole
  uint64_t* o_free = bars + 12;             // and has been read
  uint64_t* p_full = bars + 14;             // [2 row tiles][2 halves of 64 keys]
  uint64_t* drain = bars + 18;              // [2 issuers]
  uint64_t* unit_full = bars + 20;          // [kUnits]
  uint64_t* unit_done = unit_full + kUnits; // [kUnits] read by every role
  uint64_t* kv_full = unit_done + kUnits;   // [kSlots]
  uint64_t* kv_empty = kv_full + kSlots;    // [kSlots]
  uint64_t* raw_full = kv_empty + kSlots;   // [kRaw]
  uint64_t* raw_empty = raw_full + L::kRaw; // [kRaw]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(raw_empty + L::kRaw);
  int* status = p.c.plan + kCpStatus;
  uint8_t* units = smem + L::kUnit;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_let_next();
  const CachePlanView pv = cache_plan_view(p.c.plan, p.c.T, p.c.N, p.hq, p.c.hkv);
  ShareStart share;
  if (warp == 2) share = pv.first[0][blockIdx.x];      // (beside the header; of use if there is a share)
  const int valid = cached_valid_rows(p);
  if (tail) clear_rows<D>(p, valid, kThreads);
  const Shares sh = cached_shares<false>(pv.hdr);
  if (valid == 0 || (int)blockIdx.x >= sh.n) {
    grid_wait();                            // who comes behind this launch comes behind the one before it too
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 128);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_free[i], 128);
      mbar_init(&p_full[2 * i], 128);
      mbar_init(&p_full[2 * i + 1], 128);
      mbar_init(&drain[i], 1);
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&unit_full[i], 1);
      mbar_init(&unit_done[i], 1 + (kSplit ? 2 : 1) + 8 + (E4M3 ? 4 : 0));
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&kv_full[i], E4M3 ? 4 : 1);
      mbar_init(&kv_empty[i], kSplit ? 2 : 1);      // issuers
    }
    for (int i = 0; i < L::kRaw; ++i) {
      mbar_init(&raw_full[i], 1 + kScaleCopies);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) reinterpret_cast<Piece*>(smem + L::kSplits)[i].tiles = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  constexpr uint32_t kO = 256, kP = 384;

  if (warp < 4) {
    setmaxnreg_dec<kRegCtl>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      const int P = 1 << p.c.page_shift, per = kTile >> p.c.page_shift;       // pages a tile
      constexpr int kRing = E4M3 ? L::kRaw : kSlots;
      constexpr int kRowBytes = E4M3 ? D : 128;                                // of a box
      uint64_t* full = E4M3 ? raw_full : kv_full;
      uint64_t* empty = E4M3 ? raw_empty : kv_empty;
      uint32_t ring = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const Piece U = read_piece(units, unit_full, unit_done, n, true, ok, status);
        if (U.tiles == 0) break;
        auto page_of = [&](int k) {            // lane's page of the k-th tile, or -1
          const int pos = (U.last - k) * kTile + lane * P;
          if (k >= U.tiles || lane >= per || pos >= U.keys || pos + P <= U.lo) return -1;
          const int page = cache_page(p.c, U.seq, pos >> p.c.page_shift);
          return page < 0 ? -1 : page * p.c.hkv + U.h;
        };
        int next = page_of(0);
        for (int k = 0; k < U.tiles && ok; ++k) {
          const int page = next;
          next = page_of(k + 1);
          const int pages = __popc(__ballot_sync(0xffffffffu, page >= 0));
#pragma unroll
          for (int v = 0; v < 2; ++v, ++ring) {
            const uint32_t st = ring % kRing;
            if (ring >= kRing && !(ok = warp_wait(&empty[st], (ring / kRing - 1) & 1, status))) break;
            if (lane == 0) {
              if (pages) mbar_arrive_expect_tx(&full[st], pages * P * (E4M3 ? D : 2 * D));
              else mbar_arrive(&full[st]);
            }
            __syncwarp();
            if (page >= 0) {
              uint8_t* dst = smem + (E4M3 ? L::kCodes + st * L::kRawBytes : L::kKV + st * L::kTileBytes) + lane * P * kRowBytes;
#pragma unroll
              for (int b = 0; b < (E4M3 ? 1 : D / 64); ++b)
                tma_load_3d(dst + b * kTile * 128, v ? &tm_v : &tm_k, &full[st], 128 * b, page, 0);
            }
            if constexpr (E4M3) {              // a lane 16 keys' scales
              const int at_page = __shfl_sync(0xffffffffu, page, lane * 16 / P & 31);
              if (lane < kScaleCopies) {
                if (at_page >= 0)
                  cp_async16(smem + L::kScales + st * kTile + lane * 16,
                             (v ? p.c.v_scales : p.c.k_scales) + ((int64_t)at_page << p.c.page_shift) + (lane * 16 & (P - 1)));
                cp_async_arrive(&full[st]);
              }
            }
            __syncwarp();
          }
        }
      }
      // nothing may land after the CTA has left (reached early only when a wait ran out)
      for (uint32_t x = ring > kRing ? ring - kRing : 0; x < ring; ++x) mbar_wait(&full[x % kRing], (x / kRing) & 1, status);
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 2) {
      // ---------------------------------------------------------- units and their queries
      const int group = p.hq / p.c.hkv;
      uint32_t nq[2] = {0, 0};
      bool ok = true;
      int64_t f = share.from;
      const int64_t f1 = share.to;
      CachedUnit u = share.u;
      for (int n = 0; ok; ++n) {
        if (n >= kUnits && !(ok = warp_wait(&unit_done[n % kUnits], (n / kUnits - 1) & 1, status))) break;
        Piece U{};
        int2 tiles = make_int2(0, 0);
        while (f < f1 && U.tiles == 0) {
          if (f >= u.begin + kChunkExtra + u.tiles) cached_next<false>(pv, u, p.hq, p.c.hkv);
          const int2 piece = cached_piece<false>(u, f, f1);
          const int t0 = piece.x, t1 = piece.y;
          tiles = piece;
          U.tiles = t1 - t0;
          U.last = u.tile + u.tiles - 1 - t0;
          U.h = u.h;
          U.row = u.row;
          U.rows = u.rows;
          U.ntq = u.rows > kTile ? 2 : 1;
          U.start = u.start;
          U.pos0 = u.keys - u.count;
          U.keys = u.keys;
          U.lo = p.left < 0 ? 0 : max(0, U.pos0 + u.row / group - p.left);
          U.seq = u.seq;
          U.slot = U.tiles == u.tiles ? -1 : (t0 == 0 ? 1 : 0);
        }
        if (lane == 0) {
          *reinterpret_cast<Piece*>(units + (n % kUnits) * sizeof(Piece)) = U;
          mbar_arrive(&unit_full[n % kUnits]);
        }
        __syncwarp();
        if (U.tiles == 0) break;
        // (read by the softmax warps from the next unit's start on)
        auto keep_split = [&]() {
          if (lane == 0 && U.slot >= 0) {
            const int2 c = cached_owners<false>(u, sh, tiles.x, tiles.y);
            U.owner = c.x;
            U.pieces = c.y;
            *reinterpret_cast<Piece*>(smem + L::kSplits + U.slot * sizeof(Piece)) = U;
          }
          __syncwarp();
        };
        // Where the heads that share a kv head divide a tile's rows, a box of their tokens is the tile (rows behind
        // the unit's are other sequences', or zeros behind the last token: they have no say and are not stored).
        if (kTile % group == 0) {
          for (int w = 0; w < U.ntq; ++w) {
            if (nq[w] && !(ok = warp_wait(&q_empty[w], (nq[w] - 1) & 1, status))) break;
            ++nq[w];
            if (lane == 0) {
              mbar_arrive_expect_tx(&q_full[w], L::kTileBytes);
#pragma unroll
              for (int b = 0; b < D / 64; ++b)
                tma_load_3d(smem + L::kQ + w * L::kTileBytes + b * kTile * 128, &tm_q, &q_full[w], 64 * b, U.h * group,
                            U.start + (U.row + w * kTile) / group);
            }
            __syncwarp();
          }
          keep_split();
          continue;
        }
        // else two (D = 128) or four rows at a time, 16 bytes a lane, as many as there are (what lies behind them has no say;
        // zeros there and a division a row took 2.5 us more for 70 rows)
        constexpr int kLanes = D / 8, kPer = 32 / kLanes;
        const int c = lane % kLanes, dg = kPer % group;
        int r = lane / kLanes, t = (U.row + r) / group, g = (U.row + r) - t * group;
        const __nv_bfloat16* src = p.q + (((int64_t)U.start + t) * p.hq + U.h * group + g) * D + 8 * c;
        const int step = (kPer / group * p.hq + dg) * D, wrap = (p.hq - group) * D;
        for (int w = 0; w < U.ntq; ++w) {
          if (nq[w] && !(ok = warp_wait(&q_empty[w], (nq[w] - 1) & 1, status))) break;
          ++nq[w];
          uint8_t* tile = smem + L::kQ + w * L::kTileBytes + (c >> 3) * kTile * 128;
#pragma unroll 2
          for (const int end = min(U.rows, (w + 1) * kTile); r < end; r += kPer) {
            cp_async16(tile + swz_offset(r & (kTile - 1), (c & 7) * 16, 128), src);
            src += step;
            g += dg;
            if (g >= group) {
              g -= group;
              src += wrap;
            }
          }
          __syncwarp();
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (w == 0 && U.ntq == 2) continue;
          if (w == 1) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[0]);
          }
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_full[w]);
        }
        keep_split();
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (kTile % group == 0)                       // (reached early only when a wait ran out)
        for (int w = 0; w < 2; ++w)
          if (nq[w]) mbar_wait(&q_full[w], (nq[w] - 1) & 1, status);
    } else if (warp == 1 || kSplit) {
      // ---------------------------------------------------------- MMA issuer of row tiles w0 .. w1 - 1
      const int w0 = kSplit ? warp >> 1 : 0, w1 = kSplit ? w0 + 1 : 2;
      const bool leader = elect_one();
      const uint32_t base16 = (smem_u32(smem) & 0x3FFFFu) >> 4;
      const uint32_t tb = (uint32_t)warp_uniform((int)tbase);
      uint32_t ring = 0, nq0 = 0, nq1 = 0, np0 = 0, np1 = 0, ns0 = 0, ns1 = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const Piece U = read_piece(units, unit_full, unit_done, n, true, ok, status);
        const int nk = warp_uniform(U.tiles), ntq = warp_uniform(U.ntq);
        if (nk == 0) break;
        auto landed = [&](uint32_t x) { return ok = warp_wait(&kv_full[x % kSlots], (x / kSlots) & 1, status); };
        auto release = [&](uint32_t x) {
          if (leader) mma_commit(&kv_empty[x % kSlots]);
        };
        auto scores = [&](int w, int k) {          // S of key tile k.  A (Q): q_full at the unit's first; B (K): kv_full
          const uint32_t x = ring + 2 * k, st = x % kSlots;
          if (k == 0 && !(ok = warp_wait(&q_full[w], (w ? nq1 : nq0) & 1, status))) return;
          uint32_t& ns = w ? ns1 : ns0;
          if (kSplit && ns && !(ok = warp_wait(&s_free[w], (ns - 1) & 1, status))) return;   // the last ones have been read
          ++ns;
          if (!landed(x)) return;
          tc_fence_after();
          const uint32_t kv16 = base16 + st * (L::kTileBytes / 16);
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t off = (s / 4) * kTile * 128 + (s % 4) * 32;
            if (leader)
              mma_bf16(tb + w * 128, sdesc_at(base16, L::kQ + w * L::kTileBytes + off, 16, 1024, kSwizzle128B),
                       sdesc_at(kv16, L::kKV + off, 16, 1024, kSwizzle128B), idesc_bf16(128, 128, 0, 0), s > 0);
          }
          if (leader) {
            mma_commit(&s_full[w]);
            if (k == nk - 1) mma_commit(&q_empty[w]);
          }
        };
        // O += P V, half of the keys at a time as they are handed in.  A (P in TMEM): p_full; B (V): kv_full
        auto values = [&](int w, int k) {
          const uint32_t x = ring + 2 * k + 1, st = x % kSlots;
          if (!landed(x)) return;
          const uint32_t nq = w ? nq1 : nq0;
          if (k == 0 && nq && !(ok = warp_wait(&o_free[w], (nq - 1) & 1, status))) return;
          const uint32_t par = (w ? np1++ : np0++) & 1, kv16 = base16 + st * (L::kTileBytes / 16);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!(ok = warp_wait(&p_full[2 * w + half], par, status))) return;
            tc_fence_after();
#pragma unroll
            for (int s = 4 * half; s < 4 * half + 4; ++s)
              if (leader)
                mma_bf16_ta(tb + kO + w * D, tb + (kSplit ? kP + 64 * w : 128 * w) + s * 8,
                            sdesc_at(kv16, L::kKV + s * 2048, kTile * 128, 1024, kSwizzle128B), idesc_bf16(128, D, 0, 1),
                            (k != 0 || s > 0));
          }
          if (leader) {
            if (kSplit) mma_commit(&pv_done[w]);
            if (k == nk - 1) mma_commit(&o_full[w]);
          }
        };
        for (int w = w0; w < w1 && ok; ++w) {
          if (w < ntq) scores(w, 0);
          else if (kSplit) landed(ring);           // (a tile that nobody else of this issuer has waited for)
        }
        if (ok) release(ring);
        for (int k = 0; k < nk && ok; ++k) {
          for (int w = w0; w < w1 && ok; ++w) {
            const bool next = k + 1 < nk && w < ntq;
            if (kSplit && next) scores(w, k + 1);
            if (ok && w < ntq) values(w, k);
            else if (kSplit && ok) landed(ring + 2 * k + 1);
            if (kSplit && ok && !next && k + 1 < nk) landed(ring + 2 * k + 2);
            if (!kSplit && next && ok) scores(w, k + 1);     // over P, right behind its product
          }
          if (!ok) break;
          release(ring + 2 * k + 1);
          if (k + 1 < nk) release(ring + 2 * k + 2);
        }
        ++nq0;
        if (ntq > 1) ++nq1;
        ring += 2 * nk;
      }
      // every MMA has finished before tensor memory is freed
      if (leader) {
        mma_commit(&drain[w0]);
        mbar_wait(&drain[w0], 0, status);
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<kRegSoftmax>();
    const int w = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = tbase + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_addr = lane_base + w * 128, o_addr = lane_base + kO + w * D;
    const uint32_t p_addr = kSplit ? lane_base + kP + 64 * w : s_addr;
    const float scale2 = p.scale2;
    const int group = p.hq / p.c.hkv;
    const bool al32 = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;       // (whole sectors where they can be)
    // The piece that the share begins with is counted some key tiles into the next unit: right where it ends, the wait for
    // its stores kept that unit waiting (3 us).  count_at: when ns will say so, 0: no such piece so far.
    uint32_t count_at = 0;
    auto count_piece = [&](int slot) {       // (what it says is kept in shared memory until the share's end)
      if (lane == 0) {
        Piece& U = reinterpret_cast<Piece*>(smem + L::kSplits)[slot];
        U.ended[4 * w + quarter] = cached_last(pv.done + kStepCtas + 8 * U.owner + 4 * w + quarter, U.pieces);
      }
      __syncwarp();
    };
    uint32_t ring = 0, ns = 0, nu = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const Piece U = read_piece(units, unit_full, unit_done, n, true, ok, status);
      if (U.tiles == 0) break;
      const int nk = U.tiles;
      if (w >= U.ntq) {
        ring += 2 * nk;
        continue;
      }
      const int rr = w * kTile + r;
      const bool row_in = rr < U.rows;     // rows behind the unit's take no part in the warp's choices
      const int x = U.row + min(rr, U.rows - 1);
      const int pos = U.pos0 + x / group;
      const int lo = p.left < 0 ? 0 : max(0, pos - p.left);
      // tiles that every row of the row tile sees whole
      const int full_hi = (U.pos0 + (U.row + w * kTile) / group + 1) / kTile - 1;
      const int full_lo = p.left < 0 ? 0
          : max(0, U.pos0 + (U.row + min(w * kTile + kTile, U.rows) - 1) / group - p.left + kTile - 1) / kTile;
      float m = -INFINITY;
      float2 la = make_float2(0.f, 0.f), lb = la;
      bool first = true;
      for (int k = 0; k < nk; ++k) {
        const int u = U.last - k;
        const bool seen = u >= full_lo && u <= full_hi;
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[w], ns & 1, status));
        if (!ok) break;
        tc_fence_after();
        // At D = 64 without a cap a row's products stay in registers, all code unrolled: the scores' place is free for the
        // next ones early (1.31 instead of 1.50 us a key tile).  Else they are read again 32 columns at a time, in rolled loops:
        // with a cap four forms of 128 columns were some 100 KB of instructions, whose first pass took 25 us a call, and
        // spilled; at D = 128 P lies over the scores anyway (E4M3 419 instead of 427 us for a chunk of 2048 behind 14336,
        // bf16 376 and 375).
        constexpr bool kRolled = CAP || D == 128;
        uint32_t v[kRolled ? 1 : 4][32];
        float mx;
        // form 0: v f + n; 1, 2, 3: capped by 3 coefficients, by 5 or by tanh itself inside the exponent.  A capped row's
        // reference is its largest magnitude where that is little, else its capped maximum.
        int form = 0;
        if constexpr (kRolled) {
          bool plain = !seen;
          if (seen) {
            mx = columns_max<CAP>(s_addr);
            if (CAP) plain = __any_sync(0xffffffffu, row_in && !(mx * scale2 < 0x1p27f));      // (beyond, x and m are shrunk below)
          }
          if (plain) {
            // (most of a masked tile's columns are seen by all of a warp's rows)
            mx = -INFINITY;
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
              const uint32_t see = seen ? ~0u : column_mask(lo - u * kTile, pos - u * kTile, -1, 32 * g);
              const bool all = __all_sync(0xffffffffu, see == ~0u);
              float cm;
              tmem_ld32_max(s_addr + 32 * g, v[0], cm);
              tmem_ld_wait();
              if (CAP) {
                if (!all) hide(v[0], see, 0u);
                cap_columns(v[0], p.capf, row_in);
              }
              if (!all) hide(v[0], see, kMinusInf);
              if (CAP || !all) {
                float c2[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 32; j += 4)
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    c2[i] = fmax3(c2[i], __uint_as_float(v[0][j + 2 * i]), __uint_as_float(v[0][j + 2 * i + 1]));
                cm = fmaxf(c2[0], c2[1]);
                tmem_st32(s_addr + 32 * g, v[0]);
              }
              mx = fmaxf(mx, cm);
            }
            tmem_st_wait();
          } else if (CAP) {
            form = !__any_sync(0xffffffffu, row_in && !(mx <= p.capf.t3)) ? 1
                   : !__any_sync(0xffffffffu, row_in && !(mx <= p.capf.t5)) ? 2 : 3;
            if (__any_sync(0xffffffffu, row_in && !(mx * scale2 <= kLoose * 0.5f)))
              mx = p.capf.inv * tanh_any(columns_max<false>(s_addr) * p.capf.zscale);
          }
        } else {
          float cm[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) tmem_ld32_max(s_addr + 32 * g, v[g], cm[g]);
          tmem_ld_wait();
          if (kSplit) {
            tc_fence_before();
            mbar_arrive(&s_free[w]);
          }
          if (!seen) {
#pragma unroll
            for (int g = 0; g < 4; ++g) hide(v[g], column_mask(lo - u * kTile, pos - u * kTile, -1, 32 * g), kMinusInf);
#pragma unroll
            for (int g = 0; g < 4; ++g) cm[g] = -INFINITY;
#pragma unroll
            for (int j = 0; j < 32; j += 2)
#pragma unroll
              for (int g = 0; g < 4; ++g) cm[g] = fmax3(cm[g], __uint_as_float(v[g][j]), __uint_as_float(v[g][j + 1]));
          }
          mx = fmaxf(fmax3(cm[0], cm[1], cm[2]), cm[3]);
        }
        mx *= scale2;
        if (first) {
          m = mx;
        } else if (__any_sync(0xffffffffu, row_in && mx > m + kRescaleAbove)) {
          const float m_new = fmaxf(m, mx);
          const float alpha = m_new == m ? 1.f : fast_exp2(m - m_new);      // 0 where nothing was visible yet
          la = fmul2(la, make_float2(alpha, alpha));
          lb = fmul2(lb, make_float2(alpha, alpha));
          m = m_new;
          if (kSplit) {                // the last product has to be in
            ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[w], (ns - 1) & 1, status));
            if (!ok) break;
            tc_fence_after();
          }
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(o_addr + 32 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tmem_st32(o_addr + 32 * c, o);
          }
          tmem_st_wait();
        }
        if constexpr (!E4M3) {
          if ((u + 1) * kTile > U.keys || u * kTile < U.lo) {      // weight 0 does not silence an infinity
            const uint32_t y = ring + 2 * k + 1, st = y % kSlots;
            ok = __all_sync(0xffffffffu, mbar_wait(&kv_full[st], (y / kSlots) & 1, status));
            if (!ok) break;
            if (u * kTile + r >= U.keys || u * kTile + r < U.lo) clear_row<D>(smem + L::kKV + st * L::kTileBytes, r);
            fence_proxy_async_smem();
            __syncwarp();              // P is stored by the whole warp
          }
        }
        const float shrink = shrink_for(m);
        const float neg = (m == -INFINITY ? 0.f : -m) * shrink, fs = fmaxf(scale2 * shrink, 0x1p-126f);   // (0 * -inf)
        // P in two halves of 64 keys: the first one's product starts while the second is computed
        auto weights = [&](auto FORM, const uint32_t (&y)[32], uint32_t* pk) {
          constexpr int kForm = decltype(FORM)::value;
          const float2 f2 = make_float2(fs, fs), n2 = make_float2(neg, neg);
          const CapForm& F = p.capf;
          const float z2 = F.zscale * (2.f * kLog2e), top = F.inv * fs;
          auto capped = [&](float2 x) {           // x (scale2 + scale2 t(x^2)) + n
            const float2 q = fmul2(x, x);
            float2 t;
            if constexpr (kForm == 1) {
              t = ffma2(q, F.e3[3], F.e3[2]);
              t = ffma2(q, t, F.e3[1]);
              t = ffma2(q, t, F.e3[0]);
            } else {
              t = ffma2(q, F.e5[5], F.e5[4]);
              t = ffma2(q, t, F.e5[3]);
              t = ffma2(q, t, F.e5[2]);
              t = ffma2(q, t, F.e5[1]);
              t = ffma2(q, t, F.e5[0]);
            }
            return ffma2(x, t, n2);
          };
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            float2 e0 = pair_of(y, j), e1 = pair_of(y, j + 2);
            if constexpr (kForm == 3) {
              tanh4(e0, e1, z2, top + neg, -2.f * top);
            } else if constexpr (kForm == 0) {
              e0 = ffma2(e0, f2, n2);
              e1 = ffma2(e1, f2, n2);
            } else {
              e0 = capped(e0);
              e1 = capped(e1);
            }
            e0 = make_float2(fast_exp2(e0.x), fast_exp2(e0.y));
            e1 = make_float2(fast_exp2(e1.x), fast_exp2(e1.y));
            la = fadd2(la, e0);
            lb = fadd2(lb, e1);
            const __nv_bfloat162 b0 = __floats2bfloat162_rn(e0.x, e0.y), b1 = __floats2bfloat162_rn(e1.x, e1.y);
            pk[j / 2] = *reinterpret_cast<const uint32_t*>(&b0);
            pk[j / 2 + 1] = *reinterpret_cast<const uint32_t*>(&b1);
          }
        };
        auto last_p_read = [&]() {               // (split)
          if (!kSplit || !ns) return;
          ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[w], (ns - 1) & 1, status));
          tc_fence_after();
        };
        auto hand_in = [&](int half) {
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full[2 * w + half]);
        };
        if constexpr (kRolled) {
          last_p_read();
          if (!ok) break;
          auto columns = [&](auto FORM) {
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {       // (over the scores: P's 16 columns end before the next 32 begin)
              tmem_ld32(s_addr + 32 * g, v[0]);
              tmem_ld_wait();
              if (kSplit && g == 3) {
                tc_fence_before();
                mbar_arrive(&s_free[w]);
              }
              uint32_t pk[16];
              weights(FORM, v[0], pk);
              tmem_st16(p_addr + 16 * g, pk);
              if (g & 1) hand_in(g >> 1);
            }
          };
          if (CAP && form == 1) columns(std::integral_constant<int, 1>{});
          else if (CAP && form == 2) columns(std::integral_constant<int, 2>{});
          else if (CAP && form == 3) columns(std::integral_constant<int, 3>{});
          else columns(std::integral_constant<int, 0>{});
        } else {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
            weights(std::integral_constant<int, 0>{}, v[2 * half], pk);
            weights(std::integral_constant<int, 0>{}, v[2 * half + 1], pk + 16);
            if (half == 0) last_p_read();
            if (!ok) break;
            tmem_st32(p_addr + 32 * half, pk);
            hand_in(half);
          }
        }
        if (!ok) break;
        if (++ns == count_at) count_piece(0);
        first = false;
      }
      ring += 2 * nk;
      if (!ok) break;
      // O: of a whole unit divided and rounded, of a piece as it is
      const float l = (la.x + la.y) + (lb.x + lb.y);
      ok = __all_sync(0xffffffffu, mbar_wait(&o_full[w], nu & 1, status));
      if (!ok) break;
      ++nu;
      tc_fence_after();
      const int64_t tok = (int64_t)U.start + x / group;
      const int h = U.h * group + x % group;
      float* part = cached_part<false, D>(p, blockIdx.x, max(U.slot, 0));
      const float inv = 1.f / l;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        __syncwarp();              // (some rows alone have stored the last columns)
        tmem_ld32(o_addr + 32 * c, o);
        tmem_ld_wait();
        if (c == D / 32 - 1) {
          tc_fence_before();
          mbar_arrive(&o_free[w]);
        }
        if (!row_in) continue;
        if (U.slot < 0) {
          __nv_bfloat16* dst = p.out + (tok * p.hq + h) * D + 32 * c;
          uint32_t y[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
            y[j] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          if (al32) {
            st_global_v8(dst, y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]);
            st_global_v8(dst + 16, y[8], y[9], y[10], y[11], y[12], y[13], y[14], y[15]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(dst + 8 * j) = make_uint4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
          }
        } else {
          float* dst = part + (size_t)rr * D + 32 * c;
#pragma unroll
          for (int j = 0; j < 32; j += 8)
            st_global_v8(dst + j, o[j], o[j + 1], o[j + 2], o[j + 3], o[j + 4], o[j + 5], o[j + 6], o[j + 7]);
        }
      }
      __syncwarp();
      if (row_in) {
        if (U.slot < 0) {
          p.lse[(int64_t)h * p.c.T + tok] = (m + log2f(l)) * kLn2;
        } else {
          part[(size_t)kChunkRows * D + rr] = m;
          part[(size_t)kChunkRows * (D + 1) + rr] = l;
        }
      }
      if (U.slot == 0 && U.rows > w * kTile + quarter * 32) count_at = ns + 3;
    }
    // Split units: a warp's rows stay a warp's, and the last of their pieces to be finished joins them, at its share's end.
    if (ok) {
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const Piece& U = reinterpret_cast<const Piece*>(smem + L::kSplits)[i];
        if (U.tiles == 0 || U.rows <= w * kTile + quarter * 32) continue;
        if (i == 1 || ns < count_at) count_piece(i);
        if (U.ended[4 * w + quarter]) join_rows<D>(p, U, w, quarter, lane);
      }
    }
  } else {
    // ------------------------------------------------------------ unpack
    setmaxnreg_dec<kRegUnpack>();
    if constexpr (E4M3) {
      const int r = (warp & 3) * 32 + lane;
      uint32_t ring = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const Piece U = read_piece(units, unit_full, unit_done, n, true, ok, status);
        if (U.tiles == 0) break;
        for (int k = 0; k < 2 * U.tiles && ok; ++k, ++ring) {
          const uint32_t st = ring % L::kRaw, to = ring % kSlots;
          const int key = (U.last - (k >> 1)) * kTile + r;
          if (!(ok = warp_wait(&raw_full[st], (ring / L::kRaw) & 1, status))) break;
          if (ring >= kSlots && !(ok = warp_wait(&kv_empty[to], (ring / kSlots - 1) & 1, status))) break;
          const uint32_t raw = smem_u32(smem + L::kCodes + st * L::kRawBytes), tile = smem_u32(smem + L::kKV + to * L::kTileBytes);
          const uint32_t b = smem[L::kScales + st * kTile + r];
          if (key >= U.keys || key < U.lo) clear_row<D>(smem + L::kKV + to * L::kTileBytes, r);
          else if (b <= 134) unpack_row<D, false>(raw, tile, r, b);
          else unpack_row<D, true>(raw, tile, r, b);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&raw_empty[st]);
            mbar_arrive(&kv_full[to]);
          }
        }
      }
    }
  }
  grid_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, bool E4M3, bool CAP>
cudaError_t launch(const CachedParams& p, bool tail, cudaStream_t stream) {
  using L = ChunkSmem<D, E4M3>;
  CUtensorMap tq, tk, tv;
  const uint64_t P = (uint64_t)1 << p.c.page_shift, pages = (uint64_t)p.c.num_pages * p.c.hkv, row = E4M3 ? D : 2 * D;
  const int group = p.hq / p.c.hkv, heads = kTile % group == 0 ? group : 1;       // (1: the map is not used)
  const uint32_t box = row < 128 ? (uint32_t)row : 128;
  if (!make_tmap_bf16_3d(&tq, p.q, D, p.hq, p.c.T, D * 2, (uint64_t)p.hq * D * 2, 64, kTile / heads, heads) ||
      !make_tmap_u8_3d(&tk, p.c.k, row, pages, P, P * row, row, box, (uint32_t)P) ||
      !make_tmap_u8_3d(&tv, p.c.v, row, pages, P, P * row, row, box, (uint32_t)P))
    return cudaErrorInvalidValue;
  int regs = 0;
  static_assert(L::kAlloc <= 232448, "shared memory of one CTA");
  cudaError_t e = prepare_kernel<cached_chunk_kernel<D, E4M3, CAP>>(L::kAlloc, &regs);
  if (e != cudaSuccess) return e;
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;    // the register split relies on it
  // starts while the steps still run: it reads nothing of theirs
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kChunkCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = tail ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, cached_chunk_kernel<D, E4M3, CAP>, tq, tk, tv, p, tail);
}

template <int D>
cudaError_t launch_d(bool e4m3, CachedParams p, bool tail, cudaStream_t s) {
  // (products of four-bit keys lose nothing that shows as the tensor core adds them up: with the factor LSE came out
  // 4e-6 too large on 2048 behind 14336, scores of some tens)
  const double gain = e4m3 ? 1.0 : mma_gain(D);
  p.scale2 = (float)(p.scale * gain * 1.4426950408889634);
  p.capf = cap_form(p.scale * gain, (double)p.cap);
  if (e4m3) return p.cap > 0.f ? launch<D, true, true>(p, tail, s) : launch<D, true, false>(p, tail, s);
  return p.cap > 0.f ? launch<D, false, true>(p, tail, s) : launch<D, false, false>(p, tail, s);
}

}  // namespace

// tail: no steps are launched in front, so the rows behind the last sequence are cleared here.
cudaError_t launch_cached_chunk(int D, bool e4m3, const CachedParams& p, bool tail, cudaStream_t s) {
  return D == 128 ? launch_d<128>(e4m3, p, tail, s) : launch_d<64>(e4m3, p, tail, s);
}

}  // namespace flamia
