// Attention over the paged cache for steps: a sequence's few new tokens (up to 16 rows of a kv head),
// and the joining of pieces.
//
//   x = scale log2 e q.k (capped), m = running maximum, l += 2^(x - m), O += 2^(x - m) v
//
// Bound by memory: every key and value is read once, for 4 d flops a row.  A CTA streams its share of
// the key tiles (64 keys, K and V) through shared memory: one warp issues TMA copies page by page,
// four compute warps take 16 keys each with a softmax of their own and meet only where a unit ends.
// Two CTAs an SM, so that one streams while the other meets, with some 128 KB in flight between them.
//
// The products run as 16 x 8 x 16 MMAs from registers: 16 rows are one tile, and what is to be fast
// here is the stream, not the products (tcgen05 would want 64 rows at least, and the codes unpacked into
// shared memory).  Which of the head dimensions a lane's operand words stand for is free as long
// as both operands agree, so a lane takes whole 16-byte words of a key's row, and for V of one head-dim
// run in four keys' rows, whose bytes are paired by permutes; with the 128-byte swizzle of the copies
// both are free of bank conflicts.
//
// E4M3: a code is exact in fp16, two are converted at a time, and the products run in fp16.  Queries are
// scaled by a power of two a row, its largest value to [2^14, 2^15).  The key's scale multiplies the
// score.  The value's scale 2^e enters the weight: w = 2^(x - m + e - M + 13) with a running maximum M of x - m + e
// of its own (against m, so that scores of any size leave the exponents their digits): the largest w is in
// [2^13, 2^15] whatever the scales are, and what falls below fp16's range is 2^-38 of it.  Rounding w to fp16 costs 2^-12 of it at most.
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
constexpr int kUnits = 2;         // described and their queries fetched ahead

// A unit's piece as the compute warps need it.
struct alignas(16) StepPiece {
  int t0, t1, tiles, tile;        // key tiles [t0, t1) of the unit's; its first tile's number in the sequence.  t1 0: no more
  int h, rows, start, pos0;       // first token of the sequence, and its position
  int keys, lo, pad[6];
};
static_assert(sizeof(StepPiece) == 64, "");

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
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

template <int N>
__device__ __forceinline__ void scale_rows(float (&o)[N][4], int r, float f) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    o[n][2 * r] *= f;
    o[n][2 * r + 1] *= f;
  }
}

template <int D, bool E4M3>
struct StepSmem {
  static constexpr int kRowBytes = E4M3 ? D : 2 * D;
  static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kBoxes = kRowBytes / kBoxBytes;
  static constexpr int kTileBytes = kStepTile * kRowBytes;                    // of K, or of V
  [[maybe_unused]] static constexpr int kScales = 2 * kTileBytes;             // in a stage: K's and V's scale bytes
  static constexpr int kStage = 2 * kTileBytes + (E4M3 ? 1024 : 0);           // (stages stay on 1024 bytes)
  static constexpr int kStages = E4M3 ? (D == 128 ? 4 : 6) : (D == 128 ? 2 : 4);
  static constexpr int kRed = kStages * kStage;                               // [4 warps][16 rows][D] floats
  static constexpr int kStat = kRed + kComputeWarps * kStepRows * D * 4;      // [4 warps][m, l][16]
  static constexpr int kQ = kStat + kComputeWarps * 2 * kStepRows * 4;        // [2 units in turn][16 rows] queries
  static constexpr int kUnit = kQ + kUnits * kStepRows * D * 2;
  static constexpr int kBar = kUnit + kUnits * 64;
  static constexpr int kBytes = kBar + (2 * kStages + 2 * kUnits) * 8;
  static constexpr int kAlloc = kBytes + 1024;
};
static_assert(2 * (StepSmem<128, false>::kAlloc + 1024) <= 233472 && 2 * (StepSmem<128, true>::kAlloc + 1024) <= 233472,
              "two CTAs an SM");

// O = 0, LSE = +inf behind the last sequence.
__device__ __forceinline__ void clear_rows(const CachedParams& p, int D, int valid, int thread, int threads) {
  const int64_t rows = (int64_t)(p.c.T - valid) * p.hq;
  for (int64_t i = (int64_t)blockIdx.x * threads + thread; i < rows; i += (int64_t)gridDim.x * threads) {
    const int64_t row = valid + i / p.hq;
    const int h = (int)(i % p.hq);
    uint4* dst = reinterpret_cast<uint4*>(p.out + (row * p.hq + h) * D);
    for (int j = 0; j < D / 8; ++j) dst[j] = make_uint4(0, 0, 0, 0);
    p.lse[(int64_t)h * p.c.T + row] = INFINITY;
  }
}

template <int D, bool E4M3, bool CAP>
__global__ void __launch_bounds__(kThreads, 2)
    cached_step_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const CachedParams p) {
  using L = StepSmem<D, E4M3>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty = full + L::kStages;
  uint64_t* unit_full = empty + L::kStages;
  uint64_t* unit_done = unit_full + kUnits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_let_next();
  const int valid = cached_valid_rows(p);
  clear_rows(p, D, valid, threadIdx.x, kThreads);
  if (valid == 0) return;
  const CachePlanView pv = cache_plan_view(p.c.plan, p.c.T, p.c.N, p.hq, p.c.hkv);
  const Shares sh = cached_shares<true>(p, pv);
  if ((int)blockIdx.x >= sh.n) return;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kComputeWarps);
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&unit_full[i], 33);            // the producer's lanes as their copies land, and the description
      mbar_init(&unit_done[i], kComputeWarps);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  __syncthreads();
  int* status = p.c.plan + kCpStatus;
  const int group = p.hq / p.c.hkv;
  bool ok = true;
  uint32_t ring = 0;

  if (warp == kComputeWarps) {
    // ------------------------------------------------------------ producer
    const int64_t f1 = sh.begin(blockIdx.x + 1);
    const int P = 1 << p.c.page_shift, rows = min(P, kStepTile), per = kStepTile / rows;      // pages a tile
    const uint32_t page_bytes = 2 * rows * (L::kRowBytes + (E4M3 ? 1 : 0));
    CachedUnit u{};
    int64_t f = sh.begin(blockIdx.x);
    for (int n = 0; ok;) {
      int2 piece = make_int2(0, 0);
      if (f < f1) {
        const int64_t next = u.begin + kStepExtra + u.tiles;
        if (u.tiles && u.h + 1 < p.c.hkv) {    // the next head of the same sequence
          ++u.h;
          u.begin = next;
        } else {
          u = cached_unit<true>(p, pv, f);
        }
        piece = cached_piece<true>(u, f, f1);
        if (piece.y == 0) continue;            // (only the share's end)
      }
      if (n >= kUnits && !(ok = warp_wait(&unit_done[n % kUnits], (n / kUnits - 1) & 1, status))) break;
      const int t0 = piece.x, t1 = piece.y;
      if (lane == 0) {
        StepPiece x{};
        x.t0 = t0;
        x.t1 = t1;
        x.tiles = u.tiles;
        x.tile = u.tile;
        x.h = u.h;
        x.rows = u.rows;
        x.start = u.start;
        x.pos0 = u.keys - u.count;
        x.keys = u.keys;
        x.lo = u.lo;
        *reinterpret_cast<StepPiece*>(smem + L::kUnit + (n % kUnits) * sizeof(StepPiece)) = x;
      }
      // queries: 16 bytes a lane and copy, rows behind the unit's are zeros
      constexpr int kLanes = D / 8, kPer = 32 / kLanes;
#pragma unroll
      for (int i = 0; i < kStepRows / kPer; ++i) {
        const int r = i * kPer + lane / kLanes, c = lane % kLanes;
        const bool in = t1 > 0 && r < u.rows;
        const int2 at = in ? cached_row(p, u, r) : make_int2(0, 0);
        const __nv_bfloat16* src = p.q + ((int64_t)at.x * p.hq + at.y) * D + 8 * c;
        const uint32_t dst = smem_u32(smem + L::kQ + ((n % kUnits) * kStepRows + r) * D * 2 + 16 * c);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&unit_full[n % kUnits])) : "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&unit_full[n % kUnits]);
      ++n;
      if (t1 == 0) break;
      // page (or half page) i of the unit's tiles: where its keys are, or -1
      const int first = (u.tile + t0) * per, end = (u.tile + t1) * per;
      auto page_of = [&](int i) {
        const int pos = i * rows;
        if (i >= end || pos >= u.keys || pos + rows <= u.lo) return -1;
        const int page = cache_page(p.c, u.seq, pos >> p.c.page_shift);
        return page < 0 ? -1 : page * p.c.hkv + u.h;
      };
      int batch = first, now = page_of(first + lane), next = page_of(first + 32 + lane);
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
          if constexpr (E4M3) {
            const int64_t at = ((int64_t)page << p.c.page_shift) + slot;
            uint8_t* sc = smem + st * L::kStage + L::kScales + lane * rows;
            bulk_load(sc, p.c.k_scales + at, rows, &full[st]);
            bulk_load(sc + kStepTile, p.c.v_scales + at, rows, &full[st]);
          }
        }
        __syncwarp();
      }
    }
    // nothing may land after the CTA has left (reached early only when a wait ran out)
    for (uint32_t x = ring > L::kStages ? ring - L::kStages : 0; x < ring; ++x)
      mbar_wait(&full[x % L::kStages], (x / L::kStages) & 1, status);
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  // -------------------------------------------------------------- compute
  constexpr int kSteps = D / 16, kOut = D / 8;
  constexpr int kWords = L::kRowBytes / 8 / 4;       // a lane's words of a value row
  const int g = lane >> 2, q = lane & 3;
  float* red = reinterpret_cast<float*>(smem + L::kRed);
  float* stat = reinterpret_cast<float*>(smem + L::kStat);
  // this lane's places in a stage: words of key row g (8 rows on: 8 rows' bytes on) and of value rows 2 q and 2 q + 1
  constexpr int kLoads = E4M3 ? D / 64 : 2;
  int at_k[kLoads], at_v[2];
#pragma unroll
  for (int j = 0; j < kLoads; ++j)
    at_k[j] = 16 * warp * L::kBoxBytes + (E4M3 ? swz_offset(g, (D / 4) * q + 16 * j, L::kBoxBytes) : swz_offset(g, (2 * q + j) * 16, 128));
#pragma unroll
  for (int k = 0; k < 2; ++k)
    at_v[k] = L::kTileBytes + 16 * warp * L::kBoxBytes + swz_offset(2 * q + k, kWords >= 4 ? 16 * g : 8 * g, L::kBoxBytes);
  for (int n = 0; ok; ++n) {
    // (the warps meet here too: the last unit's sums have been read, and where a wait ran out all of them leave)
    ok = named_bar_and(1, kComputeWarps * 32, warp_wait(&unit_full[n % kUnits], (n / kUnits) & 1, status));
    if (!ok) break;
    const StepPiece u = *reinterpret_cast<const StepPiece*>(smem + L::kUnit + (n % kUnits) * sizeof(StepPiece));
    if (u.t1 == 0) break;
    // queries: rows g and g + 8, four head dimensions a step of 16
    uint32_t a[kSteps][4];
    float rowf[2];
    int pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      pos[i] = u.pos0 + (r < u.rows ? r : 0) / group;
      const uint8_t* src = smem + L::kQ + ((n % kUnits) * kStepRows + r) * D * 2;
      float x[kSteps][4];
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int d0 = E4M3 ? (D / 4) * q + 4 * s : (s >> 2) * 64 + (2 * q + ((s >> 1) & 1)) * 8 + (s & 1) * 4;
        const uint2 w = *reinterpret_cast<const uint2*>(src + d0 * 2);
        if constexpr (E4M3) {
          x[s][0] = __uint_as_float(w.x << 16);
          x[s][1] = __uint_as_float(w.x & 0xffff0000u);
          x[s][2] = __uint_as_float(w.y << 16);
          x[s][3] = __uint_as_float(w.y & 0xffff0000u);
          top = fmaxf(fmax3(top, fabsf(x[s][0]), fabsf(x[s][1])), fmaxf(fabsf(x[s][2]), fabsf(x[s][3])));
        } else {
          a[s][i] = w.x;
          a[s][2 + i] = w.y;
        }
      }
      rowf[i] = CAP ? 1.f : p.scale2;
      if constexpr (E4M3) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int shift = min(14 + 127 - (int)(__float_as_uint(top) >> 23), 126);     // (a row of zeros: any)
        const float up = exp2i(shift);
        rowf[i] *= exp2i(-shift);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          a[s][i] = pack2<true>(x[s][0] * up, x[s][1] * up);
          a[s][2 + i] = pack2<true>(x[s][2] * up, x[s][3] * up);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&unit_done[n % kUnits]);
    float o[kOut][4] = {};
    float m[2] = {-INFINITY, -INFINITY}, M[2] = {-INFINITY, -INFINITY};
    float neg[2] = {0.f, 0.f}, Neg[2] = {0.f, 0.f};      // -m and 13 - M, 0 while they are infinite
    float2 l[2] = {};
    const int all_see = u.pos0 + 1 - kStepTile;          // tiles up to this key hide none behind a row's position
    const int window = p.left < 0 ? -1 : u.pos0 + (u.rows - 1) / group - p.left;    // tiles from this key on none before one
    for (int t = u.t0; t < u.t1; ++t, ++ring) {
      const uint32_t st = ring % L::kStages;
      if (ok) ok = warp_wait(&full[st], (ring / L::kStages) & 1, status);
      if (!ok) continue;
      const uint8_t* stage = smem + st * L::kStage;
      const int c0 = (u.tile + t) * kStepTile;
      // scores: keys c0 + 16 warp + 8 i + 2 q + {0, 1}
      float s[2][4] = {};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (E4M3) {
          uint4 w[D / 64];
#pragma unroll
          for (int j = 0; j < D / 64; ++j) w[j] = *reinterpret_cast<const uint4*>(stage + at_k[j] + 8 * i * L::kBoxBytes);
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            const uint32_t x = (&w[j / 4].x)[j % 4];
            mma16816<true>(s[i], a[j], codes_f16(x), codes_f16_hi(x));
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint4 w = *reinterpret_cast<const uint4*>(stage + at_k[j & 1] + (j >> 1) * kStepTile * 128 + 8 * i * 128);
            mma16816<false>(s[i], a[2 * j], w.x, w.y);
            mma16816<false>(s[i], a[2 * j + 1], w.z, w.w);
          }
        }
      }
      // values of the same keys, in flight while the softmax runs
      uint32_t v[4][kWords];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t* src = stage + at_v[k & 1] + 8 * (k >> 1) * L::kBoxBytes;
        if constexpr (kWords >= 4) {
#pragma unroll
          for (int j = 0; j < kWords / 4; ++j) {
            const uint4 w = *reinterpret_cast<const uint4*>(src + j * kStepTile * 128);
            v[k][4 * j] = w.x;
            v[k][4 * j + 1] = w.y;
            v[k][4 * j + 2] = w.z;
            v[k][4 * j + 3] = w.w;
          }
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(src);
          v[k][0] = w.x;
          v[k][1] = w.y;
        }
      }
      float2 x[2][2];        // [8 keys][row]
      float2 e[2];           // exponents of the values' scales
      if constexpr (E4M3) {
        const uint8_t* sc = stage + L::kScales + 16 * warp + 2 * q;
        float2 k[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t ks = *reinterpret_cast<const uint16_t*>(sc + 8 * i);
          const uint32_t vs = *reinterpret_cast<const uint16_t*>(sc + kStepTile + 8 * i);
          // 2^(byte - 127), but 0 for byte 0: a score that counts is beyond 2^-90
          k[i] = make_float2(__uint_as_float(ks << 23 & 0x7f800000u), __uint_as_float(ks << 15 & 0x7f800000u));
          // 2^23 + byte, by its bits
          e[i] = fadd2(make_float2(__uint_as_float(__byte_perm(vs, 0x4b000000u, 0x7650)),
                                   __uint_as_float(__byte_perm(vs, 0x4b000000u, 0x7651))),
                       make_float2(-8388735.f, -8388735.f));
        }
        if (c0 + kStepTile > u.keys || c0 < u.lo) {       // what is no key of the sequence may be anything
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int j = c0 + 16 * warp + 8 * i + 2 * q;
            if (j >= u.keys || j < u.lo) k[i].x = 1.f, e[i].x = 0.f;
            if (j + 1 >= u.keys || j + 1 < u.lo) k[i].y = 1.f, e[i].y = 0.f;
          }
        }
        // byte 255: infinite, and 128
        if (__any_sync(0xffffffffu, fmaxf(fmax3(k[0].x, k[0].y, k[1].x), k[1].y) == INFINITY ||
                                        fmaxf(fmax3(e[0].x, e[0].y, e[1].x), e[1].y) > 127.5f)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (k[i].x == INFINITY) k[i].x = NAN;
            if (k[i].y == INFINITY) k[i].y = NAN;
            if (e[i].x > 127.5f) e[i].x = NAN;
            if (e[i].y > 127.5f) e[i].y = NAN;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            x[i][r] = fmul2(fmul2(make_float2(s[i][2 * r], s[i][2 * r + 1]), make_float2(rowf[r], rowf[r])), k[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r) x[i][r] = fmul2(make_float2(s[i][2 * r], s[i][2 * r + 1]), make_float2(rowf[r], rowf[r]));
      }
      if constexpr (CAP) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            x[i][r] = make_float2(cap_one(x[i][r].x, p.capf) * p.scale2, cap_one(x[i][r].y, p.capf) * p.scale2);
      }
      if (c0 > all_see || c0 < window) {
        const int j = c0 + 16 * warp + 2 * q;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int j0 = j + 8 * i;
            if (j0 > pos[r] || (p.left >= 0 && j0 < pos[r] - p.left)) x[i][r].x = -INFINITY;
            if (j0 + 1 > pos[r] || (p.left >= 0 && j0 + 1 < pos[r] - p.left)) x[i][r].y = -INFINITY;
          }
        if (c0 + kStepTile > u.keys || c0 < u.lo) {       // weight 0 does not silence an infinity
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int jv = j + 8 * (k >> 1) + (k & 1);
            if (jv >= u.keys || jv < u.lo) {
#pragma unroll
              for (int w = 0; w < kWords; ++w) v[k][w] = 0;
            }
          }
        }
      }
      float mx[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) mx[r] = fmaxf(fmax3(x[0][r].x, x[0][r].y, x[1][r].x), x[1][r].y);
      if (__any_sync(0xffffffffu, mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
          const float m1 = fmaxf(m[r], mx[r]), down = m1 == m[r] ? 0.f : m[r] - m1, f = fast_exp2(down);
          m[r] = m1;
          neg[r] = m1 == -INFINITY ? 0.f : -m1;
          l[r] = fmul2(l[r], make_float2(f, f));
          if constexpr (E4M3) {
            M[r] += down;
            Neg[r] = M[r] == -INFINITY ? 0.f : kBoost - M[r];
          } else {
            scale_rows(o, r, f);
          }
        }
      }
      uint32_t w[4];
      float2 pr[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          x[i][r] = fadd2(x[i][r], make_float2(neg[r], neg[r]));
          pr[i][r] = make_float2(fast_exp2(x[i][r].x), fast_exp2(x[i][r].y));
          l[r] = fadd2(l[r], pr[i][r]);
        }
      if constexpr (E4M3) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r) x[i][r] = fadd2(x[i][r], e[i]);
#pragma unroll
        for (int r = 0; r < 2; ++r) mx[r] = fmaxf(fmax3(x[0][r].x, x[0][r].y, x[1][r].x), x[1][r].y);
        if (__any_sync(0xffffffffu, mx[0] > M[0] + kSlack || mx[1] > M[1] + kSlack)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            const float M1 = fmaxf(M[r], mx[r]), down = M1 == M[r] ? 0.f : M[r] - M1;
            M[r] = M1;
            Neg[r] = M1 == -INFINITY ? 0.f : kBoost - M1;
            scale_rows(o, r, fast_exp2(down));
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 y = fadd2(x[i][r], make_float2(Neg[r], Neg[r]));
            w[2 * i + r] = pack2<true>(fast_exp2(y.x), fast_exp2(y.y));
          }
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 2; ++i) w[2 * i + r] = pack2<false>(pr[i][r].x, pr[i][r].y);
      }
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        if constexpr (E4M3) {
          const uint32_t a0 = __byte_perm(v[0][j], v[1][j], 0x5140), a1 = __byte_perm(v[0][j], v[1][j], 0x7362);
          const uint32_t b0 = __byte_perm(v[2][j], v[3][j], 0x5140), b1 = __byte_perm(v[2][j], v[3][j], 0x7362);
          mma16816<true>(o[4 * j], w, codes_f16(a0), codes_f16(b0));
          mma16816<true>(o[4 * j + 1], w, codes_f16_hi(a0), codes_f16_hi(b0));
          mma16816<true>(o[4 * j + 2], w, codes_f16(a1), codes_f16(b1));
          mma16816<true>(o[4 * j + 3], w, codes_f16_hi(a1), codes_f16_hi(b1));
        } else {
          mma16816<false>(o[2 * j], w, __byte_perm(v[0][j], v[1][j], 0x5410), __byte_perm(v[2][j], v[3][j], 0x5410));
          mma16816<false>(o[2 * j + 1], w, __byte_perm(v[0][j], v[1][j], 0x7632), __byte_perm(v[2][j], v[3][j], 0x7632));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    // the unit's, or its piece's, end: the warps meet
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float sum = l[r].x + l[r].y;
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (q == 0) {
        float* y = stat + warp * 2 * kStepRows + g + 8 * r;
        y[0] = m[r];
        y[kStepRows] = sum;
      }
    }
    ok = named_bar_and(1, kComputeWarps * 32, ok);
    if (!ok) break;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (g + 8 * r >= u.rows) continue;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kComputeWarps; ++w) top = fmaxf(top, stat[w * 2 * kStepRows + g + 8 * r]);
      float to = m[r] == top ? 0.f : m[r] - top;
      if constexpr (E4M3) to += M[r] - kBoost;
      to = m[r] == -INFINITY ? 0.f : fast_exp2(to);
      float* dst = red + (warp * kStepRows + g + 8 * r) * D;
      // columns 2 q and 2 q + 1 of product n
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int n = 0; n < kOut; n += 4)
          *reinterpret_cast<float4*>(dst + (E4M3 ? (2 * q + c) * kOut + n : (n >> 3) * 64 + (2 * q + c) * 8 + (n & 7))) =
              make_float4(o[n][2 * r + c] * to, o[n + 1][2 * r + c] * to, o[n + 2][2 * r + c] * to, o[n + 3][2 * r + c] * to);
    }
    named_bar_sync(1, kComputeWarps * 32);
    const bool whole = u.t0 == 0 && u.t1 == u.tiles;
    float* part = cached_part<true, D>(p, blockIdx.x, u.t0 == 0 ? 1 : 0);
    constexpr int kQuads = D / 4;
    for (int y = threadIdx.x; y < u.rows * kQuads; y += kComputeWarps * 32) {
      const int r = y / kQuads, c = y % kQuads;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float top = -INFINITY, tot = 0.f;
#pragma unroll
      for (int w = 0; w < kComputeWarps; ++w) top = fmaxf(top, stat[w * 2 * kStepRows + r]);
#pragma unroll
      for (int w = 0; w < kComputeWarps; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(red + (w * kStepRows + r) * D + 4 * c);
        sum = make_float4(sum.x + z.x, sum.y + z.y, sum.z + z.z, sum.w + z.w);
        const float mw = stat[w * 2 * kStepRows + r];
        tot += mw == -INFINITY ? 0.f : stat[w * 2 * kStepRows + kStepRows + r] * fast_exp2(mw - top);
      }
      if (whole) {
        const int64_t tok = u.start + r / group;
        const int h = u.h * group + r % group;
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
}

// Joins the pieces of the unit that begins in CTA c's share and ends behind it.  A step's row may have hundreds of
// pieces: a warp a row, a lane a piece for their weights.  A chunk's has few: eight lanes a row, so that a warp
// has four rows' loads in flight.
constexpr int kJoinWarps = 4, kStepJoin = kStepRows / kJoinWarps, kChunkJoin = kChunkRows / (4 * kJoinWarps);   // blocks a unit
template <int D, bool STEP>
__device__ __forceinline__ void join(const CachedParams& p, int valid, int c, int r) {
  constexpr int kRows = STEP ? kStepRows : kChunkRows, kLanes = STEP ? 32 : 8, kPer = D / kLanes;
  const CachePlanView pv = cache_plan_view(p.c.plan, p.c.T, p.c.N, p.hq, p.c.hkv);
  Shares sh{};
  if (valid) sh = cached_shares<STEP>(p, pv);
  CachedUnit u{};
  const int n = cached_split<STEP>(p, pv, sh, c, u);
  grid_wait();
  const int lane = threadIdx.x & (kLanes - 1);
  if (n == 0 || (STEP && r >= u.rows)) return;
  const bool in = r < u.rows;
  if (!in) r = 0;
  auto piece = [&](int i) { return cached_part<STEP, D>(p, c + i, i == 0 ? 1 : 0); };
  float top = -INFINITY, l = 0.f;
  for (int i = lane; i < n; i += kLanes) top = fmaxf(top, piece(i)[kRows * D + r]);
#pragma unroll
  for (int w = kLanes / 2; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
  const float neg = top == -INFINITY ? 0.f : -top;
  float o[kPer] = {};
  for (int b = 0; b < n; b += kLanes) {
    const int i = b + lane;
    const float wt = i < n ? fast_exp2(piece(i)[kRows * D + r] + neg) : 0.f;
    if (i < n) l += wt * piece(i)[kRows * (D + 1) + r];
    const int here = min(kLanes, n - b);
#pragma unroll 4
    for (int j = 0; j < here; ++j) {
      const float wj = __shfl_sync(0xffffffffu, wt, j, kLanes);
      const float* src = piece(b + j) + r * D;
      if constexpr (kPer == 2) {
        const float2 y = *reinterpret_cast<const float2*>(src + 2 * lane);
        o[0] = fmaf(wj, y.x, o[0]);
        o[1] = fmaf(wj, y.y, o[1]);
      } else {
#pragma unroll
        for (int k = 0; k < kPer; k += 4) {
          const float4 y = *reinterpret_cast<const float4*>(src + k * kLanes + 4 * lane);
          o[k] = fmaf(wj, y.x, o[k]);
          o[k + 1] = fmaf(wj, y.y, o[k + 1]);
          o[k + 2] = fmaf(wj, y.z, o[k + 2]);
          o[k + 3] = fmaf(wj, y.w, o[k + 3]);
        }
      }
    }
  }
#pragma unroll
  for (int w = kLanes / 2; w; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  if (!in) return;
  const int2 at = cached_row(p, u, r);
  const float inv = 1.f / l;
  __nv_bfloat16* dst = p.out + ((int64_t)at.x * p.hq + at.y) * D;
  if constexpr (kPer == 2) {
    *reinterpret_cast<uint32_t*>(dst + 2 * lane) = pack2<false>(o[0] * inv, o[1] * inv);
  } else {
#pragma unroll
    for (int k = 0; k < kPer; k += 4)
      *reinterpret_cast<uint2*>(dst + k * kLanes + 4 * lane) =
          make_uint2(pack2<false>(o[k] * inv, o[k + 1] * inv), pack2<false>(o[k + 2] * inv, o[k + 3] * inv));
  }
  if (lane == 0) p.lse[(int64_t)at.y * p.c.T + at.x] = (top + log2f(l)) * kLn2;
}
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) cached_join_kernel(const CachedParams p, const int step_blocks) {
  const int valid = cached_valid_rows(p), warp = threadIdx.x >> 5, b = blockIdx.x;
  if (b < step_blocks) {
    join<D, true>(p, valid, b / kStepJoin, (b % kStepJoin) * kJoinWarps + warp);
  } else {
    const int x = b - step_blocks;
    join<D, false>(p, valid, x / kChunkJoin, ((x % kChunkJoin) * kJoinWarps + warp) * 4 + (threadIdx.x & 31) / 8);
  }
}

template <int D, bool E4M3, bool CAP>
cudaError_t launch(const CachedParams& p, cudaStream_t stream) {
  using L = StepSmem<D, E4M3>;
  CUtensorMap tk, tv;
  const uint64_t P = (uint64_t)1 << p.c.page_shift, pages = (uint64_t)p.c.num_pages * p.c.hkv;
  const uint32_t rows = P < kStepTile ? (uint32_t)P : kStepTile;
  if (!make_tmap_u8_3d(&tk, p.c.k, L::kRowBytes, pages, P, P * L::kRowBytes, L::kRowBytes, L::kBoxBytes, rows) ||
      !make_tmap_u8_3d(&tv, p.c.v, L::kRowBytes, pages, P, P * L::kRowBytes, L::kRowBytes, L::kBoxBytes, rows))
    return cudaErrorInvalidValue;
  cudaError_t e = prepare_kernel<cached_step_kernel<D, E4M3, CAP>>(L::kAlloc);
  if (e != cudaSuccess) return e;
  cached_step_kernel<D, E4M3, CAP><<<kStepCtas, kThreads, L::kAlloc, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(bool e4m3, const CachedParams& p, cudaStream_t s) {
  if (e4m3) return p.cap > 0.f ? launch<D, true, true>(p, s) : launch<D, true, false>(p, s);
  return p.cap > 0.f ? launch<D, false, true>(p, s) : launch<D, false, false>(p, s);
}

template <int D>
cudaError_t launch_all(bool e4m3, const CachedParams& p, cudaStream_t s) {
  const int group = p.hq / p.c.hkv;
  const bool steps = group <= kStepRows, chunks = (int64_t)p.max_chunk * group > kStepRows;
  cudaError_t e = cudaSuccess;
  if (steps) e = launch_d<D>(e4m3, p, s);
  if (e == cudaSuccess && chunks) e = launch_cached_chunk(D, e4m3, p, !steps, s);
  if (e != cudaSuccess) return e;
  // starts while the launch before still runs, and waits for it where its results are needed
  const int step_blocks = steps ? kStepCtas * kStepJoin : 0;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(step_blocks + (chunks ? kChunkCtas * kChunkJoin : 0));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cached_join_kernel<D>, p, step_blocks);
}

}  // namespace

cudaError_t launch_cached_fwd(int D, bool e4m3, const CachedParams& p, cudaStream_t s) {
  return D == 128 ? launch_all<128>(e4m3, p, s) : launch_all<64>(e4m3, p, s);
}

}  // namespace flamia
