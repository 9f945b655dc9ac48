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
  static constexpr int kScales = 2 * kTileBytes;                              // in a stage: K's and V's scale bytes
  static constexpr int kStage = 2 * kTileBytes + (E4M3 ? 1024 : 0);           // (stages stay on 1024 bytes)
  static constexpr int kStages = E4M3 ? (D == 128 ? 4 : 6) : (D == 128 ? 2 : 4);
  static constexpr int kRed = kStages * kStage;                               // [4 warps][16 rows][D] floats
  static constexpr int kStat = kRed + kComputeWarps * kStepRows * D * 4;      // [4 warps][m, l, M][16]
  static constexpr int kBar = kStat + kComputeWarps * 3 * kStepRows * 4;
  static constexpr int kBytes = kBar + 2 * kStages * 8;
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
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  __syncthreads();
  const int64_t f0 = sh.begin(blockIdx.x), f1 = sh.begin(blockIdx.x + 1);
  int* status = p.c.plan + kCpStatus;
  bool ok = true;
  uint32_t ring = 0;

  if (warp == kComputeWarps) {
    // ------------------------------------------------------------ producer
    const int P = 1 << p.c.page_shift, rows = min(P, kStepTile), per = kStepTile / rows;      // pages a tile
    const uint32_t page_bytes = 2 * rows * (L::kRowBytes + (E4M3 ? 1 : 0));
    for (int64_t f = f0; f < f1 && ok;) {
      const CachedUnit u = cached_unit<true>(p, pv, f);
      const int t0 = (int)(f - u.begin), t1 = (int)min((int64_t)u.tiles, f1 - u.begin);
      f += t1 - t0;
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
    return;
  }
  // -------------------------------------------------------------- compute
  constexpr int kSteps = D / 16, kOut = D / 8;
  const int g = lane >> 2, q = lane & 3;
  float* red = reinterpret_cast<float*>(smem + L::kRed);
  float* stat = reinterpret_cast<float*>(smem + L::kStat);
  for (int64_t f = f0; f < f1 && ok;) {
    const CachedUnit u = cached_unit<true>(p, pv, f);
    const int t0 = (int)(f - u.begin), t1 = (int)min((int64_t)u.tiles, f1 - u.begin);
    f += t1 - t0;
    // queries: rows g and g + 8, four head dimensions a step of 16
    uint32_t a[kSteps][4];
    float rowf[2];
    int pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      const int2 at = cached_row(p, u, r < u.rows ? r : 0);
      pos[i] = u.keys - u.count + at.x - u.start;
      const __nv_bfloat16* src = p.q + ((int64_t)at.x * p.hq + at.y) * D;
      float x[kSteps][4];
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int d0 = E4M3 ? (D / 4) * q + 4 * s : (s >> 2) * 64 + (2 * q + ((s >> 1) & 1)) * 8 + (s & 1) * 4;
        const uint2 w = r < u.rows ? *reinterpret_cast<const uint2*>(src + d0) : make_uint2(0, 0);
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
    float o[kOut][4] = {};
    float m[2] = {-INFINITY, -INFINITY}, M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    for (int t = t0; t < t1; ++t, ++ring) {
      const uint32_t st = ring % L::kStages;
      if (ok) ok = warp_wait(&full[st], (ring / L::kStages) & 1, status);
      if (!ok) continue;
      const uint8_t* kt = smem + st * L::kStage;
      const uint8_t* vt = kt + L::kTileBytes;
      const int c0 = (u.tile + t) * kStepTile;
      // scores: keys c0 + 16 warp + 8 i + 2 q + {0, 1}
      float s[2][4] = {};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 16 * warp + 8 * i + g;
        if constexpr (E4M3) {
          uint4 w[D / 64];
#pragma unroll
          for (int j = 0; j < D / 64; ++j)
            w[j] = *reinterpret_cast<const uint4*>(kt + swz_offset(row, (D / 4) * q + 16 * j, L::kRowBytes));
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            const uint32_t x = (&w[j / 4].x)[j % 4];
            mma16816<true>(s[i], a[j], codes_f16(x), codes_f16_hi(x));
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint4 w = *reinterpret_cast<const uint4*>(
                kt + (j >> 1) * kStepTile * 128 + swz_offset(row, (2 * q + (j & 1)) * 16, 128));
            mma16816<false>(s[i], a[2 * j], w.x, w.y);
            mma16816<false>(s[i], a[2 * j + 1], w.z, w.w);
          }
        }
      }
      // values of the same keys, in flight while the softmax runs
      constexpr int kWords = L::kRowBytes / 8 / 4;       // a lane's words of a row
      uint32_t v[4][kWords];
      const bool edge = c0 + kStepTile > u.keys || c0 < u.lo;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 16 * warp + 8 * (k >> 1) + 2 * q + (k & 1);
        if constexpr (kWords >= 4) {
#pragma unroll
          for (int j = 0; j < kWords / 4; ++j) {
            const uint4 w = *reinterpret_cast<const uint4*>(vt + j * kStepTile * 128 + swz_offset(row, 16 * g, 128));
            v[k][4 * j] = w.x;
            v[k][4 * j + 1] = w.y;
            v[k][4 * j + 2] = w.z;
            v[k][4 * j + 3] = w.w;
          }
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(vt + swz_offset(row, 8 * g, 64));
          v[k][0] = w.x;
          v[k][1] = w.y;
        }
        if (edge && (c0 + row >= u.keys || c0 + row < u.lo)) {     // weight 0 does not silence an infinity
#pragma unroll
          for (int j = 0; j < kWords; ++j) v[k][j] = 0;
        }
      }
      float e[4];          // exponents of the values' scales
      if constexpr (E4M3) {
        const uint8_t* sc = kt + L::kScales + 16 * warp + 2 * q;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t ks = *reinterpret_cast<const uint16_t*>(sc + 8 * i);
          const uint32_t vs = *reinterpret_cast<const uint16_t*>(sc + kStepTile + 8 * i);
          const float k0 = cache_scale(ks & 255), k1 = cache_scale(ks >> 8);
          s[i][0] = s[i][0] * rowf[0] * k0;
          s[i][1] = s[i][1] * rowf[0] * k1;
          s[i][2] = s[i][2] * rowf[1] * k0;
          s[i][3] = s[i][3] * rowf[1] * k1;
          e[2 * i] = (vs & 255) == 255 ? NAN : (float)(vs & 255) - 127.f;
          e[2 * i + 1] = vs >> 8 == 255 ? NAN : (float)(vs >> 8) - 127.f;
        }
      } else if constexpr (!CAP) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i][k] *= rowf[0];
      }
      if constexpr (CAP) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i][k] = cap_one(s[i][k], p.capf) * p.scale2;
      }
      if (c0 + kStepTile - 1 > u.keys - u.count || (p.left >= 0 && c0 < u.keys - 1 - p.left)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = c0 + 16 * warp + 8 * i + 2 * q + (k & 1), at = pos[k >> 1];
            if (j > at || (p.left >= 0 && j < at - p.left)) s[i][k] = -INFINITY;
          }
      }
      float mx[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) mx[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
      if (__any_sync(0xffffffffu, mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
          const float m1 = fmaxf(m[r], mx[r]), down = m1 == m[r] ? 0.f : m[r] - m1;
          m[r] = m1;
          l[r] *= fast_exp2(down);
          if constexpr (E4M3) M[r] += down;
          else scale_rows(o, r, fast_exp2(down));
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float neg = m[r] == -INFINITY ? 0.f : -m[r];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s[i][2 * r] += neg;
          s[i][2 * r + 1] += neg;
        }
      }
      uint32_t w[4];
      float x[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[i][k] = fast_exp2(s[i][k]);
          l[k >> 1] += x[i][k];
        }
      if constexpr (E4M3) {
        // (a hidden key's scale may be anything)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i][k] = s[i][k] == -INFINITY ? -INFINITY : s[i][k] + e[2 * i + (k & 1)];
#pragma unroll
        for (int r = 0; r < 2; ++r) mx[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
        if (__any_sync(0xffffffffu, mx[0] > M[0] + kSlack || mx[1] > M[1] + kSlack)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            const float M1 = fmaxf(M[r], mx[r]), down = M1 == M[r] ? 0.f : M[r] - M1;
            M[r] = M1;
            scale_rows(o, r, fast_exp2(down));
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float Neg = M[r] == -INFINITY ? 0.f : kBoost - M[r];
#pragma unroll
          for (int i = 0; i < 2; ++i) w[2 * i + r] = pack2<true>(fast_exp2(s[i][2 * r] + Neg), fast_exp2(s[i][2 * r + 1] + Neg));
        }
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 2; ++i) w[2 * i + r] = pack2<false>(x[i][2 * r], x[i][2 * r + 1]);
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
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (q == 0) {
        float* x = stat + warp * 3 * kStepRows + g + 8 * r;
        x[0] = m[r];
        x[kStepRows] = l[r];
      }
    }
    ok = named_bar_and(1, kComputeWarps * 32, ok);
    if (!ok) break;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kComputeWarps; ++w) top = fmaxf(top, stat[w * 3 * kStepRows + g + 8 * r]);
      float to = m[r] == top ? 0.f : m[r] - top;
      if constexpr (E4M3) to += M[r] - kBoost;
      to = m[r] == -INFINITY ? 0.f : fast_exp2(to);
      float* dst = red + (warp * kStepRows + g + 8 * r) * D;
      // columns 2 q and 2 q + 1 of product n
      if constexpr (E4M3) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int n = 0; n < kOut; n += 4)
            *reinterpret_cast<float4*>(dst + (2 * q + c) * kOut + n) =
                make_float4(o[n][2 * r + c] * to, o[n + 1][2 * r + c] * to, o[n + 2][2 * r + c] * to, o[n + 3][2 * r + c] * to);
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int n = 0; n < kOut; n += 4)
            *reinterpret_cast<float4*>(dst + (n >> 3) * 64 + (2 * q + c) * 8 + (n & 7)) =
                make_float4(o[n][2 * r + c] * to, o[n + 1][2 * r + c] * to, o[n + 2][2 * r + c] * to, o[n + 3][2 * r + c] * to);
      }
    }
    named_bar_sync(1, kComputeWarps * 32);
    const bool whole = t0 == 0 && t1 == u.tiles;
    float* part = cached_part<true, D>(p, blockIdx.x, t0 == 0 ? 1 : 0);
    constexpr int kQuads = D / 4;
    for (int x = threadIdx.x; x < u.rows * kQuads; x += kComputeWarps * 32) {
      const int r = x / kQuads, c = x % kQuads;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float top = -INFINITY, tot = 0.f;
#pragma unroll
      for (int w = 0; w < kComputeWarps; ++w) top = fmaxf(top, stat[w * 3 * kStepRows + r]);
#pragma unroll
      for (int w = 0; w < kComputeWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(red + (w * kStepRows + r) * D + 4 * c);
        sum = make_float4(sum.x + y.x, sum.y + y.y, sum.z + y.z, sum.w + y.w);
        const float mw = stat[w * 3 * kStepRows + r];
        tot += mw == -INFINITY ? 0.f : stat[w * 3 * kStepRows + kStepRows + r] * fast_exp2(mw - top);
      }
      if (whole) {
        const int2 at = cached_row(p, u, r);
        const float inv = 1.f / tot;
        *reinterpret_cast<uint2*>(p.out + ((int64_t)at.x * p.hq + at.y) * D + 4 * c) =
            make_uint2(pack2<false>(sum.x * inv, sum.y * inv), pack2<false>(sum.z * inv, sum.w * inv));
        if (c == 0) p.lse[(int64_t)at.y * p.c.T + at.x] = (top + log2f(tot)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(part + r * D + 4 * c) = sum;
        if (c == 0) {
          part[kStepRows * D + r] = top;
          part[kStepRows * (D + 1) + r] = tot;
        }
      }
    }
    named_bar_sync(1, kComputeWarps * 32);
  }
}

// Joins the pieces of the unit that begins in CTA c's share and ends behind it: a warp a row.
constexpr int kJoinWarps = 4, kStepJoin = kStepRows / kJoinWarps, kChunkJoin = 8;      // blocks a unit
template <int D, bool STEP>
__device__ __forceinline__ void join(const CachedParams& p, int valid, int c, int first, int stride) {
  constexpr int kRows = STEP ? kStepRows : kChunkRows, kPer = D / 32;
  const CachePlanView pv = cache_plan_view(p.c.plan, p.c.T, p.c.N, p.hq, p.c.hkv);
  Shares sh{};
  if (valid) sh = cached_shares<STEP>(p, pv);
  const int lane = threadIdx.x & 31;
  CachedUnit u{};
  const bool some = c + 1 < sh.n;
  if (some) u = cached_unit<STEP>(p, pv, sh.begin(c + 1) - 1);
  grid_wait();
  if (!some || u.begin < sh.begin(c) || u.begin + u.tiles <= sh.begin(c + 1)) return;
  const int n = sh.of(u.begin + u.tiles - 1) - c + 1;
  auto piece = [&](int i) { return cached_part<STEP, D>(p, c + i, i == 0 ? 1 : 0); };
  for (int r = first; r < u.rows; r += stride) {
    float top = -INFINITY, l = 0.f;
    for (int i = lane; i < n; i += 32) top = fmaxf(top, piece(i)[kRows * D + r]);
#pragma unroll
    for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
    const float neg = top == -INFINITY ? 0.f : -top;
    float o[kPer] = {};
    for (int b = 0; b < n; b += 32) {
      const int i = b + lane;
      const float wt = i < n ? fast_exp2(piece(i)[kRows * D + r] + neg) : 0.f;
      if (i < n) l += wt * piece(i)[kRows * (D + 1) + r];
      const int here = min(32, n - b);
#pragma unroll 8
      for (int j = 0; j < here; ++j) {
        const float wj = __shfl_sync(0xffffffffu, wt, j);
        const float* src = piece(b + j) + r * D + lane * kPer;
        if constexpr (D == 128) {
          const float4 y = *reinterpret_cast<const float4*>(src);
          o[0] = fmaf(wj, y.x, o[0]);
          o[1] = fmaf(wj, y.y, o[1]);
          o[2] = fmaf(wj, y.z, o[2]);
          o[3] = fmaf(wj, y.w, o[3]);
        } else {
          const float2 y = *reinterpret_cast<const float2*>(src);
          o[0] = fmaf(wj, y.x, o[0]);
          o[1] = fmaf(wj, y.y, o[1]);
        }
      }
    }
#pragma unroll
    for (int w = 16; w; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    const int2 at = cached_row(p, u, r);
    const float inv = 1.f / l;
    __nv_bfloat16* dst = p.out + ((int64_t)at.x * p.hq + at.y) * D + lane * kPer;
#pragma unroll
    for (int j = 0; j < kPer; j += 2) *reinterpret_cast<uint32_t*>(dst + j) = pack2<false>(o[j] * inv, o[j + 1] * inv);
    if (lane == 0) p.lse[(int64_t)at.y * p.c.T + at.x] = (top + log2f(l)) * kLn2;
  }
}
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) cached_join_kernel(const CachedParams p, const int step_blocks) {
  const int valid = cached_valid_rows(p), warp = threadIdx.x >> 5, b = blockIdx.x;
  if (b < step_blocks) {
    join<D, true>(p, valid, b / kStepJoin, (b % kStepJoin) * kJoinWarps + warp, kStepRows);
  } else {
    const int x = b - step_blocks;
    join<D, false>(p, valid, x / kChunkJoin, (x % kChunkJoin) * kJoinWarps + warp, kChunkJoin * kJoinWarps);
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
