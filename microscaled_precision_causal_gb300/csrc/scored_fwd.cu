// Scored attention, forward: bf16 tcgen05 MMAs with TMEM accumulators, an online softmax.
//
//   x = (cap(scale q.k) + bias) log2 e,  running maximum m, p = 2^(x - m), l = sum p,
//   O += bf16(p) V,  O = bf16(O / l), LSE = (m + log2 l) ln 2.
//
// A unit is a forward work item of the plan (up to two document-local 128-query tiles) and
// a query head; one CTA per SM walks the cost-sorted units in boustrophedon order.  Roles
// (384 threads): warp 0 TMA producer, warp 1 MMA issuer, warp 2 TMEM allocator, warps 4-7
// and 8-11 the softmax of the item's first and second query tile (thread = query row).
// While one warpgroup converts its score tile the tensor core runs the other's products.
//
// P enters the PV product in bf16 (V is bf16 and an MMA's operands share a type): half a
// step of 2^-8 per weight, the size of the rounding of O itself.  It stays in tensor memory,
// over the first half of the score columns it came from, so no shared memory is written and
// the PV product reads V alone from there.  The running maximum follows the scores only when
// they outgrow it by more than 8 (in base 2): until then p stays below 2^8, which bf16 and
// the fp32 sums hold as exactly, and O needs no rescaling pass.
//
// TMEM columns: S_0 / P_0 [0, 128), S_1 / P_1 [128, 256), O_0 [256, 256 + D), O_1 [384, ...).
#include "ptx.cuh"
#include "scored.cuh"
#include "tmap.h"

namespace flamia {

namespace {

constexpr int kThreads = 384;
constexpr float kRescaleAbove = 8.f;
constexpr int kLaunchRegs = (65536 / kThreads) & ~7;
constexpr int kRegCtl = 88, kRegSoftmax = 208;
static_assert(kRegCtl * 128 + kRegSoftmax * 256 <= kLaunchRegs * kThreads, "register split");

template <int D>
struct FwdSmem {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kSlots = D == 128 ? 4 : 8;           // K and V tiles in turn
  static constexpr int kQ = 0;                              // [2]
  static constexpr int kKV = 2 * kTileBytes;
  static constexpr int kBias = kKV + kSlots * kTileBytes;   // [2 warpgroups][kBiasTab] floats
  static constexpr int kBar = (kBias + 2 * kBiasTab * 4 + 15) & ~15;
  static constexpr int kBytes = kBar + 256;
  static constexpr int kAlloc = kBytes + 1024;
};

struct Unit {
  int h, hk, t0, ntq, start, len, nt, pre;
  KeyTiles kt;
  int pre_tiles, klo0, klo1, khi0, khi1;
  __device__ __forceinline__ bool sees(int w, int k) const {
    const int u = kt.tile(k);
    return w < ntq && (u < pre_tiles || (w ? u >= klo1 && u <= khi1 : u >= klo0 && u <= khi0));
  }
};

__device__ __forceinline__ Unit make_unit(const ScoredParams& p, const PlanView& pv, int i) {
  Unit U;
  const int item_idx = i / p.hq;
  U.h = i % p.hq;
  U.hk = U.h / (p.hq / p.hkv);
  const int4 item = pv.fwd_items[item_idx];
  const int2 span = pv.fwd_span[item_idx];
  U.t0 = item.y;
  U.ntq = item.z;
  U.start = span.x;
  U.len = span.y;
  U.nt = (U.len + kTile - 1) / kTile;
  U.pre = prefix_of(p, item.x, U.len);
  U.pre_tiles = (U.pre + kTile - 1) / kTile;
  U.klo0 = win_klo(U.t0, p.win);
  U.khi0 = win_khi(U.t0, U.nt, p.win);
  U.klo1 = win_klo(U.t0 + 1, p.win);
  U.khi1 = win_khi(U.t0 + 1, U.nt, p.win);
  U.kt = key_tiles(U.t0, U.t0 + U.ntq - 1, U.nt, U.pre_tiles, p.win);
  return U;
}

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    scored_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const ScoredParams p) {
  using L = FwdSmem<D>;
  constexpr int kSlots = L::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_full = bars;                  // [2]
  uint64_t* q_empty = bars + 2;             // [2]
  uint64_t* s_full = bars + 4;              // [2]
  uint64_t* p_full = bars + 6;              // [2]
  uint64_t* o_full = bars + 8;              // [2]
  uint64_t* drain = bars + 10;
  uint64_t* kv_full = bars + 11;            // [kSlots]
  uint64_t* kv_empty = kv_full + kSlots;    // [kSlots]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kv_empty + kSlots);
  int* status = const_cast<int*>(p.plan) + kPlanStatus;
  const PlanView pv = plan_view(p.plan, p.T, p.N);
  const int n_units = p.plan[kPlanFwdItems] * p.hq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
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

  if (warp < 4) {
    setmaxnreg_dec<kRegCtl>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      uint32_t ring = 0;              // K / V tiles loaded so far
      uint32_t nq[2] = {0, 0};
      bool ok = true;
      auto load = [&](uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, int h, int row) {
        mbar_arrive_expect_tx(bar, L::kTileBytes);
#pragma unroll
        for (int b = 0; b < D / 64; ++b) tma_load_3d(dst + b * kTile * 128, tm, bar, 64 * b, h, row);
      };
      for (int n = 0; ok; ++n) {
        const int i = unit_index(n, n_units);
        if (i < 0) break;
        const Unit U = make_unit(p, pv, i);
        for (int w = 0; w < U.ntq && ok; ++w) {
          if (nq[w] && !(ok = mbar_wait(&q_empty[w], (nq[w] - 1) & 1, status))) break;
          ++nq[w];
          load(smem + L::kQ + w * L::kTileBytes, &tm_q, &q_full[w], U.h, U.start + (U.t0 + w) * kTile);
        }
        for (int k = 0; k < 2 * U.kt.n && ok; ++k, ++ring) {
          const uint32_t st = ring % kSlots;
          if (ring >= kSlots && !(ok = mbar_wait(&kv_empty[st], (ring / kSlots - 1) & 1, status))) break;
          load(smem + L::kKV + st * L::kTileBytes, (k & 1) ? &tm_v : &tm_k, &kv_full[st], U.hk,
               U.start + U.kt.tile(k >> 1) * kTile);
        }
      }
      // nothing may land after the CTA has left (reached early only when a wait ran out)
      for (uint32_t x = ring > kSlots ? ring - kSlots : 0; x < ring; ++x)
        mbar_wait(&kv_full[x % kSlots], (x / kSlots) & 1, status);
      for (int w = 0; w < 2; ++w)
        if (nq[w]) mbar_wait(&q_full[w], (nq[w] - 1) & 1, status);
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      const bool leader = elect_one();
      const uint32_t base16 = (smem_u32(smem) & 0x3FFFFu) >> 4;
      uint32_t ring = 0, nq[2] = {0, 0}, np[2] = {0, 0};
      bool ok = true;
      auto issue_s = [&](int w, uint32_t st) {
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t off = (s / 4) * kTile * 128 + (s % 4) * 32;
          if (leader)
            mma_bf16(tbase + w * 128, sdesc_at(base16, L::kQ + w * L::kTileBytes + off, 16, 1024, kSwizzle128B),
                     sdesc_at(base16, L::kKV + st * L::kTileBytes + off, 16, 1024, kSwizzle128B),
                     idesc_bf16(128, 128, 0, 0), s > 0);
        }
        if (leader) mma_commit(&s_full[w]);
      };
      auto issue_pv = [&](int w, uint32_t st, bool first) {
#pragma unroll
        for (int s = 0; s < kTile / 16; ++s)
          if (leader)
            mma_bf16_ta(tbase + 256 + w * 128, tbase + w * 128 + s * 8,
                        sdesc_at(base16, L::kKV + st * L::kTileBytes + s * 2048, kTile * 128, 1024, kSwizzle128B),
                        idesc_bf16(128, D, 0, 1), (!first || s > 0));
      };
      for (int n = 0; ok; ++n) {
        const int i = unit_index(n, n_units);
        if (i < 0) break;
        const Unit U = make_unit(p, pv, i);
        const int nk = U.kt.n;
        int last[2], first[2] = {-1, -1};        // a tile's last and first key tile, as a place in the list
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          last[w] = nk - 1;
          while (last[w] >= 0 && !U.sees(w, last[w])) --last[w];
        }
        auto scores = [&](int k) {               // S of key tile k for every query tile that sees it
          const uint32_t x = ring + 2 * k, st = x % kSlots;
          if (!(ok = warp_wait(&kv_full[st], (x / kSlots) & 1, status))) return;
          tc_fence_after();
          for (int w = 0; w < U.ntq; ++w) {
            if (!U.sees(w, k)) continue;
            if (first[w] < 0) {
              first[w] = k;
              if (!(ok = warp_wait(&q_full[w], nq[w]++ & 1, status))) return;
              tc_fence_after();
            }
            issue_s(w, st);
            if (k == last[w] && leader) mma_commit(&q_empty[w]);
          }
          if (leader) mma_commit(&kv_empty[st]);
        };
        auto values = [&](int w, int k) {
          if (!(ok = warp_wait(&p_full[w], np[w]++ & 1, status))) return;
          const uint32_t x = ring + 2 * k + 1, st = x % kSlots;
          if (!(ok = warp_wait(&kv_full[st], (x / kSlots) & 1, status))) return;
          tc_fence_after();
          issue_pv(w, st, k == first[w]);
          if (k == last[w] && leader) mma_commit(&o_full[w]);
        };
        scores(0);
        for (int k = 0; k < nk && ok; ++k) {
          // PV of each query tile, its next scores right behind it (the other tile's softmax runs meanwhile)
          const uint32_t xk = ring + 2 * (k + 1), sk = xk % kSlots;
          bool loaded = false;
          for (int w = 0; w < U.ntq && ok; ++w) {
            if (U.sees(w, k)) values(w, k);
            if (!ok || k + 1 >= nk || !U.sees(w, k + 1)) continue;
            if (!loaded) {
              if (!(ok = warp_wait(&kv_full[sk], (xk / kSlots) & 1, status))) break;
              tc_fence_after();
              loaded = true;
            }
            if (first[w] < 0) {
              first[w] = k + 1;
              if (!(ok = warp_wait(&q_full[w], nq[w]++ & 1, status))) break;
              tc_fence_after();
            }
            issue_s(w, sk);
            if (k + 1 == last[w] && leader) mma_commit(&q_empty[w]);
          }
          if (!ok) break;
          if (leader) {
            mma_commit(&kv_empty[(ring + 2 * k + 1) % kSlots]);
            if (k + 1 < nk) mma_commit(&kv_empty[sk]);
          }
        }
        ring += 2 * nk;
      }
      // every MMA has finished before tensor memory is freed
      if (leader) {
        mma_commit(drain);
        mbar_wait(drain, 0, status);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<kRegSoftmax>();
    const int w = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = tbase + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_addr = lane_base + w * 128, o_addr = lane_base + 256 + w * 128;
    float* tab = reinterpret_cast<float*>(smem + L::kBias) + w * kBiasTab;
    const bool has_rel = BIAS && p.rel != nullptr;
    uint32_t ring = 0, ns = 0, no = 0;
    int staged = -1;
    bool ok = true;
    ScoreHead H;
    H.scale2 = p.scale2;
    H.zscale = CAP ? p.scale / p.cap : 0.f;
    H.cap2 = p.cap * kLog2e;
    H.slope2 = 0.f;
    // a warp whose wait ran out goes on through the units without work: it still meets its
    // warpgroup at the barriers around the bias
    for (int n = 0;; ++n) {
      const int i = unit_index(n, n_units);
      if (i < 0) break;
      const Unit U = make_unit(p, pv, i);
      if constexpr (BIAS) {
        if (p.slopes) H.slope2 = p.slopes[U.h] * kLog2e;
        if (has_rel && staged != U.h) {      // each warpgroup has a table: the two need not meet
          named_bar_sync(1 + w, 128);
          stage_bias(tab, p.rel, p.R, U.h, r, 128);
          named_bar_sync(1 + w, 128);
          staged = U.h;
        }
      }
      if (!ok) continue;
      const int t = U.t0 + w, qi = t * kTile + r;
      const int lo = p.win.left < 0 ? 0 : max(0, qi - p.win.left);
      const int hi = p.win.right < 0 ? U.len - 1 : min(U.len - 1, qi + p.win.right);
      float m = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      bool first = true;
      for (int k = 0; k < U.kt.n; ++k) {
        if (!U.sees(w, k)) continue;
        const int u = U.kt.tile(k);
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[w], ns++ & 1, status));
        if (!ok) break;
        tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int g = 0; g < 4; ++g) tmem_ld32(s_addr + 32 * g, v[g]);
        tmem_ld_wait();
        TileBias B{};
        if constexpr (BIAS) B = tile_bias(tab, has_rel, p.R, H.slope2, t, u, u * kTile - qi);
#pragma unroll
        for (int g = 0; g < 4; ++g) score_chunk<CAP, BIAS, 1>(v[g], 32 * g, H, B);
        if (scored_masked(t, u, U.len, U.pre, p.win)) {
          const int c = u * kTile;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint32_t see = column_mask(lo - c, hi - c, U.pre - c, 32 * g);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[g][j] = (see >> j) & 1 ? v[g][j] : 0xff800000u;
          }
        }
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            mx = fmax3(mx, __uint_as_float(v[g][j]), __uint_as_float(v[g][j + 1]));
        // without cap and bias the products are still raw: scale (positive) them in the exponent
        const float f = (CAP || BIAS) ? 1.f : H.scale2;
        mx *= f;
        if (first) {
          m = mx;
          first = false;
        } else if (__any_sync(0xffffffffu, mx > m + kRescaleAbove)) {
          const float m_new = fmaxf(m, mx);
          const float alpha = m_new == m ? 1.f : fast_exp2(m - m_new);      // 0 where nothing was visible yet
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
          l2 = fmul2(l2, make_float2(alpha, alpha));
          m = m_new;
        }
        const float neg = m == -INFINITY ? 0.f : -m;
        const float2 f2 = make_float2(f, f), n2 = make_float2(neg, neg);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int j = 0; j < 64; j += 2) {
            const float2 s2 = make_float2(__uint_as_float(v[2 * half + j / 32][j % 32]),
                                          __uint_as_float(v[2 * half + j / 32][j % 32 + 1]));
            float2 e = (CAP || BIAS) ? fadd2(s2, n2) : ffma2(s2, f2, n2);
            e = make_float2(fast_exp2(e.x), fast_exp2(e.y));
            l2 = fadd2(l2, e);
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(e.x, e.y);
            pk[j / 2] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          tmem_st32(s_addr + 32 * half, pk);
        }
        tmem_st_wait();
        if ((u + 1) * kTile > U.len) {
          const uint32_t x = ring + 2 * k + 1, st = x % kSlots;
          ok = __all_sync(0xffffffffu, mbar_wait(&kv_full[st], (x / kSlots) & 1, status));
          if (!ok) break;
          if (u * kTile + r >= U.len) clear_row<D>(smem + L::kKV + st * L::kTileBytes, r);
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(&p_full[w]);
      }
      ring += 2 * U.kt.n;
      if (!ok || w >= U.ntq) continue;
      ok = __all_sync(0xffffffffu, mbar_wait(&o_full[w], no++ & 1, status));
      if (!ok) continue;
      tc_fence_after();
      const float l = l2.x + l2.y;
      const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);     // a row that sees nothing: O = 0
      const bool al32 = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
      const bool row_valid = qi < U.len;
      const int64_t tok = (int64_t)U.start + qi;
      __nv_bfloat16* orow = p.out + (tok * p.hq + U.h) * D;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(o_addr + 32 * c, o);
        tmem_ld_wait();
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const __nv_bfloat162 b2 =
              __floats2bfloat162_rn(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
          pk[j] = *reinterpret_cast<const uint32_t*>(&b2);
        }
        if (row_valid) {
          __nv_bfloat16* dst = orow + 32 * c;
          if (al32) {
            st_global_v8(dst, pk[0], pk[1], pk[2], pk[3], pk[4], pk[5], pk[6], pk[7]);
            st_global_v8(dst + 16, pk[8], pk[9], pk[10], pk[11], pk[12], pk[13], pk[14], pk[15]);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4*>(dst + 8 * q) = make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
          }
        }
      }
      tc_fence_before();
      if (row_valid) p.lse[(int64_t)U.h * p.T + tok] = l == 0.f ? INFINITY : (m + __log2f(l)) * kLn2;
    }
    // rows outside every document: O = 0, LSE = +inf
    const int valid = p.plan[kPlanValid];
    const int64_t rows = (int64_t)(p.T - valid) * p.hq;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x - 128; i < rows; i += (int64_t)gridDim.x * 256) {
      const int64_t row = valid + i / p.hq;
      const int h = (int)(i % p.hq);
      uint4* dst = reinterpret_cast<uint4*>(p.out + (row * p.hq + h) * D);
#pragma unroll
      for (int j = 0; j < D / 8; ++j) dst[j] = make_uint4(0, 0, 0, 0);
      p.lse[(int64_t)h * p.T + row] = INFINITY;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, bool CAP, bool BIAS>
cudaError_t launch(const ScoredParams& p, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  if (!make_tmap_bf16_3d(&tq, p.q, D, p.hq, p.T, D * 2, (uint64_t)p.hq * D * 2, 64, kTile) ||
      !make_tmap_bf16_3d(&tk, p.k, D, p.hkv, p.T, D * 2, (uint64_t)p.hkv * D * 2, 64, kTile) ||
      !make_tmap_bf16_3d(&tv, p.v, D, p.hkv, p.T, D * 2, (uint64_t)p.hkv * D * 2, 64, kTile))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0, regs = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  constexpr int smem = FwdSmem<D>::kAlloc;
  if (e == cudaSuccess) e = prepare_kernel<scored_fwd_kernel<D, CAP, BIAS>>(smem, &regs);
  if (e != cudaSuccess) return e;
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;    // the register split relies on it
  const int64_t units = ((int64_t)p.T / (kTile * kItemTiles) + p.N + 1) * p.hq;
  if (units > 0x7FFFFFFF) return cudaErrorInvalidValue;
  scored_fwd_kernel<D, CAP, BIAS><<<(unsigned)(units < sms ? units : sms), kThreads, smem, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const ScoredParams& p, cudaStream_t s) {
  const bool bias = p.slopes || p.rel;
  if (p.cap > 0.f) return bias ? launch<D, true, true>(p, s) : launch<D, true, false>(p, s);
  return bias ? launch<D, false, true>(p, s) : launch<D, false, false>(p, s);
}

}  // namespace

cudaError_t launch_scored_fwd(int D, const ScoredParams& p, cudaStream_t s) {
  return D == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace flamia
