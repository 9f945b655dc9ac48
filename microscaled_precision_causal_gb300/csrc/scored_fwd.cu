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
// TMEM columns: S_0 [0, 128), S_1 [128, 256), O_0 [256, 256 + D), O_1 [256 + D, 256 + 2 D).  At
// D = 128 that is all of it and P_w takes the first half of S_w's columns.  At D = 64 the
// P_w have columns of their own behind O (split): the next scores are then ready before the
// softmax asks for them, which matters there because two products of a tile take half as
// long and the exponentials bound the kernel.
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
  static constexpr int kBias = kKV + kSlots * kTileBytes;   // [2 query tiles][kBiasTab] floats
  static constexpr int kBar = (kBias + 2 * kBiasTab * 4 + 15) & ~15;
  static constexpr int kBytes = kBar + 256;
  static constexpr int kAlloc = kBytes + 1024;
};

// What a unit's first loads bring; fetched a unit ahead, so that their latency is not met.
struct RawUnit {
  int i;
  int4 item;
  int2 span;
  __device__ __forceinline__ void fetch(const ScoredParams& p, const PlanView& pv, int n, int n_units) {
    i = unit_index(n, n_units);
    if (i < 0) return;
    item = pv.fwd_items[i / p.hq];
    span = pv.fwd_span[i / p.hq];
  }
};

struct Unit {
  int h, hk, t0, ntq, start, len, pre;
  KeyTiles kt;
  int skip0, skip1;       // the one place of the list that the first / second query tile does not see, or -1
  __device__ __forceinline__ bool sees(int w, int k) const { return w < ntq && k != (w ? skip1 : skip0); }
  __device__ __forceinline__ int last(int w) const { return kt.n - 1 - ((w ? skip1 : skip0) == kt.n - 1 ? 1 : 0); }
};

__device__ __forceinline__ Unit make_unit(const ScoredParams& p, const RawUnit& raw) {
  Unit U;
  U.h = raw.i % p.hq;
  U.hk = U.h / (p.hq / p.hkv);
  U.t0 = raw.item.y;
  U.ntq = raw.item.z;
  U.start = raw.span.x;
  U.len = raw.span.y;
  U.pre = prefix_of(p, raw.item.x, U.len);
  const int nt = (U.len + kTile - 1) / kTile, pt = (U.pre + kTile - 1) / kTile, t1 = U.t0 + U.ntq - 1;
  U.kt = key_tiles(U.t0, t1, nt, pt, p.win);
  // the two windows start and end at most a tile apart: the second may miss the window's first
  // tile, the first its last one
  const bool late = t1 > U.t0 && win_klo(t1, p.win) > U.kt.lo && U.kt.lo >= pt;
  const bool early = t1 > U.t0 && win_khi(U.t0, nt, p.win) < U.kt.tile(U.kt.n - 1) && U.kt.tile(U.kt.n - 1) >= pt;
  U.skip1 = late ? U.kt.a : -1;
  U.skip0 = early ? U.kt.n - 1 : -1;
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
  uint64_t* o_full = bars + 6;              // [2]
  uint64_t* s_free = bars + 8;              // [2] (split)
  uint64_t* p_full = bars + 10;             // [2 query tiles][2 halves of 64 keys]
  uint64_t* drain = bars + 14;
  uint64_t* kv_full = bars + 15;            // [kSlots]
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
      mbar_init(&o_full[i], 1);
      mbar_init(&s_free[i], 128);
      mbar_init(&p_full[2 * i], 128);
      mbar_init(&p_full[2 * i + 1], 128);
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
  constexpr bool kSplit = D == 64;
  constexpr uint32_t kO = 256, kP = 384;

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
      RawUnit raw;
      raw.fetch(p, pv, 0, n_units);
      for (int n = 1; ok && raw.i >= 0; ++n) {
        const Unit U = make_unit(p, raw);
        raw.fetch(p, pv, n, n_units);
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
      uint32_t ring = 0, nq0 = 0, nq1 = 0, np0 = 0, np1 = 0, ns0 = 0, ns1 = 0;
      bool ok = true;
      RawUnit raw;
      raw.fetch(p, pv, 0, n_units);
      for (int n = 1; ok && raw.i >= 0; ++n) {
        const Unit U = make_unit(p, raw);
        raw.fetch(p, pv, n, n_units);
        const int nk = U.kt.n, last0 = U.last(0), last1 = U.last(1);
        int first0 = -1, first1 = -1;              // places in the list of key tiles
        // S of query tile w and key tile k (whose K is in the ring's slot st)
        auto scores = [&](int w, int k, uint32_t st) {
          int& first = w ? first1 : first0;
          if (first < 0) {
            first = k;
            if (!(ok = warp_wait(&q_full[w], (w ? nq1++ : nq0++) & 1, status))) return;
          }
          if (kSplit) {                            // the last scores have been read
            uint32_t& ns = w ? ns1 : ns0;
            if (ns && !(ok = warp_wait(&s_free[w], (ns - 1) & 1, status))) return;
            ++ns;
          }
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t off = (s / 4) * kTile * 128 + (s % 4) * 32;
            if (leader)
              mma_bf16(tbase + w * 128, sdesc_at(base16, L::kQ + w * L::kTileBytes + off, 16, 1024, kSwizzle128B),
                       sdesc_at(base16, L::kKV + st * L::kTileBytes + off, 16, 1024, kSwizzle128B),
                       idesc_bf16(128, 128, 0, 0), s > 0);
          }
          if (leader) {
            mma_commit(&s_full[w]);
            if (k == (w ? last1 : last0)) mma_commit(&q_empty[w]);
          }
        };
        // O += P V, half of the keys at a time as the softmax hands them in
        auto values = [&](int w, int k, uint32_t st) {
          const uint32_t par = (w ? np1++ : np0++) & 1;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!(ok = warp_wait(&p_full[2 * w + half], par, status))) return;
            tc_fence_after();
#pragma unroll
            for (int s = 4 * half; s < 4 * half + 4; ++s)
              if (leader)
                mma_bf16_ta(tbase + kO + w * D, tbase + (kSplit ? kP + 64 * w : 128 * w) + s * 8,
                            sdesc_at(base16, L::kKV + st * L::kTileBytes + s * 2048, kTile * 128, 1024, kSwizzle128B),
                            idesc_bf16(128, D, 0, 1), (k != (w ? first1 : first0) || s > 0));
          }
          if (leader && (kSplit || k == (w ? last1 : last0))) mma_commit(&o_full[w]);
        };
        auto landed = [&](uint32_t x) { return ok = warp_wait(&kv_full[x % kSlots], (x / kSlots) & 1, status); };
        if (!landed(ring)) break;
        for (int w = 0; w < 2 && ok; ++w)
          if (U.sees(w, 0)) scores(w, 0, ring % kSlots);
        if (!ok) break;
        if (leader) mma_commit(&kv_empty[ring % kSlots]);
        for (int k = 0; k < nk && ok; ++k) {
          const uint32_t xv = ring + 2 * k + 1, xk = xv + 1;
          const bool more = k + 1 < nk;
          if (kSplit && more) {
            if (!landed(xk)) break;
            for (int w = 0; w < 2 && ok; ++w)
              if (U.sees(w, k + 1)) scores(w, k + 1, xk % kSlots);
            if (!ok) break;
            if (leader) mma_commit(&kv_empty[xk % kSlots]);
          }
          if (!landed(xv)) break;
          for (int w = 0; w < 2 && ok; ++w) {
            if (U.sees(w, k)) values(w, k, xv % kSlots);
            // its next scores go over P, right behind its product; the other tile's softmax runs meanwhile
            if (!kSplit && ok && more && U.sees(w, k + 1) && landed(xk)) scores(w, k + 1, xk % kSlots);
          }
          if (ok && leader) {
            mma_commit(&kv_empty[xv % kSlots]);
            if (!kSplit && more) mma_commit(&kv_empty[xk % kSlots]);
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
    const uint32_t s_addr = lane_base + w * 128, o_addr = lane_base + kO + w * D;
    const uint32_t p_addr = kSplit ? lane_base + kP + 64 * w : s_addr;
    float* tab = reinterpret_cast<float*>(smem + L::kBias) + w * kBiasTab;
    const int R = bias_range(p), near = near_tiles(R);
    const float scale2 = p.scale2, inv_scale2 = 1.f / p.scale2;
    uint32_t ring = 0, ns = 0, no = 0;
    int staged = -1;
    bool ok = true;
    HeadBias HB{};
    RawUnit raw;
    raw.fetch(p, pv, 0, n_units);
    // a warp whose wait ran out goes on through the units without work: it still meets its
    // warpgroup at the barriers around the bias
    for (int n = 1; raw.i >= 0; ++n) {
      const Unit U = make_unit(p, raw);
      raw.fetch(p, pv, n, n_units);
      if constexpr (BIAS) {
        if (staged != U.h) {      // each warpgroup has a table: the two need not meet
          HB = head_bias(p, U.h);
          named_bar_sync(1 + w, 128);
          stage_bias(tab, p, U.h, r, 128);
          named_bar_sync(1 + w, 128);
          staged = U.h;
        }
      }
      if (!ok) continue;
      const int t = U.t0 + w, qi = t * kTile + r;
      const int lo = p.win.left < 0 ? 0 : max(0, qi - p.win.left);
      const int hi = p.win.right < 0 ? U.len - 1 : min(U.len - 1, qi + p.win.right);
      const FullTiles full = full_tiles(t, U.len, U.pre, p.win);
      const int skip = w >= U.ntq ? -2 : (w ? U.skip1 : U.skip0);
      float m = -INFINITY;
      float2 la = make_float2(0.f, 0.f), lb = la;
      bool first = true;
      for (int k = 0; k < U.kt.n && skip != -2; ++k) {
        if (k == skip) continue;
        const int u = U.kt.tile(k);
        TileBias B{};
        if constexpr (BIAS) B = tile_bias(tab, HB, R, near, inv_scale2, t, u, u * kTile - qi);
        const bool masked = !full.has(u);
        const bool plain = !BIAS || B.plain();
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[w], ns++ & 1, status));
        if (!ok) break;
        tc_fence_after();
        uint32_t v[4][32];
        float cm[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) tmem_ld32_max(s_addr + 32 * g, v[g], cm[g]);
        tmem_ld_wait();
        if (kSplit) {
          tc_fence_before();
          mbar_arrive(&s_free[w]);
        }
        float mx = fmaxf(fmax3(cm[0], cm[1], cm[2]), cm[3]);      // of the raw products, from the load
        if constexpr (CAP) {
          cap_products(v, p.capf);
          const float z = mx * p.capf.zscale;                       // monotone
          mx = fabsf(z) < 1e-3f ? mx : p.capf.inv * tanh_any(z);
        }
        const float f = BIAS ? B.factor(scale2) : scale2;
        if (masked || !plain) {
          if constexpr (BIAS) {
#pragma unroll
            for (int g = 0; g < 4; ++g) bias_chunk<1>(v[g], 32 * g, scale2, B);
          }
          if (masked) {
            const int c = u * kTile;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const uint32_t see = column_mask(lo - c, hi - c, U.pre - c, 32 * g);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[g][j] = (see >> j) & 1 ? v[g][j] : 0xff800000u;
            }
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) cm[g] = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; j += 2)
#pragma unroll
            for (int g = 0; g < 4; ++g) cm[g] = fmax3(cm[g], __uint_as_float(v[g][j]), __uint_as_float(v[g][j + 1]));
          mx = fmaxf(fmax3(cm[0], cm[1], cm[2]), cm[3]);
        }
        mx = fmaf(mx, f, B.c);
        if (first) {
          m = mx;
        } else if (__any_sync(0xffffffffu, mx > m + kRescaleAbove)) {
          const float m_new = fmaxf(m, mx);
          const float alpha = m_new == m ? 1.f : fast_exp2(m - m_new);      // 0 where nothing was visible yet
          la = fmul2(la, make_float2(alpha, alpha));
          lb = fmul2(lb, make_float2(alpha, alpha));
          m = m_new;
          if (kSplit) {                // the last product has to be in
            ok = __all_sync(0xffffffffu, mbar_wait(&o_full[w], no & 1, status));
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
        if ((u + 1) * kTile > U.len) {
          const uint32_t x = ring + 2 * k + 1, st = x % kSlots;
          ok = __all_sync(0xffffffffu, mbar_wait(&kv_full[st], (x / kSlots) & 1, status));
          if (!ok) break;
          if (u * kTile + r >= U.len) clear_row<D>(smem + L::kKV + st * L::kTileBytes, r);
          fence_proxy_async_smem();
        }
        const float neg = (m == -INFINITY ? 0.f : -m) + B.c;
        const float2 f2 = make_float2(f, f), n2 = make_float2(neg, neg);
        // P in two halves of 64 keys: the first one's product starts while the second is computed
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int j = 0; j < 64; j += 4) {
            const int g = 2 * half + j / 32, c = j % 32;
            float2 e0 = ffma2(pair_of(v[g], c), f2, n2), e1 = ffma2(pair_of(v[g], c + 2), f2, n2);
            e0 = make_float2(fast_exp2(e0.x), fast_exp2(e0.y));
            e1 = make_float2(fast_exp2(e1.x), fast_exp2(e1.y));
            la = fadd2(la, e0);
            lb = fadd2(lb, e1);
            const __nv_bfloat162 b0 = __floats2bfloat162_rn(e0.x, e0.y), b1 = __floats2bfloat162_rn(e1.x, e1.y);
            pk[j / 2] = *reinterpret_cast<const uint32_t*>(&b0);
            pk[j / 2 + 1] = *reinterpret_cast<const uint32_t*>(&b1);
          }
          if (kSplit && half == 0 && !first) {       // the last P has been read
            ok = __all_sync(0xffffffffu, mbar_wait(&o_full[w], no++ & 1, status));
            if (!ok) break;
            tc_fence_after();
          }
          tmem_st32(p_addr + 32 * half, pk);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full[2 * w + half]);
        }
        first = false;
        if (!ok) break;
      }
      ring += 2 * U.kt.n;
      if (!ok || w >= U.ntq) continue;
      ok = __all_sync(0xffffffffu, mbar_wait(&o_full[w], no++ & 1, status));
      if (!ok) continue;
      tc_fence_after();
      const float l = (la.x + la.y) + (lb.x + lb.y);
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
