// Scored attention, forward: bf16 tcgen05 MMAs with TMEM accumulators, an online softmax.
//
//   x = (cap(scale q.k) + bias) log2 e,  running maximum m, p = 2^(x - m), l = sum p,
//   O += bf16(p) V,  O = bf16(O / l), LSE = (m + log2 l) ln 2.
//
// A unit is a forward work item of the plan (up to two document-local 128-query tiles) and
// a query head, in the plan's cost order.  Below kTakeBelow units per SM the grid has a CTA
// per unit, and a running CTA takes over one that has not started (cluster launch control):
// units go to whoever is free, and a CTA's pipelines run on across them.  Taken over against dealt
// out in boustrophedon rounds to a CTA per SM, D = 128, us: documents of 84 to 2886, 16384 rows,
// 8 units per SM 205 / 220, 16 units 400 / 425, 32 units 785 / 836; two documents of 16384,
// 14 units 1698 / 1815; four of 8192, 7 units 453 / 492, 28 units 1820 / 1760.  With many units a
// round evens itself out, and rounds keep the query heads of one kv head at the same keys,
// which pays where the keys and values of a round are more than L2 holds.
// Roles (512 threads):
//   warp 0        TMA producer: Q tiles, K and V tiles through a ring
//   warp 1        MMA issuer: a query tile's products (O += P V, then its next scores over P)
//                 are queued whole before the other's, so that the two softmax warpgroups get
//                 their scores half a step apart.  Queued side by side they would finish together,
//                 and the arithmetic of both would alternate with the products of both (2.03
//                 instead of 1.73 ms on four causal documents of 8192, 32 heads on 8, slopes).
//                 At D = 64 the scores come ahead of the softmax anyway, and warp 3 issues the
//                 second query tile's, so that neither waits for the other (0.64 instead of 0.78
//                 ms on two noncausal documents of 8192, 16 heads)
//   warp 2        TMEM allocator; describes the units ahead of the other roles
//   warps 4-11    softmax, a warpgroup per query tile, thread = query row
//   warps 12-15   stage the next unit's bias table and write the finished O, while the softmax
//                 warps are in the next unit already
//
// P enters the PV product in bf16 (V is bf16 and an MMA's operands share a type): half a
// step of 2^-8 per weight, the size of the rounding of O itself.  It stays in tensor memory,
// over the first half of the score columns it came from, so no shared memory is written and
// the PV product reads V alone from there.
//
// m is a reference near the row's maximum, not the maximum: p = 2^(x - m) only has to stay in
// range, as bf16 and fp32 hold 2^-60 and 2^8 alike.  It moves when a tile outgrows it by more
// than 8, so that O is seldom rescaled, and where every key of a tile is seen it comes from the
// tensor memory load's own reduction of the raw products (plain: their maximum; capped: their
// largest magnitude, which also says how long a polynomial the cap needs; slopes: their maximum
// and the tile's largest bias), as long as it can be no more than 2^64 too high.
// x - m is one multiply-add from the raw product, exact but for its own rounding, while m was rounded: from
// |m| = 2^30 on the difference could pass 2^128.  No model means such scores, but a run that diverges has them: from
// 2^28 on a row's x and m are shrunk by the power of two that brings m below 2^29.  Products that differ at all
// there still differ by 16 and more.  (From m again in every tile: kept from tile to tile it costs 640 instead of 632
// us on the noncausal buckets case of 2 x 8192, 16 heads, d = 64, and 622 without.)
//
// TMEM columns: S_0 [0, 128), S_1 [128, 256), O_0 [256, 256 + D), O_1 [256 + D, 256 + 2 D).  At
// D = 128 that is all of it and P_w takes the first half of S_w's columns.  At D = 64 the
// P_w have columns of their own behind O (split): the next scores are then ready before the
// softmax asks for them, which matters there because two products of a tile take half as
// long and the exponentials bound the kernel.
#include <type_traits>

#include "ptx.cuh"
#include "scored.cuh"
#include "tmap.h"

namespace flamia {

namespace {

constexpr int kThreads = 512;
constexpr float kRescaleAbove = 8.f, kLoose = 64.f;
__device__ __forceinline__ float shrink_for(float m) {
  const uint32_t e = (__float_as_uint(m) >> 23) & 255;       // of 2^(e - 127), 255: nothing visible yet
  return e >= 127 + 28 && e < 255 ? __uint_as_float((2 * 127 + 28 - e) << 23) : 1.f;
}
constexpr int kLaunchRegs = (65536 / kThreads) & ~7;
constexpr int kRegCtl = 64, kRegAux = 80, kRegSoftmax = 184;
static_assert(kRegCtl * 128 + kRegAux * 128 + kRegSoftmax * 256 <= kLaunchRegs * kThreads, "register split");

// A unit's description, worked out by one warp some units ahead and read by every role from
// shared memory: the divisions and the dependent loads behind it stay off their paths.
struct alignas(16) Unit {
  int h, hk, t0, ntq;     // ntq 0: no more units
  int start, len, pre, skip0;
  KeyTiles kt;
  int index;              // in the list
  int skip1;              // skip0 / 1: the one place of the list that the first / second query tile does not see, or -1
};
static_assert(sizeof(Unit) == 64, "read as four 16-byte words");
constexpr int kUnits = 8;  // described at a time: more units than the K / V ring can hold tiles of
constexpr int kTakeBelow = 24;              // units per SM below which they are taken over, not dealt out
constexpr int kAskAhead = 1;                // the next unit is asked for before the last so many key tiles of one are loaded

__device__ __forceinline__ Unit make_unit(const ScoredParams& p, const PlanView& pv, int i) {
  Unit U{};
  if (i < 0) return U;
  const int4 item = pv.fwd_items[i / p.hq];
  const int2 span = pv.fwd_span[i / p.hq];
  U.index = i;
  U.h = i % p.hq;
  U.hk = U.h / (p.hq / p.hkv);
  U.t0 = item.y;
  U.ntq = item.z;
  U.start = span.x;
  U.len = span.y;
  U.pre = prefix_of(p, item.x, U.len);
  const int nt = (U.len + kTile - 1) / kTile, pt = (U.pre + kTile - 1) / kTile, t1 = U.t0 + U.ntq - 1;
  U.kt = key_tiles(U.t0, t1, nt, pt, p.win);
  // the two windows start and end at most a tile apart: the second may miss the window's first
  // tile, the first its last one
  const bool late = t1 > U.t0 && win_klo(t1, p.win) > U.kt.lo && U.kt.lo >= pt;
  const bool early = t1 > U.t0 && win_khi(U.t0, nt, p.win) < U.kt.tile(0) && U.kt.tile(0) >= pt;
  U.skip1 = late ? U.kt.n - 1 - U.kt.a : -1;
  U.skip0 = early ? 0 : -1;
  return U;
}
// Unit n of the CTA; ntq 0 when there is none, or when the wait ran out.
__device__ __forceinline__ Unit read_unit(const uint8_t* units, uint64_t* full, int n, bool whole_warp, bool& ok, int* status) {
  ok = mbar_wait(&full[n % kUnits], (n / kUnits) & 1, status);
  if (whole_warp) ok = __all_sync(0xffffffffu, ok);
  union {
    Unit u;
    int4 w[4];
  } x;
  const int4* src = reinterpret_cast<const int4*>(units + (n % kUnits) * sizeof(Unit));
#pragma unroll
  for (int i = 0; i < 4; ++i) x.w[i] = src[i];
  if (!ok) x.u.ntq = 0;
  return x.u;
}

// The plan orders its items by what the window lets them see and knows no prefix.  With one, a call of
// few items and several units per SM ranks them by their own work first (a thread an item,
// before the roles part), so that the long units are not the last ones: 154 -> 133 us for odd
// prefix documents of 9097 rows, 8 heads on 2.  (In the backward the same cost every call's
// loops their registers, 5% of them, and gained 3% here.)
constexpr int kRanked = 128, kRankSms = 152;
__device__ __forceinline__ bool ranked(const ScoredParams& p, int n_units) {
  return p.prefix && n_units > kRankSms && n_units <= kRanked * p.hq;
}
__device__ __forceinline__ void rank_items(const ScoredParams& p, const PlanView& pv, int n_units, uint8_t* order,
                                           int* cost) {
  if (!ranked(p, n_units)) return;
  const int i = threadIdx.x, items = n_units / p.hq;
  if (i < items) {
    const Unit U = make_unit(p, pv, i * p.hq);
    cost[i] = U.kt.n * (2 + U.ntq);      // a unit of one query tile takes three quarters of one of two
  }
  __syncthreads();
  if (i < items) {
    int rank = 0;
    for (int j = 0; j < items; ++j) rank += cost[j] > cost[i] || (cost[j] == cost[i] && j < i);
    order[rank] = (uint8_t)i;
  }
  __syncthreads();
}
__device__ __forceinline__ int ranked_unit(const ScoredParams& p, int n_units, const uint8_t* order, int i) {
  return i >= 0 && ranked(p, n_units) ? order[i / p.hq] * p.hq + i % p.hq : i;
}

template <int D>
struct FwdSmem {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kSlots = D == 128 ? 4 : 8;           // K and V tiles in turn
  static constexpr int kQ = 0;                              // [2]
  static constexpr int kKV = 2 * kTileBytes;
  static constexpr int kBias = kKV + kSlots * kTileBytes;   // [2 units in turn][kBiasTab] floats
  static constexpr int kInv = kBias + 2 * kBiasTab * 4;     // [2 query tiles][128] 1 / l
  static constexpr int kUnit = kInv + 1024;                 // [kUnits]
  static constexpr int kClc = kUnit + kUnits * 64;          // answer to a request for another CTA's unit
  static constexpr int kOrder = kClc + 16;                  // of the items, when they are ranked here, and their costs
  static constexpr int kBar = kOrder + kRanked * 5;
  static constexpr int kBytes = kBar + 512;
  static constexpr int kAlloc = kBytes + 1024;
};

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    scored_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const ScoredParams p, const bool take) {
  using L = FwdSmem<D>;
  constexpr int kSlots = L::kSlots;
  constexpr bool kSplit = D == 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_full = bars;                  // [2 query tiles], as the next seven
  uint64_t* q_empty = bars + 2;
  uint64_t* s_full = bars + 4;
  uint64_t* s_free = bars + 6;              // (split) scores read
  uint64_t* pv_done = bars + 8;             // (split) P read
  uint64_t* o_full = bars + 10;             // the unit's O is whole
  uint64_t* o_free = bars + 12;             // and written out
  uint64_t* l_ready = bars + 14;
  uint64_t* p_full = bars + 16;             // [2 query tiles][2 halves of 64 keys]
  uint64_t* tab_full = bars + 20;           // [2 units in turn]
  uint64_t* drain = bars + 22;              // [2 issuers]
  uint64_t* unit_ask = bars + 24;
  uint64_t* clc_bar = bars + 25;
  uint64_t* unit_full = bars + 26;          // [kUnits]
  uint64_t* unit_done = unit_full + kUnits; // [kUnits] written out, and read by the second query tile's softmax
  uint64_t* kv_full = unit_done + kUnits;   // [kSlots]
  uint64_t* kv_empty = kv_full + kSlots;    // [kSlots]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kv_empty + kSlots);
  int* status = const_cast<int*>(p.plan) + kPlanStatus;
  const PlanView pv = plan_view(p.plan, p.T, p.N);
  const int n_units = p.plan[kPlanFwdItems] * p.hq;
  uint8_t* units = smem + L::kUnit;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Rows outside every document (O = 0, LSE = +inf) are dealt out to the units, or to all CTAs
  // where there is none.
  auto clear_tail = [&](int64_t part, int64_t parts, int r, int threads) {
    const int valid = p.plan[kPlanValid];
    const int64_t rows = (int64_t)(p.T - valid) * p.hq;
    for (int64_t i = part * threads + r; i < rows; i += parts * threads) {
      const int64_t row = valid + i / p.hq;
      const int h = (int)(i % p.hq);
      uint4* dst = reinterpret_cast<uint4*>(p.out + (row * p.hq + h) * D);
#pragma unroll
      for (int j = 0; j < D / 8; ++j) dst[j] = make_uint4(0, 0, 0, 0);
      p.lse[(int64_t)h * p.T + row] = INFINITY;
    }
  };
  if ((int64_t)blockIdx.x >= n_units) {        // the grid goes by a bound on the units
    if (n_units == 0) clear_tail(blockIdx.x, gridDim.x, threadIdx.x, kThreads);
    return;
  }
  uint8_t* order = smem + L::kOrder;
  rank_items(p, pv, n_units, order, reinterpret_cast<int*>(order + kRanked));

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 128);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_free[i], 128);
      mbar_init(&l_ready[i], 128);
      mbar_init(&p_full[2 * i], 128);
      mbar_init(&p_full[2 * i + 1], 128);
      mbar_init(&tab_full[i], 128);
      mbar_init(&drain[i], 1);
    }
    mbar_init(unit_ask, 1);
    mbar_init(clc_bar, 1);
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&unit_full[i], 1);
      mbar_init(&unit_done[i], 1 + 4);              // (its four warps)
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], kSplit ? 2 : 1);      // issuers
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
      for (int n = 0; ok; ++n) {
        const Unit U = read_unit(units, unit_full, n, false, ok, status);
        if (U.ntq == 0) break;
        for (int w = 0; w < U.ntq && ok; ++w) {
          if (nq[w] && !(ok = mbar_wait(&q_empty[w], (nq[w] - 1) & 1, status))) break;
          ++nq[w];
          load(smem + L::kQ + w * L::kTileBytes, &tm_q, &q_full[w], U.h, U.start + (U.t0 + w) * kTile);
        }
        for (int k = 0; k < 2 * U.kt.n && ok; ++k, ++ring) {
          const uint32_t st = ring % kSlots;
          if (k == max(2 * (U.kt.n - kAskAhead), 0)) mbar_arrive(unit_ask);
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
    } else if (warp == 2 && lane == 0) {
      // ---------------------------------------------------------- units
      // Dealt out: in boustrophedon order, described as far ahead as there are slots.  Taken over: the
      // CTA's own unit first; then, whenever the loads of a unit come to their end, the unit of a CTA
      // that has not started, whose launch is cancelled.
      bool ok = true;
      int i = blockIdx.x;
      uint32_t asked = 0;
      for (int n = 0; ok; ++n) {
        if (n >= kUnits && !(ok = mbar_wait(&unit_done[n % kUnits], (n / kUnits - 1) & 1, status))) break;
        if (!take) {
          i = unit_index(n, n_units);
        } else if (n > 0) {
          if (!(ok = mbar_wait(unit_ask, (n - 1) & 1, status))) break;
          do {
            fence_proxy_async_smem();          // the last answer was read before the next one lands
            mbar_arrive_expect_tx(clc_bar, 16);
            clc_try_cancel(smem + L::kClc, clc_bar);
            if (!(ok = mbar_wait(clc_bar, asked++ & 1, status))) break;
            i = clc_cancelled_x(smem + L::kClc);
          } while (i >= n_units);              // a CTA without a unit
        }
        const Unit U = make_unit(p, pv, ok ? ranked_unit(p, n_units, order, i) : -1);
        *reinterpret_cast<Unit*>(units + (n % kUnits) * sizeof(Unit)) = U;
        mbar_arrive(&unit_full[n % kUnits]);
        if (U.ntq == 0) break;
      }
    } else if (warp == 1 || (kSplit && warp == 3)) {
      // ---------------------------------------------------------- MMA issuer of query tiles w0 .. w1 - 1
      const int w0 = kSplit ? warp >> 1 : 0, w1 = kSplit ? w0 + 1 : 2;
      const bool leader = elect_one();
      const uint32_t base16 = (smem_u32(smem) & 0x3FFFFu) >> 4;
      const uint32_t tb = (uint32_t)warp_uniform((int)tbase);
      uint32_t ring = 0, nq0 = 0, nq1 = 0, np0 = 0, np1 = 0, ns0 = 0, ns1 = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const Unit U = read_unit(units, unit_full, n, true, ok, status);
        const int ntq = warp_uniform(U.ntq);
        if (ntq == 0) break;
        const int nk = warp_uniform(U.kt.n), skip0 = warp_uniform(U.skip0), skip1 = warp_uniform(U.skip1);
        auto sees = [&](int w, int k) { return w < ntq && k != (w ? skip1 : skip0); };
        auto first = [&](int w) { return (w ? skip1 : skip0) == 0 ? 1 : 0; };
        auto last = [&](int w) { return (w ? skip1 : skip0) == nk - 1 ? nk - 2 : nk - 1; };
        auto landed = [&](uint32_t x) { return ok = warp_wait(&kv_full[x % kSlots], (x / kSlots) & 1, status); };
        auto release = [&](uint32_t x) {
          if (leader) mma_commit(&kv_empty[x % kSlots]);
        };
        auto scores = [&](int w, int k) {          // S of key tile k.  A (Q): q_full at the unit's first; B (K): kv_full
          const uint32_t x = ring + 2 * k, st = x % kSlots;
          if (k == first(w) && !(ok = warp_wait(&q_full[w], (w ? nq1 : nq0) & 1, status))) return;
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
            if (k == last(w)) mma_commit(&q_empty[w]);
          }
        };
        // O += P V, half of the keys at a time as they are handed in.  A (P in TMEM): p_full; B (V): kv_full
        auto values = [&](int w, int k) {
          const uint32_t x = ring + 2 * k + 1, st = x % kSlots;
          if (!landed(x)) return;
          const uint32_t nq = w ? nq1 : nq0;
          if (k == first(w) && nq && !(ok = warp_wait(&o_free[w], (nq - 1) & 1, status))) return;
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
                            (k != first(w) || s > 0));
          }
          if (leader) {
            if (kSplit) mma_commit(&pv_done[w]);
            if (k == last(w)) mma_commit(&o_full[w]);
          }
        };
        for (int w = w0; w < w1 && ok; ++w) {
          if (sees(w, 0)) scores(w, 0);
          else if (kSplit) landed(ring);           // (a tile that nobody else of this issuer has waited for)
        }
        if (ok) release(ring);
        for (int k = 0; k < nk && ok; ++k) {
          for (int w = w0; w < w1 && ok; ++w) {
            const bool next = k + 1 < nk && sees(w, k + 1);
            if (kSplit && next) scores(w, k + 1);
            if (ok && sees(w, k)) values(w, k);
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
    float* inv_l = reinterpret_cast<float*>(smem + L::kInv) + w * 128;
    const int R = bias_range(p), near = near_tiles(R);
    const float scale2 = p.scale2;
    uint32_t ring = 0, ns = 0, nu = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const Unit U = read_unit(units, unit_full, n, true, ok, status);
      if (U.ntq == 0) break;
      const float* tab = reinterpret_cast<const float*>(smem + L::kBias) + (n & 1) * kBiasTab;
      const int nk = U.kt.n, skip = w >= U.ntq ? -2 : (w ? U.skip1 : U.skip0);
      HeadBias HB{};
      if constexpr (BIAS) {      // (of every unit, so that the barrier's phases stay in step)
        ok = __all_sync(0xffffffffu, mbar_wait(&tab_full[n & 1], (n >> 1) & 1, status));
        if (!ok) break;
        HB = head_bias(tab);
      }
      if (w == 1) {              // a unit of one query tile asks nothing else of these warps: nobody would wait for them
        __syncwarp();
        if (lane == 0) mbar_arrive(&unit_done[n % kUnits]);
      }
      if (skip == -2) {
        ring += 2 * nk;
        continue;
      }
      const int t = U.t0 + w, qi = t * kTile + r;
      const bool row_in = qi < U.len;      // rows behind the document take no part in the warp's choices
      const int lo = p.win.left < 0 ? 0 : max(0, qi - p.win.left);
      const int hi = p.win.right < 0 ? U.len - 1 : min(U.len - 1, qi + p.win.right);
      const FullTiles full = full_tiles(t, U.len, U.pre, p.win);
      const float steep = HB.slope2 * (float)(kTile - 1);
      float m = -INFINITY;
      float2 la = make_float2(0.f, 0.f), lb = la;
      bool first = true;
      for (int k = 0; k < nk; ++k) {
        if (k == skip) continue;
        const int u = U.kt.tile(k);
        TileBias B{};
        if constexpr (BIAS) B = tile_bias(tab, HB, R, near, t, u, u * kTile - qi);
        const bool seen = full.has(u);
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[w], ns & 1, status));
        if (!ok) break;
        tc_fence_after();
        uint32_t v[4][32];
        float cm[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if constexpr (CAP) tmem_ld32_absmax(s_addr + 32 * g, v[g], cm[g]);
          else tmem_ld32_max(s_addr + 32 * g, v[g], cm[g]);
        }
        tmem_ld_wait();
        if (kSplit) {
          tc_fence_before();
          mbar_arrive(&s_free[w]);
        }
        float mx = fmaxf(fmax3(cm[0], cm[1], cm[2]), cm[3]);      // of the raw products, or of their magnitudes
        // form 0: v f + n; 1, 2: capped by 3 or 5 coefficients, then as 0; 3: v f + n + slope column
        int form = 0;
        bool quick = seen && (!BIAS || !B.tab);
        if constexpr (CAP) {
          quick = quick && B.col == 0.f && !__any_sync(0xffffffffu, row_in && !(mx <= p.capf.t5 && mx * scale2 <= kLoose * 0.5f));
          form = __any_sync(0xffffffffu, row_in && !(mx <= p.capf.t3)) ? 2 : 1;
        } else if constexpr (BIAS) {
          quick = quick && fabsf(steep) <= kLoose;
          form = 3;
        }
        if (!quick) {
          form = 0;
          uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
          if (!seen) {
            const int c = u * kTile;
#pragma unroll
            for (int g = 0; g < 4; ++g) see[g] = column_mask(lo - c, hi - c, U.pre - c, 32 * g);
          }
          if constexpr (CAP) {
            if (!seen) {
#pragma unroll
              for (int g = 0; g < 4; ++g) hide(v[g], see[g], 0u);
            }
            cap_products(v, p.capf, row_in);
          }
          if constexpr (BIAS) {
#pragma unroll
            for (int g = 0; g < 4; ++g) bias_chunk<1>(v[g], 32 * g, scale2, B);
          }
          if (!seen) {
#pragma unroll
            for (int g = 0; g < 4; ++g) hide(v[g], see[g], kMinusInf);
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) cm[g] = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; j += 2)
#pragma unroll
            for (int g = 0; g < 4; ++g) cm[g] = fmax3(cm[g], __uint_as_float(v[g][j]), __uint_as_float(v[g][j + 1]));
          mx = fmaxf(fmax3(cm[0], cm[1], cm[2]), cm[3]);
        }
        const float f = BIAS ? B.factor(scale2) : scale2;
        mx = fmaf(mx, f, B.c);
        if (BIAS && quick) mx += fmaxf(u < t ? steep : -steep, 0.f);
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
        if ((u + 1) * kTile > U.len) {
          const uint32_t x = ring + 2 * k + 1, st = x % kSlots;
          ok = __all_sync(0xffffffffu, mbar_wait(&kv_full[st], (x / kSlots) & 1, status));
          if (!ok) break;
          if (u * kTile + r >= U.len) clear_row<D>(smem + L::kKV + st * L::kTileBytes, r);
          fence_proxy_async_smem();
          __syncwarp();              // P is stored by the whole warp
        }
        const float shrink = shrink_for(m);
        const float neg = ((m == -INFINITY ? 0.f : -m) + B.c) * shrink, fs = fmaxf(f * shrink, 0x1p-126f);   // (0 * -inf)
        // P in two halves of 64 keys: the first one's product starts while the second is computed
        auto exps = [&](auto FORM) {
          constexpr int kForm = decltype(FORM)::value;
          const float2 f2 = make_float2(fs, fs), n2 = make_float2(neg, neg);
          const float s2 = B.col * fs;
          const CapForm& F = p.capf;
          auto arg = [&](int g, int c) {
            const float2 x = pair_of(v[g], c);
            if constexpr (kForm == 1 || kForm == 2) {       // x (scale2 + scale2 t(x^2)) + n
              const float2 q = fmul2(x, x);
              float2 y;
              if constexpr (kForm == 1) {
                y = ffma2(q, F.e3[3], F.e3[2]);
                y = ffma2(q, y, F.e3[1]);
                y = ffma2(q, y, F.e3[0]);
              } else {
                y = ffma2(q, F.e5[5], F.e5[4]);
                y = ffma2(q, y, F.e5[3]);
                y = ffma2(q, y, F.e5[2]);
                y = ffma2(q, y, F.e5[1]);
                y = ffma2(q, y, F.e5[0]);
              }
              return ffma2(x, y, n2);
            } else if constexpr (kForm == 3) {
              const float j = (float)(32 * g + c);
              return ffma2(x, f2, make_float2(fmaf(s2, j, neg), fmaf(s2, j + 1.f, neg)));
            } else {
              return ffma2(x, f2, n2);
            }
          };
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
#pragma unroll
            for (int j = 0; j < 64; j += 4) {
              const int g = 2 * half + j / 32, c = j % 32;
              float2 e0 = arg(g, c), e1 = arg(g, c + 2);
              e0 = make_float2(fast_exp2(e0.x), fast_exp2(e0.y));
              e1 = make_float2(fast_exp2(e1.x), fast_exp2(e1.y));
              la = fadd2(la, e0);
              lb = fadd2(lb, e1);
              const __nv_bfloat162 b0 = __floats2bfloat162_rn(e0.x, e0.y), b1 = __floats2bfloat162_rn(e1.x, e1.y);
              pk[j / 2] = *reinterpret_cast<const uint32_t*>(&b0);
              pk[j / 2 + 1] = *reinterpret_cast<const uint32_t*>(&b1);
            }
            if (kSplit && half == 0 && ns) {       // the last P has been read
              ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[w], (ns - 1) & 1, status));
              if (!ok) return;
              tc_fence_after();
            }
            tmem_st32(p_addr + 32 * half, pk);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&p_full[2 * w + half]);
          }
        };
        if constexpr (CAP) {
          if (form == 1) exps(std::integral_constant<int, 1>{});
          else if (form == 2) exps(std::integral_constant<int, 2>{});
          else exps(std::integral_constant<int, 0>{});
        } else if constexpr (BIAS) {
          if (form == 3 && B.col != 0.f) exps(std::integral_constant<int, 3>{});
          else exps(std::integral_constant<int, 0>{});
        } else {
          exps(std::integral_constant<int, 0>{});
        }
        if (!ok) break;
        ++ns;
        first = false;
      }
      ring += 2 * nk;
      if (!ok) break;
      // the last unit's 1 / l has been used
      if (nu && !(ok = __all_sync(0xffffffffu, mbar_wait(&o_free[w], (nu - 1) & 1, status)))) break;
      ++nu;
      const float l = (la.x + la.y) + (lb.x + lb.y);
      inv_l[r] = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);     // a row that sees nothing: O = 0
      mbar_arrive(&l_ready[w]);
      if (qi < U.len) p.lse[(int64_t)U.h * p.T + U.start + qi] = l == 0.f ? INFINITY : (m + __log2f(l)) * kLn2;
    }
  } else {
    // ------------------------------------------------------------ bias tables, O
    setmaxnreg_dec<kRegAux>();
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = tbase + ((uint32_t)(quarter * 32) << 16);
    float* tab = reinterpret_cast<float*>(smem + L::kBias);
    const bool al32 = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    uint32_t nu[2] = {0, 0};
    bool ok = true;
    Unit U = read_unit(units, unit_full, 0, true, ok, status);
    if (BIAS && U.ntq) {
      stage_bias(tab, p, U.h, r, 128);
      mbar_arrive(&tab_full[0]);
    }
    for (int n = 0; ok && U.ntq; ++n) {
      const int h = U.h, t0 = U.t0, ntq = U.ntq, start = U.start, len = U.len, index = U.index;
      U = read_unit(units, unit_full, n + 1, true, ok, status);
      if (BIAS && U.ntq) {            // into the table of the last unit but one, whose O is out and which all have read
        if (n && !(ok = __all_sync(0xffffffffu, mbar_wait(&unit_done[(n - 1) % kUnits], ((n - 1) / kUnits) & 1, status)))) break;
        stage_bias(tab + ((n + 1) & 1) * kBiasTab, p, U.h, r, 128);
        mbar_arrive(&tab_full[(n + 1) & 1]);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (w >= ntq || !ok) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(&l_ready[w], nu[w] & 1, status) && mbar_wait(&o_full[w], nu[w] & 1, status));
        if (!ok) continue;
        ++nu[w];
        tc_fence_after();
        const float inv = reinterpret_cast<const float*>(smem + L::kInv)[w * 128 + r];
        const int qi = (t0 + w) * kTile + r;
        __nv_bfloat16* orow = p.out + (((int64_t)start + qi) * p.hq + h) * D;
#pragma unroll 2
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          __syncwarp();              // (the rows of the document alone have stored the last columns)
          tmem_ld32(lane_base + kO + w * D + 32 * c, o);
          tmem_ld_wait();
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 b2 =
                __floats2bfloat162_rn(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
            pk[j] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          if (c == D / 32 - 1) {
            tc_fence_before();
            mbar_arrive(&o_free[w]);
          }
          if (qi < len) {
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
      }
      if (r == 0 && ok) mbar_arrive(&unit_done[n % kUnits]);
      clear_tail(index, n_units, r, 128);
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
  constexpr int smem = FwdSmem<D>::kAlloc;
  static_assert(smem <= 232448, "shared memory of one CTA");
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = prepare_kernel<scored_fwd_kernel<D, CAP, BIAS>>(smem, &regs);
  if (e != cudaSuccess) return e;
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;    // the register split relies on it
  const int64_t units = ((int64_t)p.T / (kTile * kItemTiles) + p.N + 1) * p.hq;
  if (units > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const bool take = units < (int64_t)kTakeBelow * sms;
  scored_fwd_kernel<D, CAP, BIAS>
      <<<(unsigned)(take || units < sms ? units : sms), kThreads, smem, stream>>>(tq, tk, tv, p, take);
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
