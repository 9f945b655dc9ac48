// Scored attention, backward, on bf16 tcgen05 MMAs with TMEM accumulators.
//
//   P = 2^(u log2 e - LSE log2 e), dU = P o (dO V^T - D), dS = dU o (1 - tanh^2),
//   dV = P^T dO, dK = scale dS^T Q, dQ = scale dS K, drel[h][r] = sum of dU at distance r.
//
// D = rowsum(dO o O) (memory-bound), then dK and dV per key tile (with few units per query
// head, whose parts are then added), then dQ per query tile, then drel.  P and dS are
// computed for dK and dV and again for dQ: 7 tile products a pair of tiles instead of the 5
// of a single pass.  A single pass has to add its dQ partials into memory from every key
// tile: an fp32 tile (64 KB) per step through shared memory and L2, in an order that changes
// from run to run, and needs dS^T once more as a shared-memory operand.  Here dS and P are A
// operands straight from tensor memory, and the results are the same bits every time.
//
// P and dS enter their products in bf16 (their partners are bf16): half a step of 2^-8 per
// element, as the rounding of the gradients themselves; sums stay in fp32.
#include <algorithm>
#include <type_traits>

#include "ptx.cuh"
#include "scored.cuh"
#include "tmap.h"

namespace flamia {

namespace {

constexpr int kCompute = 512;    // compute threads: four warpgroups, each 32 of a tile's 128 columns
constexpr int kThreads = 128 + kCompute;
constexpr int kLaunchRegs = (65536 / kThreads) & ~7;
constexpr int kRegCtl = 64, kRegCompute = 104;
static_assert(kRegCtl * 128 + kRegCompute * kCompute <= kLaunchRegs * kThreads, "register split");

// A row's LSE as the backward takes it.  P = exp(u - LSE) has the roundings of LSE and of u for its relative error;
// from 2^23 on, where a step of LSE is 1, nothing of P is left (and far beyond, 2^x overflows): such a row gives
// no gradient, as one that sees nothing.
__device__ __forceinline__ float usable_lse(float l) { return fabsf(l) >= 0x1p23f ? INFINITY : l; }

// One arrival for a warp, behind what all its lanes did.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ---------------------------------------------------------------- D = rowsum(dO o O)
// D/8 threads a row, one 16-byte load of each operand per thread; rows outside every
// document get zero gradients.
template <int D>
__global__ void __launch_bounds__(256) scored_prep_kernel(const ScoredParams p) {
  constexpr int kPer = D / 8, kRows = 256 / kPer;
  grid_let_next();
  const int sub = threadIdx.x % kPer;
  const int64_t nb = (p.T + kRows - 1) / kRows;
  const int h = (int)(blockIdx.x / nb);
  const int64_t t = (blockIdx.x % nb) * kRows + threadIdx.x / kPer;
  const bool in = t < p.T;
  float s = 0.f;
  if (in) {
    const int64_t at = (t * p.hq + h) * D + sub * 8;
    if (t < p.plan[kPlanValid]) {
      const uint4 a = *reinterpret_cast<const uint4*>(p.out + at), b = *reinterpret_cast<const uint4*>(p.dout + at);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(aw[i] << 16), __uint_as_float(bw[i] << 16), s);
        s = fmaf(__uint_as_float(aw[i] & 0xffff0000u), __uint_as_float(bw[i] & 0xffff0000u), s);
      }
    } else {
      const uint4 z = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(p.dq + at) = z;
      if (h < p.hkv) {
        const int64_t kt = (t * p.hkv + h) * D + sub * 8;
        *reinterpret_cast<uint4*>(p.dk + kt) = z;
        *reinterpret_cast<uint4*>(p.dv + kt) = z;
      }
    }
  }
#pragma unroll
  for (int o = kPer / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (in && sub == 0) p.dvec[(int64_t)h * p.T + t] = s;
}

// a + (the part that a's last digits lost) += x.
__device__ __forceinline__ void add_comp(float& a, float& lost, float x) {
  const float s = __fadd_rn(a, x), b = __fsub_rn(s, a);
  lost = __fadd_rn(lost, __fadd_rn(__fsub_rn(a, __fsub_rn(s, b)), __fsub_rn(x, b)));
  a = s;
}
__device__ __forceinline__ uint32_t pack2(float2 x) {
  const __nv_bfloat162 b2 = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t*>(&b2);
}
// One row of fp32 accumulators (columns c0 ..) -> bf16 in global memory, times f.  A warp's rows
// lie apart, so a store moves a sector of 32 bytes per lane where the rows allow it (wide): half as
// many as with 16 bytes, and the store path is what this waits for.  Where a document ends inside the
// warp only some lanes store; the loads from tensor memory are the whole warp's, so it meets before the next.
template <int COLS>
__device__ __forceinline__ void store_acc(uint32_t taddr, __nv_bfloat16* dst, float f, bool valid, bool wide) {
#pragma unroll 1
  for (int c = 0; c < COLS / 32; ++c) {
    uint32_t o[32];
    if (c) __syncwarp();
    tmem_ld32(taddr + 32 * c, o);
    tmem_ld_wait();
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = pack2(make_float2(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f));
    if (!valid) continue;
    if (wide) {
      st_global_v8(dst + 32 * c, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
      st_global_v8(dst + 32 * c + 16, w[8], w[9], w[10], w[11], w[12], w[13], w[14], w[15]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4*>(dst + 32 * c + 8 * q) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    }
  }
}
// The same in fp32.
template <int COLS>
__device__ __forceinline__ void store_part(uint32_t taddr, float* dst, bool valid) {
#pragma unroll 1
  for (int c = 0; c < COLS / 32; ++c) {
    uint32_t o[32];
    if (c) __syncwarp();
    tmem_ld32(taddr + 32 * c, o);
    tmem_ld_wait();
    if (valid) {                 // (the workspace's rows are whole sectors)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        st_global_v8(dst + 32 * c + 8 * q, o[8 * q], o[8 * q + 1], o[8 * q + 2], o[8 * q + 3], o[8 * q + 4], o[8 * q + 5],
                     o[8 * q + 6], o[8 * q + 7]);
    }
  }
}
// dP where P is not 0: rows of another document, or of nobody, may hold anything, and weight
// 0 does not silence an infinity.  (In its own branch: selects in the loops over every tile run
// on all of them, two operations an element.)
__device__ __forceinline__ void drop_hidden(uint32_t (&dp)[32], const uint32_t (&pr)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (__uint_as_float(pr[j]) == 0.f) dp[j] = 0u;
}
// 1 - tanh^2 from the capped product y = tanh / zscale.
__device__ __forceinline__ float2 cap_slope(float2 y, float zscale) {
  const float2 t = fmul2(y, make_float2(zscale, zscale));
  return ffma2(t, make_float2(-t.x, -t.y), make_float2(1.f, 1.f));
}

// x as the sum of three bf16 (24 bits, all of it), infinities as the largest that a bf16 holds.
__device__ __forceinline__ void split3(float x, uint32_t (&part)[3]) {
  if (fabsf(x) > 3e38f) x = copysignf(3e38f, x);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const __nv_bfloat16 b = __float2bfloat16_rn(x);
    part[i] = __bfloat16_as_ushort(b);
    x -= __bfloat162float(b);
  }
}

template <int D, int ROWS = kTile>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, int h, int row) {
  mbar_arrive_expect_tx(bar, ROWS * D * 2);
#pragma unroll
  for (int b = 0; b < D / 64; ++b) tma_load_3d(dst + b * ROWS * 128, tm, bar, 64 * b, h, row);
}

// ================================================================ dK, dV
// One CTA per SM walks (key tile, kv head) units (or query head: scored_bwd_split); a step is a
// query tile of one of the unit's query heads.  S^T = K Q^T and dP^T = V dO^T have keys in the
// TMEM lanes, so P^T and dS^T are written back over their own columns and are the A operands
// of dV += P^T dO and dK += dS^T Q.  A warp issues the chain of S^T and dV, another that of
// dP^T and dK, so that neither waits for the other's operands; nothing that one has waited for
// stands before the other's products.  K is free for the next unit once the unit's last S^T is
// done, V once its last dP^T is.
//
// LSE and D vary along a thread's columns, so every warp would read both of every query from
// shared memory: 4 quarters of keys x 128 queries x 2, at the one value a cycle that a broadcast
// delivers, beside what the products read there.  The two together kept that path 99% busy at
// D = 64.  (kFold) They go through the products instead: a last step of 16 multiplies rows of
// eight bf16 per query (-LSE / scale2 in three parts, which hold all of its 24 bits, -D in three)
// with ones, and the accumulators come out as S^T - LSE / scale2 and dP^T - D.  With a cap LSE
// comes after the cap, and stays in shared memory.
//
// D = 64 leaves room for a second S^T (kSBuf): the next one runs while this P^T is computed.
// Two noncausal documents of 8192, 16 heads, buckets, all three launches: 2.25 ms with one S^T, 2.11
// with two.
//
// At D = 128 tensor memory is full, and a step's queries go in two halves, each with its own
// 64-query tiles, products and warps, half a step apart: while one half's P^T is computed the
// other's dS^T is.  (Whole and folded, all warps wait for the same product: 6.03 instead of 5.86
// ms on four documents of 8192, 32 heads on 8, slopes.)  A product with 64 columns reads more
// shared memory than it multiplies (48 cycles instead of 32 a step of 16), and the fold would
// cost two more of them for nothing (3% more).  Where drel is wanted the warps meet at barriers on
// every tile near the diagonal anyway: whole and folded, 6% less (packed documents, 16384 rows,
// 16 heads).  (The last two were measured before dV waited for its dO.)
// Roles: warp 0 TMA, warps 1 and 2 MMA (2 also TMEM), warp 3 stages LSE and D of a step's queries,
// warps 4-19 compute: thread = key row, warpgroup = 32 of the 128 query columns.
// TMEM columns: dV [0, D), dK [D, 2 D), S^T [256, 384) (D = 64: [128, 384)), dP^T [384, 512).
template <int D, int BIAS>
struct DkvSmem {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kK = 0, kV = kTileBytes;
  static constexpr int kHalves = D == 128 && BIAS != 2 ? 2 : 1;
  static constexpr bool kFold = kHalves == 1;
  static constexpr int kStats = kFold ? 2 : 4;                 // steps whose LSE and D are staged
  static constexpr int kRows = kTile / kHalves;
  static constexpr int kStages = D == 128 ? 2 : 3;
  static constexpr int kSBuf = D == 64 ? 2 : 1;                // places of S^T
  static constexpr int kPartBytes = kTileBytes / kHalves;
  static constexpr int kQ = 2 * kTileBytes;                    // [halves][stages]
  static constexpr int kDO = kQ + kStages * kTileBytes;        // [halves][stages]
  static __device__ __forceinline__ int part_at(int half, uint32_t g) { return (half * kStages + (int)(g % kStages)) * kPartBytes; }
  // (kFold) [kStats][128 queries][8]: their LSE and D
  static constexpr int kRow = kDO + kStages * kTileBytes;
  static constexpr int kPick = kRow + (kFold ? kStats * 2048 : 0);   // [128 keys][8]: 1 where LSE is, then the same for D
  static constexpr int kZero = kPick + (kFold ? 4096 : 0);
  static constexpr int kLse = kZero + (kFold ? 2048 : 0);      // [kStats][128 -LSE log2 e, (not kFold) 128 D]
  static constexpr int kStat = kFold ? 128 : 256;
  static constexpr int kBias = kLse + kStats * kStat * 4;            // [kBiasTab]
  static constexpr int kAcc = kBias + kBiasTab * 4;      // [2 R + 1] drel of the current head
  static constexpr int kDiag = kAcc + (2 * FLAMIA_REL_MAX + 2) * 4;   // [16 warps][64]
  static constexpr int kBar = (kDiag + 16 * 64 * 4 + 15) & ~15;
  static constexpr int kBytes = kBar + 512;
  static constexpr int kAlloc = kBytes + 1024;
};

struct KeyUnit {
  int item, h0, hk, u, start, len, nt, pre, tlo, nq;      // h0: the unit's first query head
  int2 full;                // query tiles that see the key tile whole
};
// What a unit's first loads bring; fetched a unit ahead, so that their latency is not met.
struct RawUnit {
  int i;
  int4 item;
  int2 span;
};
// Units per key tile, and query heads per unit.
__device__ __forceinline__ int unit_heads(const ScoredParams& p) { return p.dk_part ? p.hq : p.hkv; }
__device__ __forceinline__ KeyUnit key_unit(const ScoredParams& p, const RawUnit& raw) {
  KeyUnit U;
  U.item = raw.i / unit_heads(p);
  U.h0 = raw.i % unit_heads(p) * (p.hq / unit_heads(p));
  U.hk = U.h0 / (p.hq / p.hkv);
  const int4 item = raw.item;
  const int2 span = raw.span;
  U.u = item.y;
  U.start = span.x;
  U.len = span.y;
  U.nt = (U.len + kTile - 1) / kTile;
  U.pre = prefix_of(p, item.x, U.len);
  U.full = full_queries(U.u, U.len, U.pre, p.win);
  const bool all = U.u * kTile < U.pre;        // every query of the document sees a prefix key
  U.tlo = all ? 0 : win_tlo(U.u, p.win);
  U.nq = (all ? U.nt - 1 : win_thi(U.u, U.nt, p.win)) - U.tlo + 1;
  return U;
}

// The steps of this CTA, unit after unit.
struct KeySteps {
  int n, n_units, group;
  KeyUnit U;
  RawUnit raw;              // the next unit's
  int h, t;                 // the step's query head and query tile
  __device__ __forceinline__ void fetch(const ScoredParams& p, const PlanView& pv, int k) {
    raw.i = unit_index(k, n_units);
    if (raw.i < 0) return;
    raw.item = pv.bwd_items[raw.i / unit_heads(p)];
    raw.span = pv.bwd_span[raw.i / unit_heads(p)];
  }
  __device__ __forceinline__ bool unit(const ScoredParams& p, const PlanView& pv) {
    if (raw.i < 0) return false;
    U = key_unit(p, raw);
    fetch(p, pv, n + 1);
    h = U.h0;
    t = U.tlo;
    return true;
  }
  __device__ __forceinline__ bool begin(const ScoredParams& p, const PlanView& pv) {
    n = 0;
    n_units = p.plan[kPlanBwdItems] * unit_heads(p);
    group = p.hq / unit_heads(p);
    fetch(p, pv, 0);
    return unit(p, pv);
  }
  __device__ __forceinline__ bool head_first() const { return t == U.tlo; }
  __device__ __forceinline__ bool head_last() const { return t == U.tlo + U.nq - 1; }
  __device__ __forceinline__ bool first() const { return h == U.h0 && head_first(); }
  __device__ __forceinline__ bool last() const { return h == U.h0 + group - 1 && head_last(); }
  __device__ __forceinline__ bool next(const ScoredParams& p, const PlanView& pv) {
    if (last()) {
      ++n;
      return unit(p, pv);
    }
    if (head_last()) {
      ++h;
      t = U.tlo;
    } else {
      ++t;
    }
    return true;
  }
};

// BIAS: 0 none, 1 a bias, 2 a bias whose gradient is wanted.
template <int D, bool CAP, int BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    scored_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                      const ScoredParams p) {
  using L = DkvSmem<D, BIAS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t *k_full = bars, *k_empty = bars + 1, *v_full = bars + 2, *v_empty = bars + 3;
  constexpr int kHalves = L::kHalves, kStages = L::kStages, kSBuf = L::kSBuf, kRows = L::kRows, kStats = L::kStats;
  constexpr bool kFold = L::kFold, kReadStat = CAP || !kFold;
  uint64_t *q_full = bars + 4, *q_empty = bars + 10, *do_full = bars + 16, *do_empty = bars + 22;   // [halves][stages]
  uint64_t *s_full = bars + 28, *dp_full = bars + 30, *p_ready = bars + 32, *ds_ready = bars + 34;  // [halves or buffers]
  uint64_t *acc_full = bars + 36, *acc_free = bars + 37, *drain = bars + 38;                       // drain [2]
  uint64_t *st_full = bars + 40, *st_empty = st_full + kStats;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(st_empty + kStats);
  int* status = const_cast<int*>(p.plan) + kPlanStatus;
  const PlanView pv = plan_view(p.plan, p.T, p.N);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 32; ++i) mbar_init(bars + i, 1);
    for (int i = 32; i < 36; ++i) mbar_init(bars + i, kCompute / 32 / kHalves);
    mbar_init(acc_full, 2);
    mbar_init(acc_free, kCompute);
    mbar_init(drain, 1);
    mbar_init(drain + 1, 1);
    for (int i = 0; i < kStats; ++i) {
      mbar_init(&st_full[i], 1);
      mbar_init(&st_empty[i], (kReadStat ? kCompute / 32 : 0) + (kFold ? (CAP ? 1 : 2) : 0));
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_do);
  }
  if (kFold && threadIdx.x < 384) {        // the ones that pick a row's LSE or D, and the zeros
    const uint32_t one = 0x3F80u;
    const int which = threadIdx.x >> 7;
    *reinterpret_cast<uint4*>(smem + L::kPick + threadIdx.x * 16) =
        which == 0 ? make_uint4(one | one << 16, one, 0, 0)
                   : which == 1 ? make_uint4(0, one << 16, one | one << 16, 0) : make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  if (warp == 2) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  constexpr uint32_t kTV = 0, kTK = D, kTS = kSBuf == 2 ? 128 : 256, kTP = 384;
  // S^T and P^T alternate between kSBuf places, with barriers of their own
  auto s_at = [&](int half, uint32_t g) { return kSBuf == 2 ? (int)(g & 1) : half; };
  auto s_phase = [&](uint32_t g) { return (kSBuf == 2 ? g >> 1 : g) & 1; };

  if (warp < 4) {
    setmaxnreg_dec<kRegCtl>();
    KeySteps S{};
    bool more = S.begin(p, pv), ok = true;
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      uint32_t nk = 0, nv = 0, nq = 0, nd = 0;       // tiles and parts of tiles loaded
      for (; more && ok; more = S.next(p, pv)) {
        const int krow = S.U.start + S.U.u * kTile;
        if (S.first()) {
          if (nk && !(ok = mbar_wait(k_empty, (nk - 1) & 1, status))) break;
          load_tile<D>(smem + L::kK, &tm_k, k_full, S.U.hk, krow);
          ++nk;
        }
#pragma unroll 1
        for (int half = 0; half < kHalves && ok; ++half) {
          const int row = S.U.start + S.t * kTile + kRows * half;
          const uint32_t g = nq / kHalves, b = half * kStages + g % kStages, ph = (g / kStages - 1) & 1;
          if (g >= kStages && !(ok = mbar_wait(&q_empty[b], ph, status))) break;
          load_tile<D, kRows>(smem + L::kQ + L::part_at(half, g), &tm_q, &q_full[b], S.h, row);
          ++nq;
          if (half == 0 && S.first()) {
            if (nv && !(ok = mbar_wait(v_empty, (nv - 1) & 1, status))) break;
            load_tile<D>(smem + L::kV, &tm_v, v_full, S.U.hk, krow);
            ++nv;
          }
          // dV has read the tile, and dP too: dK, which gave Q's stage back above, came after it
          if (g >= kStages && !(ok = mbar_wait(&do_empty[b], ph, status))) break;
          load_tile<D, kRows>(smem + L::kDO + L::part_at(half, g), &tm_do, &do_full[b], S.h, row);
          ++nd;
        }
      }
      // nothing may land after the CTA has left (open only when a wait ran out)
      if (nk) mbar_wait(k_full, (nk - 1) & 1, status);
      if (nv) mbar_wait(v_full, (nv - 1) & 1, status);
      auto landed = [&](uint64_t* full, uint32_t n) {
        for (uint32_t x = n > kHalves * kStages ? n - kHalves * kStages : 0; x < n; ++x)
          mbar_wait(&full[x % kHalves * kStages + x / kHalves % kStages], (x / kHalves / kStages) & 1, status);
      };
      landed(q_full, nq);
      landed(do_full, nd);
    } else if (warp == 1 || warp == 2) {
      // ---------------------------------------------------------- MMA issuers
      // warp 1: S^T and dV, warp 2: dP^T and dK; each half's next scores go out behind the product
      // that read what they overwrite
      const bool leader = elect_one();
      const uint32_t base16 = (smem_u32(smem) & 0x3FFFFu) >> 4;
      auto run = [&](auto WHICH) {
        constexpr bool kP = decltype(WHICH)::value;      // the chain of P
        constexpr uint32_t kA = kP ? L::kK : L::kV, kB = kP ? L::kQ : L::kDO, kB2 = kP ? L::kDO : L::kQ;
        constexpr uint32_t kT = kP ? kTS : kTP, kSum = kP ? kTV : kTK;
        uint64_t *a_full = kP ? k_full : v_full, *a_empty = kP ? k_empty : v_empty;
        uint64_t *b_full = kP ? q_full : do_full, *b2_empty = kP ? do_empty : q_empty;
        uint64_t *out = kP ? s_full : dp_full, *in = kP ? p_ready : ds_ready;
        // of step g, both operands K-major.  A (K or V): a_full at the unit's first step; B (Q or dO): b_full
        auto scores = [&](int half, uint32_t g, int unit, bool first, bool last) {
          const uint32_t b = half * kStages + g % kStages, b16 = base16 + g % kStages * (L::kPartBytes / 16);
          const uint32_t sum = tbase + kT + (kP && kSBuf == 2 ? 128 * (g & 1) : kRows * half);
          if (half == 0 && first && !(ok = warp_wait(a_full, unit & 1, status))) return;
          if (!(ok = warp_wait(&b_full[b], (g / kStages) & 1, status))) return;
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            if (leader)
              mma_bf16(sum, sdesc_at(base16, kA + (s / 4) * kTile * 128 + (s % 4) * 32, 16, 1024, kSwizzle128B),
                       sdesc_at(b16, kB + half * kStages * L::kPartBytes + (s / 4) * kRows * 128 + (s % 4) * 32, 16, 1024, kSwizzle128B),
                       idesc_bf16(128, kRows, 0, 0), s > 0);
          if constexpr (kFold && (!kP || !CAP)) {        // less the query's LSE or D
            const uint32_t row = L::kRow + half * kRows * 16, st = g % kStats;
            if (half == 0 && !(ok = warp_wait(&st_full[st], (g / kStats) & 1, status))) return;
            constexpr uint32_t pick = kP ? L::kPick : L::kPick + 2048;
            if (leader) {
              mma_bf16(sum, sdesc_at(base16, pick, L::kZero - pick, 128, kSwizzleNone),
                       sdesc_at(base16 + st * 128, row, kStats * 2048, 128, kSwizzleNone), idesc_bf16(128, kRows, 0, 0), 1);
              if (half == kHalves - 1) mma_commit(&st_empty[st]);
            }
          }
          if (leader) {
            mma_commit(&out[kP ? s_at(half, g) : half]);
            if (half == kHalves - 1 && last) mma_commit(a_empty);
          }
          if (kP && kFold) ok = warp_wait(&do_full[b], (g / kStages) & 1, status);      // for this step's dV
        };
        // A from TMEM (P^T or dS^T): in; B over its rows: dK's Q by `in` too, as dS^T came from an S^T that had
        // read it.  dV's dO not, as P^T needs Q and K alone and the producer asks for dO last: by a wait of its own,
        // which takes 100 cycles of whoever makes it.  Not folded, the warp that stages D makes it, and `in` covers
        // dO with D: 5990 us on four documents of 8192, 32 heads on 8, slopes, 6060 to 6130 with the wait behind the
        // scores above, 6100 here.  Folded, S^T itself would wait for dO (2257 us on the noncausal case): the
        // wait is behind the scores, 2230
        auto product = [&](int half, uint32_t g, bool first) {
          if (!(ok = warp_wait(&in[kP ? s_at(half, g) : half], kP ? s_phase(g) : g & 1, status))) return;
          tc_fence_after();
          const uint32_t b16 = base16 + g % kStages * (L::kPartBytes / 16);
          const uint32_t a = tbase + kT + (kP && kSBuf == 2 ? 128 * (g & 1) : kRows * half);
#pragma unroll
          for (int s = 0; s < kRows / 16; ++s)
            if (leader)
              mma_bf16_ta(tbase + kSum, a + 32 * (s >> 1) + 8 * (s & 1),
                          sdesc_at(b16, kB2 + half * kStages * L::kPartBytes + s * 2048, kRows * 128, 1024, kSwizzle128B),
                          idesc_bf16(128, D, 0, 1), (!(first && half == 0) || s > 0));
          if (leader) mma_commit(&b2_empty[half * kStages + g % kStages]);
        };
        int steps = more ? S.group * S.U.nq : 0;      // of the unit
        if (steps) {
          scores(0, 0, 0, true, steps == 1);
          if (kHalves == 2 && ok) scores(1, 0, 0, true, steps == 1);
        }
        uint32_t g = 0;
        for (int unit = 0; steps && ok; ++unit) {
          ++S.n;
          const int next_steps = S.unit(p, pv) ? S.group * S.U.nq : 0;
          for (int i = 0; i < steps && ok; ++i, ++g) {
            const bool last = i == steps - 1, next = !last || next_steps;
            const bool next_last = last ? next_steps == 1 : i + 2 == steps;
            // with a second place for them the next scores need not wait for this P
            const bool ahead = kP && kSBuf == 2 && !last;
            if (ahead) scores(0, g + 1, unit, false, next_last);
            // the unit's first product overwrites the sums of the last one: those have to be out
            if (ok && i == 0 && unit) ok = warp_wait(acc_free, (unit - 1) & 1, status);
#pragma unroll
            for (int half = 0; half < kHalves; ++half) {
              if (ok) product(half, g, i == 0);
              if (ok && next && !ahead) scores(half, g + 1, unit + last, last, next_last);
            }
            if (ok && last && leader) mma_commit(acc_full);
          }
          steps = next_steps;
        }
      };
      if (warp == 1) run(std::true_type{});
      else run(std::false_type{});
      if (leader) {
        mma_commit(&drain[warp - 1]);
        mbar_wait(&drain[warp - 1], 0, status);
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------- LSE and D of a step's queries
      // as rows of eight bf16: minus LSE in three parts, minus D in three, 0, 0
      const float to_products = -kLog2e / p.scale2;
      grid_wait();               // D is there: nothing else here reads what the launch before wrote
      grid_let_next();           // nor does dQ read what this one writes
      for (uint32_t g = 0; more && ok; more = S.next(p, pv), ++g) {
        const int b = g % kStats;
        float l[4], d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int q = S.t * kTile + 32 * e + lane;
          const int64_t at = (int64_t)S.h * p.T + S.U.start + q;
          l[e] = q < S.U.len ? usable_lse(p.lse[at]) : INFINITY;
          d[e] = q < S.U.len ? p.dvec[at] : 0.f;
        }
        if (g >= kStats && !(ok = warp_wait(&st_empty[b], (g / kStats - 1) & 1, status))) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float* stat = reinterpret_cast<float*>(smem + L::kLse) + b * L::kStat + 32 * e + lane;
          if (kReadStat) stat[0] = -l[e] * kLog2e;
          if constexpr (!kFold) {
            stat[128] = d[e];
            continue;
          }
          uint32_t x[3] = {0, 0, 0}, y[3];
          if (!CAP) split3(l[e] * to_products, x);
          split3(-d[e], y);
          *reinterpret_cast<uint4*>(smem + L::kRow + b * 2048 + (32 * e + lane) * 16) =
              make_uint4(x[0] | x[1] << 16, x[2] | y[0] << 16, y[1] | y[2] << 16, 0);
        }
        if (kFold) fence_proxy_async_smem();
        if (!kFold) {            // for this step's dV: no P^T is computed without D
#pragma unroll
          for (int half = 0; half < kHalves; ++half)
            if (ok) ok = warp_wait(&do_full[half * kStages + g % kStages], (g / kStages) & 1, status);
          if (!ok) break;
        }
        warp_arrive(&st_full[b]);
      }
    }
  } else {
    // ------------------------------------------------------------ compute
    setmaxnreg_inc<kRegCompute>();
    const int w = (warp - 4) >> 2, quarter = warp & 3, half = kHalves == 2 ? w >> 1 : 0;
    const int r = quarter * 32 + lane, tid = threadIdx.x - 128;
    const uint32_t lane_base = tbase + ((uint32_t)(quarter * 32) << 16);
    const uint32_t dp_addr = lane_base + kTP + 32 * w;
    float* tab = reinterpret_cast<float*>(smem + L::kBias);
    float* acc = reinterpret_cast<float*>(smem + L::kAcc);
    const int R = bias_range(p);
    const int near = near_tiles(R);
    const float scale2 = p.scale2;
    HeadBias HB{};
    int staged = -1;
    float far_lo = 0.f, far_hi = 0.f, lost_lo = 0.f, lost_hi = 0.f;
    bool ok = true;
    KeySteps S{};
    // a warp whose wait ran out goes on through the steps without work: it still meets the others
    // at the barriers
    uint32_t g = 0;
    for (bool more = S.begin(p, pv); more; ++S.n, more = S.unit(p, pv)) {
     const KeyUnit U = S.U;
     const int kj = U.u * kTile + r;
     int lo0 = 0, hi0 = U.len - 1;              // queries that see the key
     if (kj >= U.len) {
       hi0 = -1;
     } else if (kj >= U.pre) {
       if (p.win.right >= 0) lo0 = kj - p.win.right;
       if (p.win.left >= 0) hi0 = min(hi0, kj + p.win.left);
     }
     for (int h = U.h0; h < U.h0 + S.group; ++h) {
      if constexpr (BIAS != 0) {
        if (staged != h) {
          named_bar_sync(1, kCompute);
          stage_bias(tab, p, h, tid, kCompute);
          named_bar_sync(1, kCompute);
          HB = head_bias(tab);
          staged = h;
        }
        if (BIAS == 2) {
          for (int i = tid; i < 2 * R + 1; i += kCompute) acc[i] = 0.f;
          far_lo = far_hi = lost_lo = lost_hi = 0.f;
          named_bar_sync(1, kCompute);
        }
      }
      for (int t = U.tlo; t < U.tlo + U.nq; ++t, ++g) {
      float du_lo = 0.f;      // (BIAS 2) sum of the thread's dU of a far tile
      uint32_t v[32];
      const float* nl = reinterpret_cast<const float*>(smem + L::kLse) + (g % kStats) * L::kStat + 32 * w;
      if (kReadStat) ok = ok && mbar_wait(&st_full[g % kStats], (g / kStats) & 1, status);
      ok = __all_sync(0xffffffffu, ok && mbar_wait(&s_full[s_at(half, g)], s_phase(g), status));
      const uint32_t s_addr = lane_base + kTS + (kSBuf == 2 ? 128 * (g & 1) : 0) + 32 * w;
      if (ok) {
        tc_fence_after();
        tmem_ld32(s_addr, v);
        tmem_ld_wait();
        uint32_t gr[32];
        TileBias B{};
        if constexpr (BIAS != 0) B = tile_bias(tab, HB, R, near, t, U.u, kj - (t * kTile + 32 * w));
        const float f = BIAS != 0 ? B.factor(scale2) : scale2;
        const bool masked = t < U.full.x || t > U.full.y;
        const bool edge = (t + 1) * kTile > U.len || (BIAS == 2 && (U.u + 1) * kTile > U.len);
        const int lo = lo0 - (t * kTile + 32 * w), hi = hi0 - (t * kTile + 32 * w);
        const uint32_t see = masked ? column_mask(lo, hi, 0, 0) : ~0u;
        if constexpr (CAP) {
          if (masked) hide(v, see, 0u);
          cap_products(v, p.capf, true);
#pragma unroll
          for (int j = 0; j < 32; j += 2) put_pair(gr, j, cap_slope(pair_of(v, j), p.capf.zscale));
        }
        uint32_t pk[16];
        if constexpr (BIAS != 0) bias_chunk<-1>(v, 0, scale2, B);
        if (masked) hide(v, see, kMinusInf);
        const float2 f2 = make_float2(f, f), c2 = make_float2(B.c, B.c);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          float2 e0 = pair_of(v, j), e1 = pair_of(v, j + 2);
          if constexpr (kReadStat) {
            const float4 n4 = *reinterpret_cast<const float4*>(nl + j);
            float2 n0 = make_float2(n4.x, n4.y), n1 = make_float2(n4.z, n4.w);
            if constexpr (BIAS != 0) {
              n0 = fadd2(n0, c2);
              n1 = fadd2(n1, c2);
            }
            e0 = ffma2(e0, f2, n0);
            e1 = ffma2(e1, f2, n1);
          } else if constexpr (BIAS != 0) {
            e0 = ffma2(e0, f2, c2);
            e1 = ffma2(e1, f2, c2);
          } else {
            e0 = fmul2(e0, f2);
            e1 = fmul2(e1, f2);
          }
          e0 = make_float2(fast_exp2(e0.x), fast_exp2(e0.y));
          e1 = make_float2(fast_exp2(e1.x), fast_exp2(e1.y));
          pk[j / 2] = pack2(e0);
          pk[j / 2 + 1] = pack2(e1);
          put_pair(v, j, e0);
          put_pair(v, j + 2, e1);
        }
        if constexpr (CAP && BIAS != 2) {       // dS needs P (1 - tanh^2) alone
#pragma unroll
          for (int j = 0; j < 32; j += 2) put_pair(v, j, fmul2(pair_of(v, j), pair_of(gr, j)));
        }
        tmem_st16(s_addr, pk);
        tmem_st_wait();
        if (t * kTile + kRows * half + kRows > U.len) {
          // queries behind the document: the products below sum over them
          ok = __all_sync(0xffffffffu, mbar_wait(&do_full[half * kStages + g % kStages], (g / kStages) & 1, status));
          const int which = w % (4 / kHalves);
          if (ok && which < 2 && r < kRows && t * kTile + kRows * half + r >= U.len)
            clear_row<D, kRows>(smem + (which ? L::kQ : L::kDO) + L::part_at(half, g), r);
          fence_proxy_async_smem();
        }
        if (ok) {
          tc_fence_before();
          warp_arrive(&p_ready[s_at(half, g)]);
          ok = __all_sync(0xffffffffu, mbar_wait(&dp_full[half], g & 1, status));
        }
        if (ok) {
          tc_fence_after();
          float2 sum = make_float2(0.f, 0.f);
          uint32_t dp[32];
          tmem_ld32(dp_addr, dp);
          tmem_ld_wait();
          if (edge) drop_hidden(dp, v);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            float2 a0 = pair_of(dp, j), a1 = pair_of(dp, j + 2);
            if constexpr (!kFold) {
              const float4 d4 = *reinterpret_cast<const float4*>(nl + 128 + j);
              a0 = fadd2(a0, make_float2(-d4.x, -d4.y));
              a1 = fadd2(a1, make_float2(-d4.z, -d4.w));
            }
            a0 = fmul2(pair_of(v, j), a0);
            a1 = fmul2(pair_of(v, j + 2), a1);
            if constexpr (BIAS == 2) {
              put_pair(v, j, a0);
              put_pair(v, j + 2, a1);
              sum = fadd2(sum, fadd2(a0, a1));
              if constexpr (CAP) {
                a0 = fmul2(a0, pair_of(gr, j));
                a1 = fmul2(a1, pair_of(gr, j + 2));
              }
            }
            pk[j / 2] = pack2(a0);
            pk[j / 2 + 1] = pack2(a1);
          }
          du_lo = sum.x + sum.y;
          tmem_st16(dp_addr, pk);
          tmem_st_wait();
          tc_fence_before();
          warp_arrive(&ds_ready[half]);
          if (kReadStat && lane == 0) mbar_arrive(&st_empty[g % kStats]);
        }
      }
      if constexpr (BIAS == 2) {
        const int tile_rel = (U.u - t) * kTile;
        if (tile_rel + kTile - 1 <= -R) {
          add_comp(far_lo, lost_lo, du_lo);
        } else if (tile_rel - (kTile - 1) >= R) {
          add_comp(far_hi, lost_hi, du_lo);
        } else {
          // sums along the diagonals: a running value moves one lane up per column, so it stays on its
          // diagonal; lane 31's is complete
          float* dg = reinterpret_cast<float*>(smem + L::kDiag);
          named_bar_sync(1, kCompute);           // the last tile's are read
          float* mine = dg + (warp - 4) * 64;
          float run = 0.f;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            run += __uint_as_float(v[c]);
            if (lane == 31) mine[62 - c] = run;
            run = __shfl_up_sync(0xffffffffu, run, 1);
            if (lane == 0) run = 0.f;
          }
          if (lane > 0) mine[lane - 1] = run;      // after the last shift lane l holds diagonal l - 1
          named_bar_sync(1, kCompute);
          if (tid < 255) {
            const int x = tid - 127;               // key row - query column
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const int at = x - 32 * (q & 3) + 32 * (q >> 2) + 31;
              if (at >= 0 && at < 63) s += dg[q * 64 + at];
            }
            const int rel = tile_rel + x;
            if (rel <= -R) add_comp(far_lo, lost_lo, s);
            else if (rel >= R) add_comp(far_hi, lost_hi, s);
            else acc[rel + R] += s;
          }
          __syncwarp();
        }
      }
      }
      if constexpr (BIAS == 2) {
        // the head's sums of this key tile: the two ends over all threads in a fixed order
        float* red = reinterpret_cast<float*>(smem + L::kDiag);
        named_bar_sync(1, kCompute);
        far_lo += lost_lo;
        far_hi += lost_hi;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          far_lo += __shfl_xor_sync(0xffffffffu, far_lo, o);
          far_hi += __shfl_xor_sync(0xffffffffu, far_hi, o);
        }
        if (lane == 0) {
          red[2 * (warp - 4)] = far_lo;
          red[2 * (warp - 4) + 1] = far_hi;
        }
        named_bar_sync(1, kCompute);
        float* part = p.drel_part + ((size_t)h * p.plan[kPlanBwdItems] + U.item) * (2 * R + 1);
        for (int i = tid; i < 2 * R + 1; i += kCompute) {
          float s = acc[i];
          if (i == 0 || i == 2 * R) {
            s = 0.f;
            for (int q = 0; q < 16; ++q) s += red[2 * q + (i ? 1 : 0)];
          }
          part[i] = s;
        }
        named_bar_sync(1, kCompute);
      }
     }
     if (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(acc_full, S.n & 1, status));
        if (ok) {
          tc_fence_after();
          const bool valid = kj < U.len;
          const int c = (w & 1) * (D / 2);
          const uint32_t sum = lane_base + (w < 2 ? kTV : kTK) + c;
          if (p.dk_part) {
            float* part = w < 2 ? p.dv_part : p.dk_part;
            store_part<D / 2>(sum, part + ((int64_t)(U.start + kj) * p.hq + U.h0) * D + c, valid);
          } else {
            __nv_bfloat16* out = w < 2 ? p.dv : p.dk;
            store_acc<D / 2>(sum, out + ((int64_t)(U.start + kj) * p.hkv + U.hk) * D + c, w < 2 ? 1.f : p.scale, valid,
                             (reinterpret_cast<uintptr_t>(out) & 31) == 0);
          }
          tc_fence_before();
          mbar_arrive(acc_free);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ================================================================ dQ
// One CTA per SM walks (query tile, query head) units; a step is a key tile.  S = Q K^T and
// dP = dO V^T have queries in the TMEM lanes; Q and dO are A operands from tensor memory,
// copied there once a unit, which leaves shared memory to three K and three V tiles and
// halves what these products read from it.  dS goes over dP's columns and is the A operand
// of dQ += dS K.  The thread's row keeps its LSE and D in registers.
// What bounds a step is the chain dS -> dQ -> dP -> dS, as the next S runs while P is computed.
// At D = 64 there is room for a second dP (kPBuf), which cuts the chain, and S has an issuing warp of
// its own: 2% each on the noncausal case above when they came (now, with that warp, 2.08 ms with
// one dP and 2.11 with two).  At D = 128 a step goes in two halves of 64 keys as above, which
// costs the products nothing here (A comes from tensor memory: 33 cycles a step of 16 for half the
// columns): 5.90 -> 5.86 ms on the slopes case above, 622 -> 608 us on packed buckets.
// A cap makes the arithmetic longer than the chain, and its warps agree on the polynomial by
// votes: whole, 0.428 instead of 0.447 ms (odd prefix documents, 8 heads on 2).
// Roles: warp 0 TMA, warp 1 issues S, warp 2 dP and dQ, warps 4-19 compute as above.
// TMEM columns: dQ [0, D), S [128, 256), dP [256, 384), Q [384, ...), dO [448, ...); at D = 64
// Q [64, ...), dO [96, ...), dP [256, 512).
template <int D>
struct DqSmem {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = 3;
  static constexpr int kK = 0;                                   // [kStages]
  static constexpr int kV = kStages * kTileBytes;                // [kStages]
  static constexpr int kBias = 2 * kStages * kTileBytes;         // [kBiasTab]
  static constexpr int kBar = (kBias + kBiasTab * 4 + 15) & ~15;
  static constexpr int kBytes = kBar + 256;
  static constexpr int kAlloc = kBytes + 1024;
};

struct QuerySteps {
  int n, n_units;
  RawUnit raw;              // the next unit's
  int h, hk, t, start, len, nt, pre;
  KeyTiles kt;
  int k;
  // units: the two query tiles of a forward item for every head, the later one first (it sees
  // more); an item of one tile has empty units
  __device__ __forceinline__ void fetch(const ScoredParams& p, const PlanView& pv) {
    for (;; ++n) {
      raw.i = unit_index(n, n_units);
      if (raw.i < 0) return;
      raw.item = pv.fwd_items[raw.i / (2 * p.hq)];
      raw.span = pv.fwd_span[raw.i / (2 * p.hq)];
      if (kItemTiles - 1 - raw.i % (2 * p.hq) / p.hq < raw.item.z) {
        ++n;
        return;
      }
    }
  }
  __device__ __forceinline__ bool unit(const ScoredParams& p, const PlanView& pv) {
    if (raw.i < 0) return false;
    const int x = raw.i % (2 * p.hq);
    h = x % p.hq;
    hk = h / (p.hq / p.hkv);
    t = raw.item.y + kItemTiles - 1 - x / p.hq;
    start = raw.span.x;
    len = raw.span.y;
    nt = (len + kTile - 1) / kTile;
    pre = prefix_of(p, raw.item.x, len);
    kt = key_tiles(t, t, nt, (pre + kTile - 1) / kTile, p.win);
    k = 0;
    fetch(p, pv);
    return true;
  }
  __device__ __forceinline__ bool begin(const ScoredParams& p, const PlanView& pv) {
    n = 0;
    n_units = p.plan[kPlanFwdItems] * 2 * p.hq;
    fetch(p, pv);
    return unit(p, pv);
  }
  __device__ __forceinline__ bool first() const { return k == 0; }
  __device__ __forceinline__ bool last() const { return k == kt.n - 1; }
  __device__ __forceinline__ int tile() const { return kt.tile(k); }
  __device__ __forceinline__ bool next(const ScoredParams& p, const PlanView& pv) {
    if (last()) return unit(p, pv);
    ++k;
    return true;
  }
};

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    scored_dq_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const ScoredParams p) {
  using L = DqSmem<D>;
  constexpr int kStages = L::kStages, kPBuf = D == 64 ? 2 : 1, kHalves = D == 64 || CAP ? 1 : 2, kCols = kTile / kHalves;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t *k_full = bars, *k_empty = bars + kStages, *v_full = bars + 2 * kStages, *v_empty = bars + 3 * kStages;
  uint64_t *s_full = bars + 4 * kStages, *dp_full = s_full + 2, *s_free = s_full + 4, *ds_ready = s_full + 6;   // [halves or places]
  uint64_t *acc_full = s_full + 8, *acc_free = s_full + 9, *q_ready = s_full + 10, *drain = s_full + 11;        // drain [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_full + 13);
  int* status = const_cast<int*>(p.plan) + kPlanStatus;
  const PlanView pv = plan_view(p.plan, p.T, p.N);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4 * kStages + 4; ++i) mbar_init(bars + i, 1);
    for (int i = 0; i < 4; ++i) mbar_init(s_free + i, kCompute / 32 / kHalves);
    mbar_init(acc_full, 1);
    mbar_init(acc_free, kCompute / 32);
    mbar_init(q_ready, kCompute);
    mbar_init(drain, 1);
    mbar_init(drain + 1, 1);
    fence_mbar_init();
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
  constexpr uint32_t kTQ = 0, kTS = 128, kTP = 256, kTA = D == 64 ? 64 : 384, kTB = D == 64 ? 96 : 448;
  // dP and dS alternate between kPBuf places, with barriers of their own
  auto p_at = [&](int half, uint32_t g) { return kPBuf == 2 ? (int)(g & 1) : half; };
  auto p_phase = [&](uint32_t g) { return (kPBuf == 2 ? g >> 1 : g) & 1; };

  if (warp < 4) {
    setmaxnreg_dec<kRegCtl>();
    QuerySteps S{};
    bool more = S.begin(p, pv), ok = true;
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      uint32_t nk = 0, nv = 0;                       // tiles loaded
      for (; more && ok; more = S.next(p, pv)) {
        const int row = S.start + S.tile() * kTile;
        const uint32_t b = nk % kStages, par = (nk / kStages - 1) & 1;
        if (nk >= kStages && !(ok = mbar_wait(&k_empty[b], par, status))) break;
        load_tile<D>(smem + L::kK + b * L::kTileBytes, &tm_k, &k_full[b], S.hk, row);
        ++nk;
        if (nv >= kStages && !(ok = mbar_wait(&v_empty[b], par, status))) break;
        load_tile<D>(smem + L::kV + b * L::kTileBytes, &tm_v, &v_full[b], S.hk, row);
        ++nv;
      }
      for (uint32_t x = nk > kStages ? nk - kStages : 0; x < nk; ++x)
        mbar_wait(&k_full[x % kStages], (x / kStages) & 1, status);
      for (uint32_t x = nv > kStages ? nv - kStages : 0; x < nv; ++x)
        mbar_wait(&v_full[x % kStages], (x / kStages) & 1, status);
    } else if (warp == 1 || warp == 2) {
      // ---------------------------------------------------------- MMA issuers
      // warp 1: S, warp 2: dP and dQ
      const bool leader = elect_one();
      const uint32_t base16 = (smem_u32(smem) & 0x3FFFFu) >> 4;
      // A (Q or dO in TMEM): q_ready at the unit's first step; B (K or V): k_full, v_full
      auto scores = [&](uint32_t a, uint32_t b_off, uint32_t d, int half) {
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          if (leader)
            mma_bf16_ta(tbase + d, tbase + a + 8 * s,
                        sdesc_at(base16, b_off + (s / 4) * kTile * 128 + half * kCols * 128 + (s % 4) * 32, 16, 1024, kSwizzle128B),
                        idesc_bf16(128, kCols, 0, 0), s > 0);
      };
      auto issue_s = [&](uint32_t g, int half) {
        const uint32_t b = g % kStages;
        if (half == 0 && !(ok = warp_wait(&k_full[b], (g / kStages) & 1, status))) return;
        tc_fence_after();
        scores(kTA, L::kK + b * L::kTileBytes, kTS + kCols * half, half);
        if (leader) mma_commit(&s_full[half]);
      };
      auto issue_dp = [&](uint32_t g, int half) {
        const uint32_t b = g % kStages;
        if (half == 0 && !(ok = warp_wait(&v_full[b], (g / kStages) & 1, status))) return;
        tc_fence_after();
        scores(kTB, L::kV + b * L::kTileBytes, kTP + (kPBuf == 2 ? 128 * (g & 1) : kCols * half), half);
        if (leader) {
          mma_commit(&dp_full[p_at(half, g)]);
          if (half == kHalves - 1) mma_commit(&v_empty[b]);
        }
      };
      uint32_t units = 0;
      for (uint32_t g = 0; more && ok; ++g) {
        const bool first = S.first(), last = S.last();
        if (first) {
          if (!(ok = warp_wait(q_ready, units++ & 1, status))) break;
          tc_fence_after();
#pragma unroll
          for (int half = 0; half < kHalves; ++half) {
            if (!ok) continue;
            if (warp == 1) issue_s(g, half);
            else issue_dp(g, half);
          }
        }
        if (warp == 1) {
#pragma unroll
          for (int half = 0; half < kHalves; ++half)
            if (ok && !last && (ok = warp_wait(&s_free[half], g & 1, status))) issue_s(g + 1, half);
        } else {
          const uint32_t b = g % kStages;
          if (ok && kPBuf == 2 && !last) issue_dp(g + 1, 0);
          // dQ += dS K.  A (dS in TMEM): ds_ready; B (K): ds_ready too, as the same threads have read the
          // whole of the S that came from this K (k_full is the other warp's; it cannot have moved on,
          // because this product gives the stage back).  The unit's first product overwrites the sums of
          // the last one: those have to be out
          if (ok && first && units > 1) ok = warp_wait(acc_free, units & 1, status);
#pragma unroll
          for (int half = 0; half < kHalves; ++half) {
            if (!ok || !(ok = warp_wait(&ds_ready[p_at(half, g)], p_phase(g), status))) continue;
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < kCols / 16; ++s)
              if (leader)
                mma_bf16_ta(tbase + kTQ, tbase + kTP + (kPBuf == 2 ? 128 * (g & 1) : kCols * half) + 32 * (s >> 1) + 8 * (s & 1),
                            sdesc_at(base16, L::kK + b * L::kTileBytes + half * kCols * 128 + s * 2048, kTile * 128, 1024, kSwizzle128B),
                            idesc_bf16(128, D, 0, 1), (!(first && half == 0) || s > 0));
            if (leader && half == kHalves - 1) {
              mma_commit(&k_empty[b]);
              if (last) mma_commit(acc_full);
            }
            if (!last && kPBuf == 1) issue_dp(g + 1, half);
          }
        }
        more = S.next(p, pv);
      }
      if (leader) {
        mma_commit(&drain[warp - 1]);
        mbar_wait(&drain[warp - 1], 0, status);
      }
    }
  } else {
    // ------------------------------------------------------------ compute
    setmaxnreg_inc<kRegCompute>();
    const int w = (warp - 4) >> 2, quarter = warp & 3, half = kHalves == 2 ? w >> 1 : 0;
    const int r = quarter * 32 + lane, tid = threadIdx.x - 128;
    const uint32_t lane_base = tbase + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_addr = lane_base + kTS + 32 * w, dp_base = lane_base + kTP + 32 * w;
    float* tab = reinterpret_cast<float*>(smem + L::kBias);
    const int R = bias_range(p);
    const int near = near_tiles(R);
    const float scale2 = p.scale2;
    HeadBias HB{};
    int staged = -1;
    bool ok = true;
    float nl = 0.f, dv = 0.f;
    int lo = 0, hi = 0;
    FullTiles full{};
    QuerySteps S{};
    // The unit's A operands (warpgroups 0 and 1: Q, 2 and 3: dO; rows behind the document as zeros), LSE and D.
    auto start_unit = [&]() {
      const int qi = S.t * kTile + r;
      const bool in = qi < S.len;
      const int64_t tok = (int64_t)S.start + qi;
      const int c = (w & 1) * (D / 2);
      const uint4* src = reinterpret_cast<const uint4*>((w < 2 ? p.q : p.dout) + (tok * p.hq + S.h) * D + c);
      uint32_t a[D / 4];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint4 x = in ? src[i] : make_uint4(0, 0, 0, 0);
        a[4 * i] = x.x;
        a[4 * i + 1] = x.y;
        a[4 * i + 2] = x.z;
        a[4 * i + 3] = x.w;
      }
      nl = in ? -usable_lse(p.lse[(int64_t)S.h * p.T + tok]) * kLog2e : -INFINITY;
      dv = in ? p.dvec[(int64_t)S.h * p.T + tok] : 0.f;
      lo = p.win.left < 0 ? 0 : max(0, qi - p.win.left);
      hi = p.win.right < 0 ? S.len - 1 : min(S.len - 1, qi + p.win.right);
      full = full_tiles(S.t, S.len, S.pre, p.win);
      const uint32_t at = lane_base + (w < 2 ? kTA : kTB) + c / 2;
      if constexpr (D == 128) tmem_st32(at, a);
      else tmem_st16(at, a);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(q_ready);
    };
    uint32_t g = 0, units = 0;
    bool more = S.begin(p, pv);
    if (more) start_unit();
    for (; more; ++g) {
      if constexpr (BIAS) {
        if (S.first() && staged != S.h) {
          named_bar_sync(1, kCompute);
          stage_bias(tab, p, S.h, tid, kCompute);
          named_bar_sync(1, kCompute);
          HB = head_bias(tab);
          staged = S.h;
        }
      }
      const int t = S.t, u = S.tile(), qi = t * kTile + r;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&s_full[half], g & 1, status));
      if (ok) {
        tc_fence_after();
        uint32_t v[32], gr[32];
        tmem_ld32(s_addr, v);
        tmem_ld_wait();
        tc_fence_before();
        warp_arrive(&s_free[half]);
        TileBias B{};
        if constexpr (BIAS) B = tile_bias(tab, HB, R, near, t, u, u * kTile + 32 * w - qi);
        const float f = BIAS ? B.factor(scale2) : scale2;
        const bool masked = !full.has(u);
        const int c0 = u * kTile + 32 * w;
        const uint32_t see = masked ? column_mask(lo - c0, hi - c0, S.pre - c0, 0) : ~0u;
        if constexpr (CAP) {
          if (masked) hide(v, see, 0u);
          cap_products(v, p.capf, qi < S.len);
#pragma unroll
          for (int j = 0; j < 32; j += 2) put_pair(gr, j, cap_slope(pair_of(v, j), p.capf.zscale));
        }
        const float2 f2 = make_float2(f, f), n2 = make_float2(nl + B.c, nl + B.c);
        if constexpr (BIAS) bias_chunk<1>(v, 0, scale2, B);
        if (masked) hide(v, see, kMinusInf);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          float2 e = ffma2(pair_of(v, j), f2, n2);
          e = make_float2(fast_exp2(e.x), fast_exp2(e.y));
          if constexpr (CAP) e = fmul2(e, pair_of(gr, j));
          put_pair(v, j, e);
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&dp_full[p_at(half, g)], p_phase(g), status));
        if (ok) {
          tc_fence_after();
          const float2 d2 = make_float2(-dv, -dv);
          uint32_t pk[16];
          uint32_t dp[32];
          const uint32_t dp_addr = dp_base + (kPBuf == 2 ? 128 * (g & 1) : 0);
          tmem_ld32(dp_addr, dp);
          tmem_ld_wait();
          if ((u + 1) * kTile > S.len) drop_hidden(dp, v);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 e = pair_of(v, j);
            const float2 a = fmul2(e, fadd2(pair_of(dp, j), d2));
            pk[j / 2] = pack2(a);
          }
          tmem_st16(dp_addr, pk);
          tmem_st_wait();
          if ((u + 1) * kTile > S.len) {       // keys behind the document: dQ sums over them
            if (w % (4 / kHalves) == 0 && r / kCols == half && u * kTile + r >= S.len) clear_row<D>(smem + L::kK + (g % kStages) * L::kTileBytes, r);
            fence_proxy_async_smem();
          }
          tc_fence_before();
          warp_arrive(&ds_ready[p_at(half, g)]);
        }
      }
      const bool last = S.last();
      const int h = S.h;
      const int64_t tok = (int64_t)S.start + qi;
      const bool valid = qi < S.len;
      more = S.next(p, pv);
      if (last && ok) {
        // when every product that reads Q and dO of this unit is done, the next unit's go in, while its
        // last dQ product runs
        if (kHalves == 2)
          ok = __all_sync(0xffffffffu, mbar_wait(w < 2 ? &s_full[1] : &dp_full[0], g & 1, status));
        if (ok && more) start_unit();
        ok = ok && __all_sync(0xffffffffu, mbar_wait(acc_full, units & 1, status));
        ++units;
        if (ok) {
          tc_fence_after();
          if (w < D / 32) store_acc<32>(lane_base + kTQ + 32 * w, p.dq + (tok * p.hq + h) * D + 32 * w, p.scale, valid,
                                       (reinterpret_cast<uintptr_t>(p.dq) & 31) == 0);
          tc_fence_before();
          warp_arrive(acc_free);
        }
      }
    }
  }
  grid_wait();                   // who comes behind dQ in the stream comes behind dK and dV too
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// drel[h][i] = sum over the key tiles of their partial sums: a warp per eighth of the tiles,
// in 64 bits (a chain of hundreds of fp32 sums would cost the last digits), then the warps' in order.
__global__ void __launch_bounds__(256) scored_drel_kernel(const float* __restrict__ part, const int* __restrict__ plan,
                                                          int R, float* __restrict__ drel) {
  __shared__ double sums[8][32];
  const int width = 2 * R + 1, items = plan[kPlanBwdItems], h = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
  double s = 0.0;
  if (i < width) {
    const float* src = part + (size_t)h * items * width + i;
#pragma unroll 4
    for (int n = warp; n < items; n += 8) s += (double)src[(size_t)n * width];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && i < width) {
    for (int q = 1; q < 8; ++q) s += sums[q][lane];
    drel[(size_t)h * width + i] = (float)s;
  }
}

// dK and dV of a kv head from those of its query heads, in their order (split): four columns
// a thread.
template <int D>
__global__ void __launch_bounds__(256) scored_heads_kernel(const ScoredParams p) {
  const int group = p.hq / p.hkv;
  const int64_t n = (int64_t)p.plan[kPlanValid] * p.hkv * (D / 4);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / (D / 4);                       // token * hkv + kv head
    const int c = (int)(i % (D / 4)) * 4;
    const float* part = blockIdx.y ? p.dv_part : p.dk_part;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = 0; g < group; ++g) {
      const float4 x = *reinterpret_cast<const float4*>(part + (row * group + g) * D + c);
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    const float f = blockIdx.y ? 1.f : p.scale;
    const uint2 out = make_uint2(pack2(make_float2(s.x * f, s.y * f)), pack2(make_float2(s.z * f, s.w * f)));
    *reinterpret_cast<uint2*>((blockIdx.y ? p.dv : p.dk) + row * D + c) = out;
  }
}

template <int D, bool CAP, int BIAS>
cudaError_t launch(const ScoredParams& p, cudaStream_t stream) {
  CUtensorMap tq, tk, tv, tdo;
  if (!make_tmap_bf16_3d(&tq, p.q, D, p.hq, p.T, D * 2, (uint64_t)p.hq * D * 2, 64, DkvSmem<D, BIAS>::kRows) ||
      !make_tmap_bf16_3d(&tk, p.k, D, p.hkv, p.T, D * 2, (uint64_t)p.hkv * D * 2, 64, kTile) ||
      !make_tmap_bf16_3d(&tv, p.v, D, p.hkv, p.T, D * 2, (uint64_t)p.hkv * D * 2, 64, kTile) ||
      !make_tmap_bf16_3d(&tdo, p.dout, D, p.hq, p.T, D * 2, (uint64_t)p.hq * D * 2, 64, DkvSmem<D, BIAS>::kRows))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0, regs1 = 0, regs2 = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  constexpr int smem1 = DkvSmem<D, BIAS>::kAlloc, smem2 = DqSmem<D>::kAlloc;
  static_assert(smem1 <= 232448 && smem2 <= 232448, "shared memory of one CTA");
  if (e == cudaSuccess) e = prepare_kernel<scored_dkv_kernel<D, CAP, BIAS>>(smem1, &regs1);
  if (e == cudaSuccess) e = prepare_kernel<scored_dq_kernel<D, CAP, BIAS != 0>>(smem2, &regs2);
  if (e != cudaSuccess) return e;
  if (regs1 != kLaunchRegs || regs2 != kLaunchRegs) return cudaErrorInvalidConfiguration;
  const int64_t tiles = (int64_t)p.T / kTile + p.N + 1, items = (int64_t)p.T / (kTile * kItemTiles) + p.N + 1;
  constexpr int kRows = 256 / (D / 8);
  const int64_t prep = (((int64_t)p.T + kRows - 1) / kRows) * p.hq;
  if (tiles * p.hq > 0x7FFFFFFF || items * 2 * p.hq > 0x7FFFFFFF || prep > 0x7FFFFFFF) return cudaErrorInvalidValue;
  scored_prep_kernel<D><<<(unsigned)prep, 256, 0, stream>>>(p);
  const unsigned g1 = (unsigned)std::min<int64_t>(tiles * (p.dk_part ? p.hq : p.hkv), sms), g2 = (unsigned)std::min<int64_t>(items * 2 * p.hq, sms);
  // dK/dV and dQ start while the launch before still runs (32 -> 18 us for one document of 256, 650 ->
  // 632 for packed documents with buckets, 429 -> 435 where the parts of dK are added in between):
  // they wait for D alone, and dQ for the rest at its end
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(g1);
  cfg.dynamicSmemBytes = smem1;
  e = cudaLaunchKernelEx(&cfg, scored_dkv_kernel<D, CAP, BIAS>, tq, tk, tv, tdo, p);
  if (e != cudaSuccess) return e;
  if (p.dk_part) {               // the parts are added while L2 holds them
    scored_heads_kernel<D><<<dim3(sms, 2), 256, 0, stream>>>(p);
    cfg.numAttrs = 0;
  }
  cfg.gridDim = dim3(g2);
  cfg.dynamicSmemBytes = smem2;
  e = cudaLaunchKernelEx(&cfg, scored_dq_kernel<D, CAP, BIAS != 0>, tk, tv, p);
  if (e != cudaSuccess) return e;
  if (BIAS == 2) {
    const dim3 grid((2 * p.R + 1 + 31) / 32, p.hq);
    scored_drel_kernel<<<grid, 256, 0, stream>>>(p.drel_part, p.plan, p.R, p.drel);
  }
  return cudaGetLastError();
}

template <int D, bool CAP>
cudaError_t launch_cap(const ScoredParams& p, cudaStream_t s) {
  if (p.drel) return launch<D, CAP, 2>(p, s);
  return p.slopes || p.rel ? launch<D, CAP, 1>(p, s) : launch<D, CAP, 0>(p, s);
}

}  // namespace

cudaError_t launch_scored_bwd(int D, const ScoredParams& p, cudaStream_t s) {
  if (D == 128) return p.cap > 0.f ? launch_cap<128, true>(p, s) : launch_cap<128, false>(p, s);
  return p.cap > 0.f ? launch_cap<64, true>(p, s) : launch_cap<64, false>(p, s);
}

}  // namespace flamia
