// Scored attention: what its kernels and the ABI share (parameters, the bucket rule,
// the visible-key sets and the backward's workspace layout).
#pragma once
#include <algorithm>
#include <cmath>

#include "common.cuh"

namespace flamia {

// tanh cap of raw products S (s = softmax scale S): S (1 + t) with t = tanh(z) / z - 1 and
// z = zscale S, the capped score over the softmax scale.
struct CapForm {
  float zscale;      // softmax scale / cap
  float inv;         // cap / softmax scale
  float t3, t5;      // up to this |S| the polynomials of 3 and of 5 coefficients serve (-1: never, not even for 0)
  float2 k3[3], k5[5];    // their coefficients of S^2, S^4, ... (twice: packed operands)
  float2 e3[4], e5[6];    // the same with 1 in front, times the scale in base 2
};

struct ScoredParams {
  const __nv_bfloat16 *q, *k, *v;
  const int* plan;
  const int32_t* prefix;     // [N] or null
  int N, T, hq, hkv;
  float scale;               // softmax scale
  float scale2;              // softmax scale log2 e, with the products' mean truncation taken back
  float cap;                 // 0: none
  CapForm capf;
  const float* slopes;       // [hq] or null
  const float* rel;          // [hq, 2R+1] or null
  int R;
  Window win;
  __nv_bfloat16* out;        // forward: written; backward: read
  float* lse;
  // backward
  const __nv_bfloat16* dout;
  __nv_bfloat16 *dq, *dk, *dv;
  float* drel;               // [hq, 2R+1] or null
  float* dvec;               // workspace: D [hq, T]
  float* drel_part;          // workspace: partial sums of drel
  float *dk_part, *dv_part;  // workspace: dK, dV of each query head [T, hq, D] (split) or null
};

// The dK/dV units are key tiles of a kv head, which walk the query heads that share it one
// after the other.  With fewer than four such units an SM the longest one sets the time (a
// prefix that every query sees: one unit of 132 steps beside 70 on average), so each query
// head's share becomes a unit of its own, and its sums go through memory in fp32 (odd prefix
// documents of 9097 rows, 8 heads on 2: 472 -> 441 us).
constexpr int64_t kSplitBelow = 4 * 152;
inline bool scored_bwd_split(int64_t T, int N, int hq, int hkv) {
  return hq > hkv && plan_capacity(T, N) * hkv < kSplitBelow;
}
struct ScoredBwdWorkspace {
  size_t dvec, drel, dk, dv, total;
};
inline ScoredBwdWorkspace scored_bwd_layout(int64_t T, int N, int hq, int hkv, int d, int R) {
  auto round256 = [](size_t x) { return (x + 255) & ~size_t(255); };
  ScoredBwdWorkspace w;
  size_t off = 0;
  w.dvec = off;
  off = round256(off + (size_t)T * hq * 4);
  w.drel = off;
  if (R > 0) off = round256(off + (size_t)plan_capacity(T, N) * hq * (2 * R + 1) * 4);
  const size_t part = scored_bwd_split(T, N, hq, hkv) ? round256((size_t)T * hq * d * 4) : 0;
  w.dk = off;
  w.dv = off + part;
  off += 2 * part;
  w.total = off > 0 ? off : 256;
  return w;
}

// The tensor core truncates as it accumulates, so a product of D terms comes out too small:
// on 65,536 rows of normal values by 9.9e-8 of the product at D = 128 (eight steps of 16 terms)
// and 5.5e-8 at D = 64 on average, beside a spread of 7e-8.  The score scale takes the mean back;
// it would enter every probability with the score's own size as a factor.  How much a product
// loses depends on its terms.  LSE's rms error over 2048 causal rows with it / without, 1e-7, D = 64
// and 128: normal values 4.3 / 5.7, 4.4 / 6.6; positive 6.1 / 8.8, 8.0 / 15; of mean 1 7.0 / 11,
// 7.8 / 18; one term alone 4.3 / 4.4, 4.2 / 4.3; uniform 4.2 / 4.3, 4.1 / 4.4; heavy tails 5.7 / 8.4,
// 5.8 / 9.3; small whole numbers, whose sums lose nothing, 6.5 / 6.3, 6.9 / 5.2.
inline double mma_gain(int D) { return D == 128 ? 1.0 + 9.9e-8 : 1.0 + 5.5e-8; }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

// Bias entries below this hide the pair, as -inf does (the lowest float would lose the
// score's own value in the sum and overflow in base 2).
constexpr float kHideBelow = -1.2676506002282294e30f;   // -2^100

// ---------------------------------------------------------------- visible tiles
// Key tiles that a run of query tiles [t0, t1] of a document sees: the a tiles of the prefix
// that lie before the window's first tile, then the n - a tiles from lo on (the window's, and
// prefix tiles behind its first).  They are walked from the last to the first: a bias that
// falls with the distance then puts a causal row's maximum into its first tiles, and the
// running maximum stays.
struct KeyTiles {
  int a, lo, n;
  __device__ __forceinline__ int tile(int k) const {
    const int x = n - 1 - k;
    return x < a ? x : lo + (x - a);
  }
};
__device__ __forceinline__ KeyTiles key_tiles(int t0, int t1, int nt, int pre_tiles, Window w) {
  KeyTiles s;
  s.lo = win_klo(t0, w);
  s.a = min(pre_tiles, s.lo);
  const int hi = max(win_khi(t1, nt, w), pre_tiles - 1);
  s.n = s.a + hi - s.lo + 1;
  return s;
}
// Key tiles that every query of query tile t sees whole: those below pre, and [lo, hi].
struct FullTiles {
  int pre, lo, hi;
  __device__ __forceinline__ bool has(int u) const { return u < pre || (u >= lo && u <= hi); }
};
__device__ __forceinline__ FullTiles full_tiles(int t, int len, int pre, Window w) {
  FullTiles f;
  f.pre = pre / kTile;                       // pre <= len
  f.lo = w.left < 0 ? 0 : max(0, t * kTile + 2 * kTile - 2 - w.left) / kTile;
  f.hi = len / kTile - 1;
  if (w.right >= 0) f.hi = min(f.hi, (t * kTile + w.right + 1) / kTile - 1);
  return f;
}
// Query tiles of which every query sees key tile u whole: [lo, hi] (whole query tiles only).
__device__ __forceinline__ int2 full_queries(int u, int len, int pre, Window w) {
  int lo = 0, hi = len / kTile - 1;
  if ((u + 1) * kTile > len) hi = -1;
  if ((u + 1) * kTile > pre) {
    if (w.right >= 0) lo = max(0, u * kTile + 2 * kTile - 2 - w.right) / kTile;
    if (w.left >= 0) hi = min(hi, u * kTile + w.left >= kTile - 1 ? (u * kTile + w.left - (kTile - 1)) / kTile : -1);
  }
  return make_int2(lo, hi);
}
// Bits of 32 columns starting at column c0: the columns [lo, hi] and those below pre.
__device__ __forceinline__ uint32_t below_mask(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }
__device__ __forceinline__ uint32_t column_mask(int lo, int hi, int pre, int c0) {
  return (below_mask(hi + 1 - c0) & ~below_mask(lo - c0)) | below_mask(pre - c0);
}

// Unit number k of this CTA, or -1: boustrophedon rounds over the cost-sorted list.
__device__ __forceinline__ int unit_index(int k, int n_units) {
  const int G = gridDim.x, c = blockIdx.x;
  if ((int64_t)k * G >= n_units) return -1;
  const int i = k * G + ((k & 1) ? G - 1 - c : c);
  return i < n_units ? i : -1;
}
__device__ __forceinline__ int prefix_of(const ScoredParams& p, int doc, int len) {
  return p.prefix ? min(max(p.prefix[doc], 0), len) : 0;
}
// Clear row r of a TMA-staged [ROWS][D] bf16 tile (64-column boxes): a tile's rows
// behind the document belong to the next one, or to nobody, and may hold anything;
// weight 0 does not silence an infinity.
template <int D, int ROWS = kTile>
__device__ __forceinline__ void clear_row(uint8_t* tile, int r) {
#pragma unroll
  for (int b = 0; b < D / 64; ++b) {
    uint4* row = reinterpret_cast<uint4*>(tile + b * ROWS * 128 + r * 128);
#pragma unroll
    for (int c = 0; c < 8; ++c) row[c] = make_uint4(0, 0, 0, 0);
  }
}

// ---------------------------------------------------------------- scores in base 2
// The kernels hold u log2(e), so that the softmax is 2^x.
//
// tanh cap.  tanh(z) / z - 1 = w Q(w), w = z^2, by least squares in relative error reweighted
// towards equal ripple on Chebyshev nodes of w: three coefficients up to |z| = 0.375 (7e-8),
// five up to 0.8 (6.5e-8), each with zscale folded in, so that a capped product costs n + 2
// packed fp32 operations and stays in the products' units.  The fp32 pipe bounds this (one
// operation an element is 128 cycles a tile, a tile's two products at D = 128 are 1024), so a
// warp takes the shorter form when all its values allow it.  Beyond 0.8, tanh(z) = 1 - 2 /
// (1 + 2^(2 z log2 e)), which loses nothing there.
constexpr float kTanh3To = 0.375f, kTanh5To = 0.8f;
constexpr float kTanh3[3] = {-0.33332332968711853f, 0.1328972578048706f, -0.048487283289432526f};
constexpr float kTanh5a = -0.3333286643028259f, kTanh5b = 0.1332276612520218f, kTanh5c = -0.053176309913396835f,
                kTanh5d = 0.01919075846672058f, kTanh5e = -0.004410882946103811f;
inline CapForm cap_form(double scale, double cap) {
  const double scale2 = scale * 1.4426950408889634;
  auto two = [](double x) { return make_float2((float)x, (float)x); };
  CapForm c{};
  if (!(cap > 0.0)) return c;
  const double z = scale / cap;
  c.zscale = (float)z;
  c.inv = (float)(cap / scale);
  // A folded coefficient that left the fp32 range would make 0 * inf of a product of 0 (a hidden pair's, a
  // row of zeros'): where the largest one does, its polynomial serves nothing, and its coefficients stay 0.
  const double most = std::max(1.0, scale2);
  const bool use3 = z > 1e-6 && std::pow(z, 6) * most < 1e38, use5 = z > 3e-4 && std::pow(z, 10) * most < 1e38;
  c.t3 = use3 ? (float)(kTanh3To / z) : -1.f;
  c.t5 = use5 ? (float)(kTanh5To / z) : -1.f;
  const float k5[5] = {kTanh5a, kTanh5b, kTanh5c, kTanh5d, kTanh5e};
  double f = z * z;
  for (int i = 0; i < 5; ++i, f *= z * z) {
    if (use3 && i < 3) c.k3[i] = two(kTanh3[i] * f), c.e3[i + 1] = two(kTanh3[i] * f * scale2);
    if (use5) c.k5[i] = two(k5[i] * f), c.e5[i + 1] = two(k5[i] * f * scale2);
  }
  c.e3[0] = c.e5[0] = two(scale2);
  return c;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float tanh_any(float z) {
  return fmaf(-2.f, fast_rcp(1.f + fast_exp2(z * (2.f * kLog2e))), 1.f);
}

// A tile's bias is a function of the distance: near the diagonal (some distance below R, or
// both signs of it) a value per distance from a staged table; elsewhere a constant, or with a
// slope a constant and a multiple of the column.
struct TileBias {
  const float* tab; // table entry of the thread's column 0, or null
  float col;        // the slope's part per unit of distance, in the products' units
  float c;          // the rest, added in the exponent
  __device__ __forceinline__ float factor(float scale2) const { return tab ? 1.f : scale2; }
};
__device__ __forceinline__ float2 pair_of(const uint32_t (&v)[32], int j) {
  return make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
}
__device__ __forceinline__ void put_pair(uint32_t (&v)[32], int j, float2 x) {
  v[j] = __float_as_uint(x.x);
  v[j + 1] = __float_as_uint(x.y);
}
// x for the columns of a row without their bit in the mask.
__device__ __forceinline__ void hide(uint32_t (&v)[32], uint32_t see, uint32_t x) {
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = (see >> j) & 1 ? v[j] : x;
}
constexpr uint32_t kMinusInf = 0xff800000u;
// A group of N x 32 raw products -> capped, in the same units.  The warp's length of the
// polynomial shows in a result's last bits, so only products that count choose it: those of
// hidden pairs are 0 by now, and a row outside the document (counts false) has no say.  A
// result thus depends on its warp's 32 rows of the document and on keys that they see.
template <int N>
__device__ __forceinline__ void cap_products(uint32_t (&v)[N][32], const CapForm& F, bool counts) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int g = 0; g < N; ++g)
#pragma unroll
    for (int j = 0; j < 32; j += 2)
      m[(j / 2) % 4] = fmax3(m[(j / 2) % 4], fabsf(__uint_as_float(v[g][j])), fabsf(__uint_as_float(v[g][j + 1])));
  const float am = fmaxf(fmax3(m[0], m[1], m[2]), m[3]);
  if (!__any_sync(0xffffffffu, counts && !(am <= F.t3))) {
#pragma unroll
    for (int g = 0; g < N; ++g)
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float2 x = pair_of(v[g], j), w = fmul2(x, x);
        float2 t = ffma2(w, F.k3[2], F.k3[1]);
        t = ffma2(w, t, F.k3[0]);
        put_pair(v[g], j, ffma2(x, fmul2(w, t), x));
      }
  } else if (!__any_sync(0xffffffffu, counts && !(am <= F.t5))) {
#pragma unroll
    for (int g = 0; g < N; ++g)
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float2 x = pair_of(v[g], j), w = fmul2(x, x);
        float2 t = ffma2(w, F.k5[4], F.k5[3]);
        t = ffma2(w, t, F.k5[2]);
        t = ffma2(w, t, F.k5[1]);
        t = ffma2(w, t, F.k5[0]);
        put_pair(v[g], j, ffma2(x, fmul2(w, t), x));
      }
  } else {
#pragma unroll
    for (int g = 0; g < N; ++g)
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float x = __uint_as_float(v[g][j]), z = x * F.zscale, w = z * z;
        float t = fmaf(w, kTanh5e, kTanh5d);
        t = fmaf(w, t, kTanh5c);
        t = fmaf(w, t, kTanh5b);
        t = fmaf(w, t, kTanh5a);
        v[g][j] = __float_as_uint(fabsf(z) <= kTanh5To ? fmaf(x, w * t, x) : F.inv * tanh_any(z));
      }
  }
}
__device__ __forceinline__ void cap_products(uint32_t (&v)[32], const CapForm& F, bool counts) {
  cap_products(reinterpret_cast<uint32_t(&)[1][32]>(v), F, counts);
}
// Column numbers as constants that a packed operation reads in place; as immediates each takes
// a move of its own (slopes, two noncausal documents of 8192, 16 heads, d = 64: 832 / 803 us
// forward, 2150 / 2028 backward).
static __constant__ float kColumn[128] = {
    0.f, 1.f, 2.f, 3.f, 4.f, 5.f, 6.f, 7.f, 8.f, 9.f, 10.f, 11.f, 12.f, 13.f, 14.f, 15.f, 16.f, 17.f, 18.f,
    19.f, 20.f, 21.f, 22.f, 23.f, 24.f, 25.f, 26.f, 27.f, 28.f, 29.f, 30.f, 31.f, 32.f, 33.f, 34.f, 35.f,
    36.f, 37.f, 38.f, 39.f, 40.f, 41.f, 42.f, 43.f, 44.f, 45.f, 46.f, 47.f, 48.f, 49.f, 50.f, 51.f, 52.f,
    53.f, 54.f, 55.f, 56.f, 57.f, 58.f, 59.f, 60.f, 61.f, 62.f, 63.f, 64.f, 65.f, 66.f, 67.f, 68.f, 69.f,
    70.f, 71.f, 72.f, 73.f, 74.f, 75.f, 76.f, 77.f, 78.f, 79.f, 80.f, 81.f, 82.f, 83.f, 84.f, 85.f, 86.f,
    87.f, 88.f, 89.f, 90.f, 91.f, 92.f, 93.f, 94.f, 95.f, 96.f, 97.f, 98.f, 99.f, 100.f, 101.f, 102.f,
    103.f, 104.f, 105.f, 106.f, 107.f, 108.f, 109.f, 110.f, 111.f, 112.f, 113.f, 114.f, 115.f, 116.f, 117.f,
    118.f, 119.f, 120.f, 121.f, 122.f, 123.f, 124.f, 125.f, 126.f, 127.f};
// The table's or the slope's part for columns c0 .. c0 + 31 (column c: distance DIR c more);
// with a table the result is in base 2, else the products' units stay.
template <int DIR>
__device__ __forceinline__ void bias_chunk(uint32_t (&v)[32], int c0, float scale2, const TileBias& B) {
  if (B.tab) {
    const float2 f2 = make_float2(scale2, scale2);
    const float* tab = B.tab + DIR * c0;
#pragma unroll
    for (int j = 0; j < 32; j += 2) put_pair(v, j, ffma2(pair_of(v, j), f2, make_float2(tab[DIR * j], tab[DIR * (j + 1)])));
  } else if (B.col != 0.f) {
    const float2 s2 = make_float2(DIR * B.col, DIR * B.col);
#pragma unroll
    for (int j = 0; j < 32; j += 2)
      put_pair(v, j, ffma2(make_float2(kColumn[c0 + j], kColumn[c0 + j + 1]), s2, pair_of(v, j)));
  }
}

// Staged bias of one head in base 2: entry r + R + 255 of the table holds the bias of distance
// r, clipped to R on both sides and long enough for every tile that holds a distance below R,
// so that no index is clipped in the loops.  Without a bias by distance R counts as 1: the
// table then serves the tiles on the diagonal, where a slope's sign changes.
constexpr int kBiasReach = 2 * kTile - 1;
constexpr int kBiasHead = 2 * (FLAMIA_REL_MAX + kBiasReach) + 2;  // behind the table: the head's constants
constexpr int kBiasTab = kBiasHead + 4;                            // floats, an even number
// (Comparisons that a NaN fails: it stays one, and shows in the outputs.)
__device__ __forceinline__ float bias_base2(float b) {
  return b < kHideBelow ? -INFINITY : (b > -kHideBelow ? -kHideBelow : b) * kLog2e;
}
// A slope steeper than 2^100 counts as 2^100 (times the longest distance it stays in the fp32 range); in
// the products' units it is held to 2^119, whose multiple by a column is finite too.  (At that steepness a
// step of distance outweighs any score, so that only the nearest or the farthest visible key counts.)
__device__ __forceinline__ float slope_base2(float s) { return (fabsf(s) > -kHideBelow ? copysignf(-kHideBelow, s) : s) * kLog2e; }
__device__ __forceinline__ float slope_products(float slope2, float scale2) {
  return fminf(fmaxf(slope2 / scale2, -0x1p119f), 0x1p119f);
}
__device__ __forceinline__ int bias_range(const ScoredParams& p) { return p.rel ? p.R : 1; }
struct HeadBias {
  float slope2, lo, hi;      // slope, and the bias of the distances up to -R and from R on
  float col;                 // the slope in the products' units
};
__device__ __forceinline__ void stage_bias(float* tab, const ScoredParams& p, int h, int first, int stride) {
  const int R = bias_range(p);
  const float slope2 = p.slopes ? slope_base2(p.slopes[h]) : 0.f;
  const float* src = p.rel ? p.rel + (size_t)h * (2 * R + 1) : nullptr;
  for (int i = first; i < 2 * (R + kBiasReach) + 1; i += stride) {
    const float b = src ? bias_base2(src[min(max(i - kBiasReach, 0), 2 * R)]) : 0.f;
    tab[i] = fmaf(fabsf((float)(i - R - kBiasReach)), -slope2, b);
    if (i == 0) tab[kBiasHead] = slope2;
    if (i == 0) tab[kBiasHead + 1] = b;
    if (i == 0) tab[kBiasHead + 3] = slope_products(slope2, p.scale2);
    if (i == 2 * (R + kBiasReach)) tab[kBiasHead + 2] = b;
  }
}
__device__ __forceinline__ HeadBias head_bias(const float* tab) {
  return HeadBias{tab[kBiasHead], tab[kBiasHead + 1], tab[kBiasHead + 2], tab[kBiasHead + 3]};
}
// Key tiles closer to the query tile than this hold a distance below R.
__device__ __forceinline__ int near_tiles(int R) { return (R + kTile - 2) / kTile; }
// The bias of query tile t x key tile u for the thread whose column 0 has distance rel0.
__device__ __forceinline__ TileBias tile_bias(const float* tab, const HeadBias& H, int R, int near, int t, int u,
                                              int rel0) {
  TileBias B;
  const bool low = u < t;
  const float sl = low ? H.slope2 : -H.slope2;      // bias per unit of distance
  B.tab = abs(u - t) <= near ? tab + rel0 + R + kBiasReach : nullptr;
  B.c = B.tab ? 0.f : fmaf(sl, (float)rel0, low ? H.lo : H.hi);
  B.col = low ? H.col : -H.col;
  return B;
}

}  // namespace flamia
