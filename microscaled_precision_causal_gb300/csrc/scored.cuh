// Scored attention: what its kernels and the ABI share (parameters, the bucket rule,
// the visible-key sets and the backward's workspace layout).
#pragma once
#include "common.cuh"

namespace flamia {

struct ScoredParams {
  const __nv_bfloat16 *q, *k, *v;
  const int32_t* cu;
  const int* plan;
  const int32_t* prefix;     // [N] or null
  int N, T, hq, hkv;
  float scale;               // softmax scale
  float scale2;              // softmax scale log2 e, with the products' mean truncation taken back
  float cap;                 // 0: none
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
};

struct ScoredBwdWorkspace {
  size_t dvec, drel, total;
};
inline ScoredBwdWorkspace scored_bwd_layout(int64_t T, int N, int hq, int R) {
  auto round256 = [](size_t x) { return (x + 255) & ~size_t(255); };
  ScoredBwdWorkspace w;
  size_t off = 0;
  w.dvec = off;
  off = round256(off + (size_t)T * hq * 4);
  w.drel = off;
  if (R > 0) off = round256(off + (size_t)plan_capacity(T, N) * hq * (2 * R + 1) * 4);
  w.total = off > 0 ? off : 256;
  return w;
}

// The tensor core truncates as it accumulates, so a product of D terms comes out too small
// by a part that does not depend on its size: measured on 65,536 rows of normal values
// -9.9e-8 of the product at D = 128 (eight steps of 16 terms) and -5.5e-8 at D = 64, beside
// a spread of 7e-8.  The score scale takes the mean back; it would enter every probability
// with the score's own size as a factor.
inline double mma_gain(int D) { return D == 128 ? 1.0 + 9.9e-8 : 1.0 + 5.5e-8; }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

// Bias entries below this hide the pair, as -inf does (the lowest float would lose the
// score's own value in the sum and overflow in base 2).
constexpr float kHideBelow = -1.2676506002282294e30f;   // -2^100

// ---------------------------------------------------------------- visible tiles
// Key tiles that a run of query tiles [t0, t1] of a document sees, in increasing order:
// the a tiles of the prefix that lie before the window's first tile, then the n - a tiles
// from lo on (the window's, and prefix tiles behind its first).
struct KeyTiles {
  int a, lo, n;
  __device__ __forceinline__ int tile(int k) const { return k < a ? k : lo + (k - a); }
};
__device__ __forceinline__ KeyTiles key_tiles(int t0, int t1, int nt, int pre_tiles, Window w) {
  KeyTiles s;
  s.lo = win_klo(t0, w);
  s.a = min(pre_tiles, s.lo);
  const int hi = max(win_khi(t1, nt, w), pre_tiles - 1);
  s.n = s.a + hi - s.lo + 1;
  return s;
}
// True when some key of key tile u is hidden from a query of tile t or lies outside the document.
__device__ __forceinline__ bool scored_masked(int t, int u, int len, int pre, Window w) {
  if ((u + 1) * kTile > len) return true;
  return (u + 1) * kTile > pre && win_masked(t, u, len, w);
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
// Clear rows first .. 127 of a TMA-staged [128][D] bf16 tile (64-column boxes): the tile's
// rows behind the document belong to the next one, or to nobody, and may hold anything;
// weight 0 does not silence an infinity.  r: the calling thread's row.
template <int D>
__device__ __forceinline__ void clear_row(uint8_t* tile, int r) {
#pragma unroll
  for (int b = 0; b < D / 64; ++b) {
    uint4* row = reinterpret_cast<uint4*>(tile + b * kTile * 128 + r * 128);
#pragma unroll
    for (int c = 0; c < 8; ++c) row[c] = make_uint4(0, 0, 0, 0);
  }
}

// ---------------------------------------------------------------- scores in base 2
// The kernels hold u log2(e), so that the softmax is 2^x.
//
// tanh cap: y = cap tanh(z), z = s / cap.  Up to |z| = kTanhPolyTo, tanh(z) = z + z w Q(w)
// with w = z^2 and Q of degree 4 (least squares in relative error, reweighted towards equal
// ripple, on Chebyshev nodes of w: 6.5e-8, 1.4e-7 with the fp32 roundings), on the fp32 pipe
// in packed pairs.  Beyond it tanh(z) = 1 - 2 / (1 + 2^(2 z log2 e)), which loses nothing
// there but costs two MUFU operations beside the softmax's own; a warp takes that branch for
// 32 columns when one of its values needs it.
constexpr float kTanhPolyTo = 0.8f;
// z w Q(w) / z = tanh(z) / z - 1.
__device__ __forceinline__ float2 tanh_poly(float2 z) {
  const float2 w = fmul2(z, z);
  auto c = [](float x) { return make_float2(x, x); };
  float2 p = ffma2(w, c(-0.004410882946103811f), c(0.01919075846672058f));
  p = ffma2(w, p, c(-0.053176309913396835f));
  p = ffma2(w, p, c(0.1332276612520218f));
  p = ffma2(w, p, c(-0.3333286643028259f));
  return fmul2(w, p);
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float tanh_any(float z) {
  return fmaf(-2.f, fast_rcp(1.f + fast_exp2(z * (2.f * kLog2e))), 1.f);
}

// Constants of a call.
struct ScoreHead {
  float scale2;     // softmax scale log2 e
  float zscale;     // softmax scale / cap
  float cap2;       // cap log2 e
};
// A tile's bias is a function of the distance: near the diagonal (some distance below R, or
// both signs of it) a value per distance from a staged table; elsewhere a constant, or with a
// slope a constant and a multiple of the column, which is staged too.
struct TileBias {
  const float* tab; // table entry of the thread's column 0, or null
  const float* col; // the slope's part of columns 0 .. 127, or null
  float c;          // the rest, added in the exponent
  __device__ __forceinline__ bool plain() const { return !tab && !col; }
};
__device__ __forceinline__ float2 pair_of(const uint32_t (&v)[32], int j) {
  return make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
}
__device__ __forceinline__ void put_pair(uint32_t (&v)[32], int j, float2 x) {
  v[j] = __float_as_uint(x.x);
  v[j + 1] = __float_as_uint(x.y);
}
// 32 raw products -> cap log2 e tanh(s / cap).
__device__ __forceinline__ void cap_chunk(uint32_t (&v)[32], const ScoreHead& H) {
  float ma = 0.f, mb = 0.f;
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    ma = fmax3(ma, fabsf(__uint_as_float(v[j])), fabsf(__uint_as_float(v[j + 1])));
    mb = fmax3(mb, fabsf(__uint_as_float(v[j + 2])), fabsf(__uint_as_float(v[j + 3])));
  }
  const float mx = fmaxf(ma, mb);
  const float2 zs = make_float2(H.zscale, H.zscale), s2 = make_float2(H.scale2, H.scale2);
  const bool big = __any_sync(0xffffffffu, !(mx * H.zscale <= kTanhPolyTo));
  if (!big) {
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 y = fmul2(pair_of(v, j), s2);
      put_pair(v, j, ffma2(y, tanh_poly(fmul2(pair_of(v, j), zs)), y));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 z = fmul2(pair_of(v, j), zs), y = fmul2(pair_of(v, j), s2);
      float2 t = ffma2(y, tanh_poly(z), y);
      if (!(fabsf(z.x) <= kTanhPolyTo)) t.x = H.cap2 * tanh_any(z.x);
      if (!(fabsf(z.y) <= kTanhPolyTo)) t.y = H.cap2 * tanh_any(z.y);
      put_pair(v, j, t);
    }
  }
}
// x f + the table's or the slope's part for columns c0 .. c0 + 31 (column c: distance DIR c more).
template <int DIR>
__device__ __forceinline__ void bias_chunk(uint32_t (&v)[32], int c0, float f, const TileBias& B) {
  const float2 f2 = make_float2(f, f);
  if (B.tab) {
    const float* tab = B.tab + DIR * c0;
#pragma unroll
    for (int j = 0; j < 32; j += 2) put_pair(v, j, ffma2(pair_of(v, j), f2, make_float2(tab[DIR * j], tab[DIR * (j + 1)])));
  } else if (B.col) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 b = *reinterpret_cast<const float4*>(B.col + c0 + j);
      put_pair(v, j, ffma2(pair_of(v, j), f2, make_float2(b.x, b.y)));
      put_pair(v, j + 2, ffma2(pair_of(v, j + 2), f2, make_float2(b.z, b.w)));
    }
  }
}

// Staged bias of one head in base 2: entry r + R + 255 of the table holds the bias of distance
// r, clipped to R on both sides and long enough for every tile that holds a distance below R,
// so that no index is clipped in the loops.  Without a bias by distance R counts as 1: the
// table then serves the tiles on the diagonal, where a slope's sign changes.
// Before it: the slope times column (128), and its negative (128).
constexpr int kBiasReach = 2 * kTile - 1;
constexpr int kBiasTab = 2 * kTile + 2 * (FLAMIA_REL_MAX + kBiasReach) + 2;
__device__ __forceinline__ float bias_base2(float b) {
  return b < kHideBelow ? -INFINITY : fminf(b, -kHideBelow) * kLog2e;
}
__device__ __forceinline__ int bias_range(const ScoredParams& p) { return p.rel ? p.R : 1; }
__device__ __forceinline__ float head_slope2(const ScoredParams& p, int h) {
  return p.slopes ? p.slopes[h] * kLog2e : 0.f;
}
__device__ __forceinline__ void stage_bias(float* buf, const ScoredParams& p, int h, int first, int stride) {
  const int R = bias_range(p);
  const float slope2 = head_slope2(p, h);
  const float* src = p.rel ? p.rel + (size_t)h * (2 * R + 1) : nullptr;
  for (int i = first; i < 2 * kTile; i += stride) buf[i] = slope2 * (float)(i < kTile ? i : kTile - i);
  for (int i = first; i < 2 * (R + kBiasReach) + 1; i += stride) {
    const float b = src ? bias_base2(src[min(max(i - kBiasReach, 0), 2 * R)]) : 0.f;
    buf[2 * kTile + i] = fmaf(fabsf((float)(i - R - kBiasReach)), -slope2, b);
  }
}
struct HeadBias {
  float slope2, lo, hi;      // slope, and the bias of the distances up to -R and from R on
};
__device__ __forceinline__ HeadBias head_bias(const ScoredParams& p, int h) {
  HeadBias H;
  H.slope2 = head_slope2(p, h);
  H.lo = p.rel ? bias_base2(p.rel[(size_t)h * (2 * p.R + 1)]) : 0.f;
  H.hi = p.rel ? bias_base2(p.rel[(size_t)h * (2 * p.R + 1) + 2 * p.R]) : 0.f;
  return H;
}
// The bias of query tile t x key tile u for the thread whose column 0 has distance rel0.
template <int DIR>
__device__ __forceinline__ TileBias tile_bias(const float* buf, const HeadBias& H, int R, int t, int u, int rel0) {
  const int rmax = (u - t) * kTile + kTile - 1, rmin = (u - t) * kTile - (kTile - 1);
  const float* tab = buf + 2 * kTile;
  TileBias B;
  B.tab = B.col = nullptr;
  B.c = 0.f;
  if (rmax > -R && rmin < R) {
    B.tab = tab + rel0 + R + kBiasReach;
    return B;
  }
  const bool low = rmax <= -R;
  B.c = low ? H.lo : H.hi;
  if (H.slope2 != 0.f) {
    const float sl = low ? H.slope2 : -H.slope2;      // bias per unit of distance
    B.c = fmaf(sl, (float)rel0, B.c);
    B.col = buf + ((low == (DIR > 0)) ? 0 : kTile);
  }
  return B;
}

}  // namespace flamia
