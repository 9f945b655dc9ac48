// Attention of new tokens over the paged cache: steps by the step kernel, the others a warp per query row and head,
// keys one by one in fp32.
#include "cache.cuh"

namespace flamia {

cudaError_t launch_cached_step(int D, bool e4m3, const CachedParams& p, cudaStream_t s);
cudaError_t launch_cached_join(int D, bool step, const CachedParams& p, cudaStream_t s);

namespace {

constexpr int kWarps = 8;

template <int D, bool E4M3>
__device__ __forceinline__ void load_row(const uint8_t* pool, const uint8_t* scales, int64_t at, int lane, float* x) {
  constexpr int kPer = D / 32;
  if constexpr (E4M3) {
    const float f = cache_scale(scales[at]);
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = e4m3_to_f32(pool[at * D + lane * kPer + i]) * f;
  } else {
    const __nv_bfloat16* r = reinterpret_cast<const __nv_bfloat16*>(pool) + at * D + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = __bfloat162float(r[i]);
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) cached_rows_kernel(const CachedParams p) {
  constexpr int kPer = D / 32;
  const int64_t job = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (job >= (int64_t)p.c.T * p.hq) return;
  const int lane = threadIdx.x & 31, row = (int)(job / p.hq), h = (int)(job % p.hq), hk = h / (p.hq / p.c.hkv);
  float o[kPer] = {}, q[kPer];
  float m = -INFINITY, l = 0.f;
  const bool in = row < cached_valid_rows(p);
  if (in) {
    const int4* seq = reinterpret_cast<const int4*>(p.c.plan + kCpHeaderWords);
    const int n = warp_upper(p.c.N, row, [&](int i) { return seq[i].x; });
    const int4 r = seq[n];
    const int pos = r.z - r.y + row - r.x;
    if (r.y * (p.hq / p.c.hkv) <= kStepRows) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i) q[i] = __bfloat162float(p.q[((int64_t)row * p.hq + h) * D + lane * kPer + i]);
    for (int j = p.left < 0 ? 0 : max(0, pos - p.left); j <= pos; ++j) {
      const int page = cache_page(p.c, n, j >> p.c.page_shift);
      if (page < 0) continue;
      const int64_t at = (((int64_t)page * p.c.hkv + hk) << p.c.page_shift) + (j & ((1 << p.c.page_shift) - 1));
      float x[kPer], s = 0.f;
      load_row<D, E4M3>(p.c.k, p.c.k_scales, at, lane, x);
#pragma unroll
      for (int i = 0; i < kPer; ++i) s = fmaf(q[i], x[i], s);
#pragma unroll
      for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      if (p.cap > 0.f) s = p.capf.inv * tanhf(s * p.capf.zscale);
      s *= p.scale2;
      const float top = fmaxf(m, s), a = exp2f(m - top), e = exp2f(s - top);
      m = top;
      l = l * a + e;
      load_row<D, E4M3>(p.c.v, p.c.v_scales, at, lane, x);
#pragma unroll
      for (int i = 0; i < kPer; ++i) o[i] = o[i] * a + e * x[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    p.out[((int64_t)row * p.hq + h) * D + lane * kPer + i] = __float2bfloat16(in && l != 0.f ? o[i] / l : 0.f);
  if (lane == 0) p.lse[(int64_t)h * p.c.T + row] = in && l != 0.f ? (m + log2f(l)) * kLn2 : INFINITY;
}

}  // namespace

cudaError_t launch_cached_fwd(int D, bool e4m3, const CachedParams& p, cudaStream_t s) {
  const int group = p.hq / p.c.hkv;
  if (group <= kStepRows) {
    cudaError_t e = launch_cached_step(D, e4m3, p, s);
    if (e == cudaSuccess) e = launch_cached_join(D, true, p, s);
    if (e != cudaSuccess || (int64_t)p.max_chunk * group <= kStepRows) return e;
  }
  const int64_t blocks = ((int64_t)p.c.T * p.hq + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const auto f = D == 128 ? (e4m3 ? cached_rows_kernel<128, true> : cached_rows_kernel<128, false>)
                          : (e4m3 ? cached_rows_kernel<64, true> : cached_rows_kernel<64, false>);
  f<<<(unsigned)blocks, kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace flamia
