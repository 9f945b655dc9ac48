// Scored attention, backward: one warp per row, fp32 throughout.
//
// For query i and key j of a document:  s = scale q_i . k_j,  t = cap tanh(s / cap),
// u = t - slope |j - i| + rel[clamp(j - i)];  O_i = sum_j softmax_j(u_ij) v_j with a running
// maximum and sum; backward P = exp(u - LSE), dU = P o (dO V^T - D), dS = dU (1 - tanh^2).
#include "scored.cuh"

namespace flamia {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int D>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, int lane, float (&r)[D / 32]) {
#pragma unroll
  for (int e = 0; e < D / 32; ++e) r[e] = __bfloat162float(p[lane * (D / 32) + e]);
}
template <int D>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, int lane, const float (&r)[D / 32], float f) {
#pragma unroll
  for (int e = 0; e < D / 32; ++e) p[lane * (D / 32) + e] = __float2bfloat16(r[e] * f);
}
template <int D>
__device__ __forceinline__ float dot(const float (&a)[D / 32], const float (&b)[D / 32]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) s = fmaf(a[e], b[e], s);
  return warp_sum(s);
}

// Row -> document-local position; false for a row outside every document.
struct Row {
  int start, len, pos, pre;
};
__device__ __forceinline__ bool find_row(const ScoredParams& p, int t, Row& r) {
  if (t >= p.plan[kPlanValid]) return false;
  const int n = upper_doc(p.cu, p.N, t);
  r.start = p.cu[n];
  r.len = p.cu[n + 1] - r.start;
  r.pos = t - r.start;
  r.pre = p.prefix ? min(max(p.prefix[n], 0), r.len) : 0;
  return true;
}
__device__ __forceinline__ bool visible(const ScoredParams& p, int i, int j, int pre) {
  return j < pre || ((p.win.left < 0 || j >= i - p.win.left) && (p.win.right < 0 || j <= i + p.win.right));
}
// u of one pair and, for the backward, 1 - tanh^2.
__device__ __forceinline__ float score(const ScoredParams& p, float dotp, int h, int rel, float& g) {
  float u = dotp * p.scale;
  g = 1.f;
  if (p.cap > 0.f) {
    const float th = tanhf(u / p.cap);
    u = p.cap * th;
    g = 1.f - th * th;
  }
  if (p.slopes) u -= p.slopes[h] * fabsf((float)rel);
  if (p.rel) {
    const float b = p.rel[(size_t)h * (2 * p.R + 1) + min(max(rel, -p.R), p.R) + p.R];
    u = b < kHideBelow ? -INFINITY : u + b;
  }
  return u;
}

template <int D>
__global__ void scored_dvec_kernel(const ScoredParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id >= (int64_t)p.T * p.hq) return;
  float a[D / 32], b[D / 32];
  load_row<D>(p.out + id * D, lane, a);
  load_row<D>(p.dout + id * D, lane, b);
  const float s = dot<D>(a, b);
  if (lane == 0) p.dvec[(id % p.hq) * p.T + id / p.hq] = s;
}

template <int D>
__global__ void scored_dq_kernel(const ScoredParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id >= (int64_t)p.T * p.hq) return;
  const int t = (int)(id / p.hq), h = (int)(id % p.hq), hk = h / (p.hq / p.hkv);
  Row r;
  float dq[D / 32] = {};
  if (find_row(p, t, r)) {
    float q[D / 32], k[D / 32], v[D / 32], gr[D / 32], g;
    load_row<D>(p.q + id * D, lane, q);
    load_row<D>(p.dout + id * D, lane, gr);
    const float lse = p.lse[(int64_t)h * p.T + t], dv = p.dvec[(int64_t)h * p.T + t];
    for (int j = 0; j < r.len; ++j) {
      if (!visible(p, r.pos, j, r.pre)) continue;
      const int64_t kr = ((int64_t)(r.start + j) * p.hkv + hk) * D;
      load_row<D>(p.k + kr, lane, k);
      load_row<D>(p.v + kr, lane, v);
      const float u = score(p, dot<D>(q, k), h, j - r.pos, g);
      const float e = u == -INFINITY ? 0.f : expf(u - lse);
      const float du = e * (dot<D>(gr, v) - dv);
      if (p.drel && lane == 0)
        atomicAdd(p.drel + (size_t)h * (2 * p.R + 1) + min(max(j - r.pos, -p.R), p.R) + p.R, du);
      const float ds = du * g * p.scale;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) dq[x] = fmaf(ds, k[x], dq[x]);
    }
  }
  store_row<D>(p.dq + id * D, lane, dq, 1.f);
}

template <int D>
__global__ void scored_dkv_kernel(const ScoredParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id >= (int64_t)p.T * p.hkv) return;
  const int t = (int)(id / p.hkv), hk = (int)(id % p.hkv), group = p.hq / p.hkv;
  Row r;
  float dk[D / 32] = {}, dv[D / 32] = {};
  if (find_row(p, t, r)) {
    float q[D / 32], k[D / 32], v[D / 32], gr[D / 32], g;
    load_row<D>(p.k + id * D, lane, k);
    load_row<D>(p.v + id * D, lane, v);
    for (int h = hk * group; h < (hk + 1) * group; ++h) {
      for (int i = 0; i < r.len; ++i) {
        if (!visible(p, i, r.pos, r.pre)) continue;
        const int64_t tq = r.start + i, qr = (tq * p.hq + h) * D;
        load_row<D>(p.q + qr, lane, q);
        load_row<D>(p.dout + qr, lane, gr);
        const float u = score(p, dot<D>(q, k), h, r.pos - i, g);
        const float e = u == -INFINITY ? 0.f : expf(u - p.lse[(int64_t)h * p.T + tq]);
        const float ds = e * (dot<D>(gr, v) - p.dvec[(int64_t)h * p.T + tq]) * g * p.scale;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          dv[x] = fmaf(e, gr[x], dv[x]);
          dk[x] = fmaf(ds, q[x], dk[x]);
        }
      }
    }
  }
  store_row<D>(p.dk + id * D, lane, dk, 1.f);
  store_row<D>(p.dv + id * D, lane, dv, 1.f);
}

inline unsigned blocks(int64_t rows) { return (unsigned)((rows + kWarps - 1) / kWarps); }

template <int D>
cudaError_t bwd_d(const ScoredParams& p, cudaStream_t s) {
  const int64_t rq = (int64_t)p.T * p.hq, rk = (int64_t)p.T * p.hkv;
  if (p.drel) {
    const cudaError_t e = cudaMemsetAsync(p.drel, 0, (size_t)p.hq * (2 * p.R + 1) * 4, s);
    if (e != cudaSuccess) return e;
  }
  scored_dvec_kernel<D><<<blocks(rq), kWarps * 32, 0, s>>>(p);
  scored_dq_kernel<D><<<blocks(rq), kWarps * 32, 0, s>>>(p);
  scored_dkv_kernel<D><<<blocks(rk), kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scored_bwd(int D, const ScoredParams& p, cudaStream_t s) {
  if ((int64_t)p.T * p.hq > 0x7fffffffLL * kWarps) return cudaErrorInvalidValue;
  return D == 128 ? bwd_d<128>(p, s) : bwd_d<64>(p, s);
}

}  // namespace flamia
