// Bucketed relative position bias: a table [buckets, heads] spread over the clipped
// distances (expand), and a gradient by clipped distance summed back (reduce).
//
// A pair's bucket depends on its distance only, and from max_distance on it stays the
// same, so the scored attention kernels see a bias by clipped distance: 2R + 1 floats a
// head instead of a bucket per pair.  Both kernels touch a few KB (32 buckets, 16 heads,
// R = 128: 16 KB each) and are bound by their launch.
#include <cmath>

#include "common.cuh"

namespace flamia {

namespace {

struct Buckets {
  int nb, md, both;
  double per_log;      // far buckets per unit of the logarithm
};
Buckets make_buckets(int nb, int md, int both) {
  const int side = both ? nb / 2 : nb, e = side / 2;
  return {nb, md, both, (side - e) / std::log((double)md / e)};
}

// Bucket of distance r (key minus query).  The logarithm is in 64 bits: a distance n with
// (n / e) ^ (B - e) a whole power of max_distance / e lies on a bucket's border, and 2^-36
// puts it into the upper bucket whatever the last bits of the product.  Over every B up to 1024,
// max_distance up to 1024 and n (whole numbers decide what is a border) the product's error
// there is at most 5e-13, and the nearest distance below a border lies 3.7e-10 from it (B 73,
// max_distance 905, n 347): 2^-36, 1.5e-11, is between.
__device__ int rel_bucket(int r, const Buckets& B) {
  int base = 0, n, nb = B.nb;
  if (B.both) {
    nb >>= 1;
    base = r > 0 ? nb : 0;
    n = r < 0 ? -r : r;
  } else {
    n = r < 0 ? -r : 0;
  }
  const int e = nb >> 1;
  if (n < e) return base + n;
  if (n >= B.md) return base + nb - 1;
  const int b = e + (int)floor(log((double)n / e) * B.per_log + 0x1p-36);
  return base + (b < nb - 1 ? b : nb - 1);
}

__global__ void relbias_expand_kernel(const float* __restrict__ table, int hq, Buckets B, float* __restrict__ rel,
                                      int R) {
  const int width = 2 * R + 1;
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= width) return;
  const int b = rel_bucket(i - R, B);
  for (int h = blockIdx.y; h < hq; h += gridDim.y) rel[(size_t)h * width + i] = table[(size_t)b * hq + h];
}

// One block per head: the entries' buckets go to shared memory, then a warp sums a bucket at
// a time, lane l the distances l, l + 32, ... in order, and the lanes' sums in a fixed tree.
__global__ void __launch_bounds__(512) relbias_reduce_kernel(const float* __restrict__ drel, int R, int hq, Buckets B,
                                                             float* __restrict__ dtable) {
  __shared__ float val[2 * FLAMIA_REL_MAX + 1];
  __shared__ short id[2 * FLAMIA_REL_MAX + 1];
  const int width = 2 * R + 1, h = blockIdx.x;
  for (int i = threadIdx.x; i < width; i += blockDim.x) {
    val[i] = drel[(size_t)h * width + i];
    id[i] = (short)rel_bucket(i - R, B);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int b = threadIdx.x >> 5; b < B.nb; b += blockDim.x >> 5) {
    float s = 0.f;
    for (int i = lane; i < width; i += 32)
      if (id[i] == b) s += val[i];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) dtable[(size_t)b * hq + h] = s;
  }
}

}  // namespace

cudaError_t launch_relbias_expand(const float* table, int nb, int hq, int md, int both, float* rel, int R,
                                  cudaStream_t s) {
  const dim3 grid((2 * R + 1 + 127) / 128, hq < 128 ? hq : 128);
  relbias_expand_kernel<<<grid, 128, 0, s>>>(table, hq, make_buckets(nb, md, both), rel, R);
  return cudaGetLastError();
}

cudaError_t launch_relbias_reduce(const float* drel, int R, int nb, int hq, int md, int both, float* dtable,
                                  cudaStream_t s) {
  relbias_reduce_kernel<<<hq, 512, 0, s>>>(drel, R, hq, make_buckets(nb, md, both), dtable);
  return cudaGetLastError();
}

}  // namespace flamia
