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

// Bias entries below this hide the pair, as -inf does (the lowest float would lose the
// score's own value in the sum and overflow in base 2).
constexpr float kHideBelow = -1.2676506002282294e30f;   // -2^100

}  // namespace flamia
