// A token's scores in the registers of a warp: what routing, its gradient and the
// balance loss share.
#pragma once

#include "mx_internal.cuh"

namespace imc {
namespace mx {

constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// Scores of one token from its logits (-inf where there is no expert): lane l holds experts
// l, l + 32, ... (VPT of them).  softmax: exp(x - max) / sum; a row of -inf alone has scores 0.
template <int VPT>
__device__ __forceinline__ void scores_of(int sigmoid, float (&s)[VPT]) {
  if (sigmoid) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) s[j] = 1.0f / (1.0f + expf(-s[j]));
  } else {
    float m = s[0];
#pragma unroll
    for (int j = 1; j < VPT; ++j) m = fmaxf(m, s[j]);
    m = warp_max(m);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      s[j] = m == -INFINITY && s[j] == m ? 0.0f : expf(s[j] - m);
      sum += s[j];
    }
    sum = warp_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int j = 0; j < VPT; ++j) s[j] *= inv;
  }
}
template <int VPT, typename T>
__device__ __forceinline__ void scores(const T* row, int E, int sigmoid, float (&s)[VPT]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = lane + 32 * j;
    s[j] = e < E ? to_f32<T>(row[e]) : -INFINITY;
  }
  scores_of<VPT>(sigmoid, s);
}

// The chosen experts' scores may be far below 1 (chosen by a bias, say): one over their sum, in
// the gradient of the weights, passes fp32's range for sums below 2^-128, the product with a score
// does not.  Below this sum the gradient of a weight is divided by 2^64 until it has met its score.
constexpr float kSmallChosen = 0x1p-64f;

template <int VPT>
__device__ __forceinline__ float pick(const float (&s)[VPT], int j) {
  float v = s[0];
#pragma unroll
  for (int i = 1; i < VPT; ++i)
    if (i == j) v = s[i];
  return v;
}

}  // namespace mx
}  // namespace imc
