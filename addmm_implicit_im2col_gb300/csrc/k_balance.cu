// The routers' balance loss with the experts' counts, and the gradient of the logits:
//
//   loss[s] = E / (k n^2) * sum_e c[s,e] * sum_t p[t,e]
//
// over the n tokens of sequence s, c[s,e] of whose slots chose expert e; p are the
// softmax scores, or the sigmoid scores divided by their sum.
#include "adapters.cuh"
#include "ptx.cuh"
#include "scores.cuh"

namespace imc {
namespace mx {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kFlush = 64;  // tokens whose scores a lane sums in fp32

__device__ __forceinline__ int64_t clamped(int64_t v, int64_t T) { return v < 0 ? 0 : (v > T ? T : v); }

// Divides the scores of a token by their sum (sigmoid; softmax scores have the sum 1).
// Returns 1 / sum.
template <int VPT>
__device__ __forceinline__ float normalise(float (&s)[VPT]) {
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) sum += s[j];
  sum = warp_sum(sum);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int j = 0; j < VPT; ++j) s[j] *= inv;
  return inv;
}

// One cluster of CTAs per sequence, a warp per token.  A lane sums its experts' scores
// of kFlush tokens in fp32, then in 64 bits: an error of a few fp32 roundings however
// long the sequence is.  Every sum has a fixed order; the counts are whole numbers.
template <int VPT, typename T>
__global__ void __launch_bounds__(kThreads) k_balance(const BalanceArgs a, const int log_ctas) {
  extern __shared__ double sm_sums[];  // [warp][E], then (CTA 0) [CTA][E]
  const int E = a.E, C = 1 << log_ctas, rank = (int)ptx::cluster_rank();
  double* gathered = sm_sums + kWarps * E;
  int32_t* count = reinterpret_cast<int32_t*>(gathered + C * E);  // [E], then (CTA 0) [CTA][E]
  int32_t* counts = count + E;
  __shared__ double loss[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, s = blockIdx.x >> log_ctas;
  ptx::cluster_arrive();
  for (int i = threadIdx.x; i < kWarps * E; i += kThreads) sm_sums[i] = 0.0;
  for (int i = threadIdx.x; i < E; i += kThreads) count[i] = 0;
  __syncthreads();
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int64_t t0 = a.offsets ? clamped(a.offsets[s], a.T) : 0;
  const int64_t t1 = a.offsets ? clamped(a.offsets[s + 1], a.T) : a.T;
  double* mine = sm_sums + warp * E;
  float acc[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) acc[j] = 0.0f;
  auto flush = [&] {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (lane + 32 * j < E) mine[lane + 32 * j] += acc[j];
      acc[j] = 0.0f;
    }
  };
  int held = 0;
  for (int64_t t = t0 + rank * kWarps + warp; t < t1; t += (int64_t)C * kWarps) {
    if (lane < a.k) {
      const int e = __ldg(a.experts + t * a.k + lane);
      if (e >= 0 && e < E) atomicAdd(count + e, 1);
    }
    float v[VPT];
    scores<VPT, T>(static_cast<const T*>(a.logits) + t * a.ld, E, a.sigmoid, v);
    if (a.sigmoid) normalise<VPT>(v);
#pragma unroll
    for (int j = 0; j < VPT; ++j) acc[j] += v[j];
    if (++held == kFlush) {
      flush();
      held = 0;
    }
  }
  flush();
  __syncthreads();
  ptx::cluster_wait();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sm_sums[w * E + e];
    const uint32_t at = ptx::cluster_addr(gathered + rank * E + e, 0);
    ptx::st_cluster(at, (uint32_t)__double2loint(sum));
    ptx::st_cluster(at + 4, (uint32_t)__double2hiint(sum));
    ptx::st_cluster(ptx::cluster_addr(counts + rank * E + e, 0), (uint32_t)count[e]);
  }
  ptx::cluster_sync();
  if (rank) return;
  double part = 0.0;
  for (int e = threadIdx.x; e < E; e += kThreads) {
    double sum = 0.0;
    int32_t c = 0;
    for (int q = 0; q < C; ++q) {
      sum += gathered[q * E + e];
      c += counts[q * E + e];
    }
    a.counts[(int64_t)s * E + e] = c;
    part += sum * c;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) part += __shfl_xor_sync(kAll, part, d);
  if (lane == 0) loss[warp] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += loss[w];
    const double n = (double)(t1 - t0);
    a.loss[s] = t1 > t0 ? (float)(sum * E / (a.k * n * n)) : 0.0f;
  }
}

// The sequence of token t: the number of offsets that are at most t, less one (a warp's
// lanes look at 32 places at once).
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, int64_t t) {
  const int lane = threadIdx.x & 31;
  int low = 0, n = S + 1;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const bool in = lane * step < n;
    const int c = __popc(__ballot_sync(kAll, in && __ldg(offsets + low + lane * step) <= t));
    if (c == 0) break;
    const int past = (c - 1) * step + 1;
    low += past;
    n = min(step - 1, n - past);
  }
  return low - 1;
}

// A warp per token.  With u_e = grad_loss[s] * E / (k n^2) * c[s,e], the counts constant,
//   softmax: dx_e = p_e (u_e - sum u p),  sigmoid: dx_e = s_e (1 - s_e) / sum s * (u_e - sum u p);
// with grad_weights the gradient of the routing weights (k_route_backward's) is added
// before the one rounding to the logits' type.
template <int VPT, typename T>
__global__ void __launch_bounds__(128) k_balance_backward(const BalanceArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
  const int64_t t = (int64_t)blockIdx.x * 4 + warp;
  if (t >= a.T) return;
  int id = -1;
  float gi = 0.0f;
  if (a.grad_weights && lane < a.k) {
    id = a.experts[t * a.k + lane];
    gi = a.grad_weights[t * a.k + lane];
    if (id < 0 || id >= E) id = -1;
  }
  // rest: the derivative of a score with respect to its logit without the softmax's sum.
  // 1 - s is taken from exp(-|x|), not from s, which is 1 to fp32's precision for x of 17.
  float s[VPT], u[VPT], rest[VPT];
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const float x = lane + 32 * j < E ? to_f32<T>(row[lane + 32 * j]) : -INFINITY;
      const float small = expf(-fabsf(x)), inv = 1.0f / (1.0f + small);
      s[j] = x < 0.0f ? small * inv : inv;
      rest[j] = small * inv * inv;
    }
  } else {
    scores<VPT, T>(row, E, 0, s);
#pragma unroll
    for (int j = 0; j < VPT; ++j) rest[j] = s[j];
  }
  const int q = a.offsets ? sequence_of(a.offsets, a.S, t) : 0;
  float coef = 0.0f;
  if (q >= 0 && q < a.S) {
    const int64_t t0 = a.offsets ? clamped(a.offsets[q], a.T) : 0;
    const int64_t t1 = a.offsets ? clamped(a.offsets[q + 1], a.T) : a.T;
    const float n = (float)(t1 - t0);
    coef = a.grad_loss[q] * ((float)E / ((float)a.k * n) / n);
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = lane + 32 * j;
    u[j] = coef != 0.0f && e < E ? coef * (float)__ldg(a.counts + (int64_t)q * E + e) : 0.0f;
  }
  // the balance loss: d = u - sum u p, over the sum of the scores
  float sum = 0.0f, dot = 0.0f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    sum += s[j];
    dot += u[j] * s[j];
  }
  dot = warp_sum(dot);
  float inv = 1.0f;
  if (a.sigmoid) {
    sum = warp_sum(sum);
    inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  }
  dot *= inv;
#pragma unroll
  for (int j = 0; j < VPT; ++j) u[j] = (u[j] - dot) * inv;
  // the weights
  if (a.grad_weights) {
    float total = 0.0f, along = 0.0f, si = 0.0f;
    for (int i = 0; i < a.k; ++i) {
      const int e = __shfl_sync(kAll, id, i);
      if (e < 0) continue;
      const float p = __shfl_sync(kAll, pick<VPT>(s, e >> 5), e & 31);
      total += p;
      along += p * __shfl_sync(kAll, gi, i);
      if (lane == i) si = p;
    }
    float di = id >= 0 ? gi : 0.0f;
    if (a.renorm) di = total == 0.0f || id < 0 ? 0.0f : (gi - along / total) / total;
    di *= a.scale;
    const float inner = a.sigmoid ? 0.0f : warp_sum(di * si);
#pragma unroll
    for (int j = 0; j < VPT; ++j) u[j] -= inner;
    for (int i = 0; i < a.k; ++i) {
      const int e = __shfl_sync(kAll, id, i);
      const float v = __shfl_sync(kAll, di, i);
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (e == lane + 32 * j) u[j] += v;
    }
  }
  T* grad = static_cast<T*>(a.grad) + t * E;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = lane + 32 * j;
    if (e < E) grad[e] = from_f32<T>(u[j] * rest[j]);
  }
}

// ------------------------------------------------------------------- host
template <int VPT, typename T>
cudaError_t forward(const BalanceArgs& a, cudaStream_t s) {
  const int log_ctas = 3;
  const size_t smem = (size_t)a.E * (kWarps + (1 << log_ctas)) * 8 + (size_t)a.E * (1 + (1 << log_ctas)) * 4;
  cudaError_t e = cudaFuncSetAttribute(k_balance<VPT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.S << log_ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1u << log_ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, k_balance<VPT, T>, a, log_ctas);
  note_launch();
  return e;
}

template <int VPT, typename T>
cudaError_t backward(const BalanceArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_after_previous(k_balance_backward<VPT, T>, dim3((unsigned)ceil_div(a.T, 4)),
                                              dim3(128), 0, s, a);
  note_launch();
  return e;
}

template <typename T>
cudaError_t of_size(const BalanceArgs& a, bool back, cudaStream_t s) {
#define IMC_BALANCE(V) return back ? backward<V, T>(a, s) : forward<V, T>(a, s)
  if (a.E <= 32) IMC_BALANCE(1);
  if (a.E <= 64) IMC_BALANCE(2);
  if (a.E <= 128) IMC_BALANCE(4);
  if (a.E <= 256) IMC_BALANCE(8);
  if (a.E <= 512) IMC_BALANCE(16);
  IMC_BALANCE(32);
#undef IMC_BALANCE
}

cudaError_t of_type(const BalanceArgs& a, int dtype, bool back, cudaStream_t s) {
  if (dtype == IMC_F32) return of_size<float>(a, back, s);
  if (dtype == IMC_F16) return of_size<__half>(a, back, s);
  return of_size<__nv_bfloat16>(a, back, s);
}

}  // namespace

cudaError_t launch_balance(const BalanceArgs& a, int dtype, cudaStream_t s) {
  note_kernel_name("k_balance");
  return of_type(a, dtype, false, s);
}

cudaError_t launch_balance_backward(const BalanceArgs& a, int dtype, cudaStream_t s) {
  note_kernel_name("k_balance_backward");
  return of_type(a, dtype, true, s);
}

}  // namespace mx
}  // namespace imc
