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

// A sum as two fp32 numbers, exact to 2^-46 or so of its terms' magnitudes: 64-bit adds run
// at a 64th of the fp32 rate here (with them a chunk's sums took 2 us more, and a sequence's
// loss 1 to 2.5).  The steps that give a rounding error exactly are not the compiler's to
// contract: a product taken unrounded into one of them would enter its error twice.
struct Sum {
  float hi, lo;
  __device__ __forceinline__ void add(float v) {
    const float t = __fadd_rn(hi, v), z = __fsub_rn(t, hi);
    lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(t, z)), __fsub_rn(v, z));
    hi = t;
  }
  __device__ __forceinline__ void add(const Sum& o) {
    add(o.hi);
    lo += o.lo;
  }
  __device__ __forceinline__ void add_times(const Sum& o, float c) {
    const float v = __fmul_rn(o.hi, c);
    add(v);
    lo += fmaf(o.hi, c, -v) + o.lo * c;
  }
  // the warp's sum, the same in lane 0 whatever the timing
  __device__ __forceinline__ void over_lanes() {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const Sum o = {__shfl_xor_sync(kAll, hi, d), __shfl_xor_sync(kAll, lo, d)};
      add(o);
    }
  }
};

// 1 / (1 + e^-x) and, times e^-x over 1 + e^-x, its derivative: 1 - s is taken from
// e^-|x|, not from s, which is 1 to fp32's precision for x of 17.
__device__ __forceinline__ float sigmoid(float x, float& rest) {
  const float small = expf(-fabsf(x)), inv = __fdividef(1.0f, 1.0f + small), low = small * inv;
  rest = low * inv;
  return x < 0.0f ? low : inv;
}

// Sigmoids that sum to less than this are e^x to fp32's precision each, and divided by their sum
// the softmax, which is what such a token's scores are made by: the sigmoids lose bits below
// 2^-126, and a sum below 2^-128 has no reciprocal in fp32.  (A row of -inf alone: zeros.)
constexpr float kSmallSum = 0x1p-100f;

// The logits of one token, -inf where there is no expert: lane l has experts l, l + 32, ...
template <int VPT, typename T>
__device__ __forceinline__ void load_logits(const T* row, int E, float (&v)[VPT]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < VPT; ++j) v[j] = lane + 32 * j < E ? to_f32<T>(row[lane + 32 * j]) : -INFINITY;
}

// The tokens first, first + step, ... before `last`, two of them at a time (their loads and
// sums overlap): their scores are added to mine [E], their slots counted in count [E].  A
// lane sums its experts' scores of kFlush tokens in fp32 before: an error of a few fp32
// roundings however long the sequence is.
template <int VPT, typename T>
__device__ __forceinline__ void add_tokens(const BalanceArgs& a, int64_t first, int64_t last, int64_t step,
                                           Sum* mine, int32_t* count) {
  constexpr int U = VPT <= 8 ? 2 : 1;
  const int lane = threadIdx.x & 31, E = a.E;
  float acc[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) acc[j] = 0.0f;
  auto flush = [&] {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (lane + 32 * j < E) mine[lane + 32 * j].add(acc[j]);
      acc[j] = 0.0f;
    }
  };
  int held = 0;
  for (int64_t t0 = first; t0 < last; t0 += U * step) {
    float v[U][VPT];
    int e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * step;
      const T* row = static_cast<const T*>(a.logits) + t * a.ld;
      e[u] = t < last && lane < a.k ? __ldg(a.experts + t * a.k + lane) : -1;
#pragma unroll
      for (int j = 0; j < VPT; ++j) v[u][j] = t < last && lane + 32 * j < E ? to_f32<T>(row[lane + 32 * j]) : -INFINITY;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (e[u] >= 0 && e[u] < E) atomicAdd(count + e[u], 1);
      if (a.sigmoid) {  // over their sum
        float sum = 0.0f, rest;
#pragma unroll
        for (int j = 0; j < VPT; ++j) sum += v[u][j] = sigmoid(v[u][j], rest);
        sum = warp_sum(sum);
        const int64_t t = t0 + u * step;
        if (sum < kSmallSum && t < last) {  // the whole warp
          load_logits<VPT>(static_cast<const T*>(a.logits) + t * a.ld, E, v[u]);
          scores_of<VPT>(0, v[u]);
        } else {
          const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // (0: no token)
#pragma unroll
          for (int j = 0; j < VPT; ++j) v[u][j] *= inv;
        }
      } else {
        scores_of<VPT>(0, v[u]);
      }
#pragma unroll
      for (int j = 0; j < VPT; ++j) acc[j] += v[u][j];  // (no token: scores of 0)
    }
    held += U;
    if (held >= kFlush) {
      flush();
      held = 0;
    }
  }
  flush();
}

// What a cluster's CTAs have summed for sequence s (sums and counts [E] of each, in its
// shared memory), in the order of the CTAs: counts and loss, by CTA 0.  All threads of the
// cluster; n tokens.
template <int THREADS = kThreads>
__device__ __forceinline__ void finish(const BalanceArgs& a, int s, int64_t n, int C, int rank, const Sum* sums,
                                       const int32_t* count, Sum* gathered, int32_t* counts) {
  __shared__ Sum loss[THREADS / 32];
  const int E = a.E, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < E; e += THREADS) {
    const uint32_t at = ptx::cluster_addr(gathered + rank * E + e, 0);
    ptx::st_cluster(at, __float_as_uint(sums[e].hi));
    ptx::st_cluster(at + 4, __float_as_uint(sums[e].lo));
    ptx::st_cluster(ptx::cluster_addr(counts + rank * E + e, 0), (uint32_t)count[e]);
  }
  ptx::cluster_sync();
  if (rank) return;
  Sum part = {0.0f, 0.0f};
  for (int e = threadIdx.x; e < E; e += THREADS) {
    Sum sum = {0.0f, 0.0f};
    int32_t c = 0;
    for (int q = 0; q < C; ++q) {
      sum.add(gathered[q * E + e]);
      c += counts[q * E + e];
    }
    a.counts[(int64_t)s * E + e] = c;
    part.add_times(sum, (float)c);
  }
  part.over_lanes();
  if (lane == 0) loss[warp] = part;
  __syncthreads();
  if (warp) return;
  part = lane < THREADS / 32 ? loss[lane] : Sum{0.0f, 0.0f};
  part.over_lanes();
  if (lane == 0) a.loss[s] = n > 0 ? (part.hi + part.lo) * ((float)E / ((float)a.k * (float)n) / (float)n) : 0.0f;
}

// Sums of the block's warps [warp][E], into the first one's place.
__device__ __forceinline__ void over_warps(Sum* sums, int E) {
  for (int e = threadIdx.x; e < E; e += kThreads) {
    Sum sum = sums[e];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) sum.add(sums[w * E + e]);
    sums[e] = sum;
  }
}

// One cluster of CTAs per sequence.  Every sum has a fixed order; counts are whole numbers.
template <int VPT, typename T>
__global__ void __launch_bounds__(kThreads) k_balance(const BalanceArgs a, const int log_ctas) {
  extern __shared__ Sum sm_sums[];  // [warp][E], then (CTA 0) [CTA][E]
  const int E = a.E, C = 1 << log_ctas, rank = (int)ptx::cluster_rank();
  Sum* gathered = sm_sums + kWarps * E;
  int32_t* count = reinterpret_cast<int32_t*>(gathered + C * E);  // [E], then (CTA 0) [CTA][E]
  const int warp = threadIdx.x >> 5, s = blockIdx.x >> log_ctas;
  ptx::cluster_arrive();  // this CTA runs: its shared memory may be written
  for (int i = threadIdx.x; i < kWarps * E; i += kThreads) sm_sums[i] = {0.0f, 0.0f};
  for (int i = threadIdx.x; i < E; i += kThreads) count[i] = 0;
  __syncthreads();
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int64_t t0 = a.offsets ? clamped(a.offsets[s], a.T) : 0;
  const int64_t t1 = a.offsets ? clamped(a.offsets[s + 1], a.T) : a.T;
  add_tokens<VPT, T>(a, t0 + rank * kWarps + warp, t1, C * kWarps, sm_sums + warp * E, count);
  __syncthreads();
  over_warps(sm_sums, E);
  ptx::cluster_wait();
  finish(a, s, t1 - t0, C, rank, sm_sums, count, gathered, count + E);
}

// Many tokens: a CTA for each `chunk` of them.  Where chunk c and sequence s meet, their
// sums and counts go to row c + s of the workspace; along the tokens c or s grows from one
// meeting to the next, so a row is written once.
template <int VPT, typename T>
__global__ void __launch_bounds__(kThreads) k_balance_chunks(const BalanceArgs a, const int chunk) {
  extern __shared__ Sum sm_sums[];  // [warp][E]
  const int E = a.E, warp = threadIdx.x >> 5;
  int32_t* count = reinterpret_cast<int32_t*>(sm_sums + kWarps * E);
  const int64_t rows = (int64_t)gridDim.x + a.S;
  Sum* sums = static_cast<Sum*>(a.workspace);
  int32_t* counts = reinterpret_cast<int32_t*>(sums + rows * E);
  for (int i = threadIdx.x; i < kWarps * E; i += kThreads) sm_sums[i] = {0.0f, 0.0f};
  for (int i = threadIdx.x; i < E; i += kThreads) count[i] = 0;
  __syncthreads();
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int64_t end = (int64_t)(blockIdx.x + 1) * chunk < a.T ? (int64_t)(blockIdx.x + 1) * chunk : a.T;
  int64_t t = (int64_t)blockIdx.x * chunk;
  if (a.offsets && t < clamped(a.offsets[0], a.T)) t = clamped(a.offsets[0], a.T);
  while (t < end) {
    const int s = a.offsets ? sequence_of(a.offsets, a.S, t) : 0;
    if (s < 0 || s >= a.S) break;  // behind the last sequence
    int64_t last = a.offsets ? clamped(a.offsets[s + 1], a.T) : a.T;
    last = last < end ? last : end;
    if (last <= t) break;  // (offsets that do not ascend)
    add_tokens<VPT, T>(a, t + warp, last, kWarps, sm_sums + warp * E, count);
    __syncthreads();
    over_warps(sm_sums, E);
    const int64_t row = blockIdx.x + (int64_t)s;
    for (int e = threadIdx.x; e < E; e += kThreads) {  // (each thread's own sums)
      sums[row * E + e] = sm_sums[e];
      counts[row * E + e] = count[e];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sm_sums[w * E + e] = {0.0f, 0.0f};
      count[e] = 0;
    }
    __syncthreads();
    t = last;
  }
}
// ... and a cluster per sequence that joins its rows.
constexpr int kJoin = 1024;
__global__ void __launch_bounds__(kJoin)
    k_balance_join(const BalanceArgs a, const int chunk, const int chunks, const int log_ctas) {
  extern __shared__ Sum sm_sums[];  // [E], then (CTA 0) [CTA][E]
  __shared__ Sum part_sums[1024];
  __shared__ int32_t part_counts[1024];
  const int E = a.E, C = 1 << log_ctas, rank = (int)ptx::cluster_rank(), s = blockIdx.x >> log_ctas;
  Sum* gathered = sm_sums + E;
  int32_t* count = reinterpret_cast<int32_t*>(gathered + C * E);
  const int64_t rows = (int64_t)chunks + a.S;
  const Sum* sums = static_cast<const Sum*>(a.workspace);
  const int32_t* counts = reinterpret_cast<const int32_t*>(sums + rows * E);
  ptx::cluster_arrive();
  const int64_t t0 = a.offsets ? clamped(a.offsets[s], a.T) : 0;
  const int64_t t1 = a.offsets ? clamped(a.offsets[s + 1], a.T) : a.T;
  ptx::griddep_wait();
  ptx::griddep_launch();
  // (T <= 2^27; a 64-bit division takes half a microsecond)
  const int c0 = (int)t0 / chunk, c1 = t1 > t0 ? (int)(t1 - 1) / chunk + 1 : c0;
  const int per = (c1 - c0 + C - 1) >> log_ctas;
  const int from = min(c0 + rank * per, c1), to = min(from + per, c1);
  // the threads are `parts` groups of E or more, group p of which takes every parts-th row
  const int parts = E <= kJoin / 2 ? kJoin / E : 1, p = parts > 1 ? threadIdx.x / E : 0;
  for (int e = threadIdx.x - p * E; e < E && p < parts; e += kJoin) {
    Sum sum = {0.0f, 0.0f};
    int32_t n = 0;
#pragma unroll 8
    for (int c = from + p; c < to; c += parts) {
      const int64_t row = (int64_t)c + s;
      sum.add(sums[row * E + e]);
      n += counts[row * E + e];
    }
    part_sums[p * E + e] = sum;
    part_counts[p * E + e] = n;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kJoin) {
    Sum sum = part_sums[e];
    int32_t n = part_counts[e];
    for (int q = 1; q < parts; ++q) {
      sum.add(part_sums[q * E + e]);
      n += part_counts[q * E + e];
    }
    sm_sums[e] = sum;
    count[e] = n;
  }
  ptx::cluster_wait();
  finish<kJoin>(a, s, t1 - t0, C, rank, sm_sums, count, gathered, count + E);
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
  __shared__ float words[4][32 * VPT];
  float* mine = words[warp];
  const int64_t t = (int64_t)blockIdx.x * 4 + warp;
  if (t >= a.T) return;
  int id = -1;
  float gi = 0.0f;
  if (a.grad_weights && lane < a.k) {
    id = a.experts[t * a.k + lane];
    gi = a.grad_weights[t * a.k + lane];
    if (id < 0 || id >= E) id = -1;
  }
  // rest: the derivative of a score with respect to its logit without the softmax's sum
  float s[VPT], u[VPT], rest[VPT];
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  load_logits<VPT>(row, E, s);
  const int q = a.offsets ? sequence_of(a.offsets, a.S, t) : 0;
  T* grad = static_cast<T*>(a.grad) + t * E;
  float coef = 0.0f;
  if (q >= 0 && q < a.S) {
    const int64_t t0 = a.offsets ? clamped(a.offsets[q], a.T) : 0;
    const int64_t t1 = a.offsets ? clamped(a.offsets[q + 1], a.T) : a.T;
    const float n = (float)(t1 - t0);
    coef = a.grad_loss[q] * ((float)E / ((float)a.k * n) / n);
  } else if (!a.grad_weights) {  // padding, whose logits may be anything
    for (int e = lane; e < E; e += 32) grad[e] = from_f32<T>(0.0f);
    return;
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = lane + 32 * j;
    u[j] = coef != 0.0f && e < E ? coef * (float)__ldg(a.counts + (int64_t)q * E + e) : 0.0f;
  }
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) s[j] = sigmoid(s[j], rest[j]);
  } else {
    scores_of<VPT>(0, s);
#pragma unroll
    for (int j = 0; j < VPT; ++j) rest[j] = s[j];
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
    if (sum < kSmallSum) {  // the whole warp
      // (the weights, of the sigmoids themselves: sum times the scores used here, or their
      // quotients; where the sigmoids are 0 in fp32, the weights are 0, too)
      if (sum == 0.0f) id = -1;
      if (!a.renorm) gi *= sum;
      load_logits<VPT>(row, E, s);
      scores_of<VPT>(0, s);
      dot = 0.0f;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        rest[j] = s[j];
        dot += u[j] * s[j];
      }
      dot = warp_sum(dot);
    } else {
      inv = 1.0f / sum;
    }
  }
  dot *= inv;
#pragma unroll
  for (int j = 0; j < VPT; ++j) u[j] = (u[j] - dot) * inv;
  // the weights
  if (a.grad_weights) {
    // The chosen scores are picked up from shared memory, and their gradients added there.
#pragma unroll
    for (int j = 0; j < VPT; ++j) mine[lane + 32 * j] = s[j];
    __syncwarp();
    const float si = id >= 0 ? mine[id] : 0.0f;
    const float total = warp_sum(si), along = warp_sum(si * gi);
    float di = id >= 0 ? gi : 0.0f;
    if (a.renorm) {
      if (total < kSmallChosen && total > 0.0f) {  // the whole warp
        di = id < 0 ? 0.0f : (gi - along / total) / (total * 0x1p64f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          u[j] *= 0x1p-64f;
          rest[j] *= 0x1p64f;
        }
      } else {
        di = total == 0.0f || id < 0 ? 0.0f : (gi - along / total) / total;
      }
    }
    di *= a.scale;
    const float inner = a.sigmoid ? 0.0f : warp_sum(di * si);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < VPT; ++j) mine[lane + 32 * j] = u[j] - inner;
    __syncwarp();
    const uint32_t same = __match_any_sync(kAll, id >= 0 ? id : -1 - lane);
    if (__all_sync(kAll, (same & (same - 1)) == 0)) {
      if (id >= 0) mine[id] += di;
    } else {  // an expert twice: in the order of the choices
      for (int i = 0; i < a.k; ++i) {
        if (lane == i && id >= 0) mine[id] += di;
        __syncwarp();
      }
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < VPT; ++j) u[j] = mine[lane + 32 * j];
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = lane + 32 * j;
    if (e < E) grad[e] = from_f32<T>(u[j] * rest[j]);
  }
}

// ------------------------------------------------------------------- host
// Tokens of a CTA of the form for many of them (whatever the GPU: the workspace's size
// depends on it): 257 to 512 CTAs, of sixteen tokens at least.
int64_t chunk_of(int64_t T) {
  int64_t chunk = 16;
  while (ceil_div(T, chunk) > 512) chunk *= 2;
  return chunk;
}
// The form in chunks takes two launches, and a row of sums for each chunk and sequence (us with
// it / without: 512 tokens of 64 experts 6.2 / 5.8, 768 6.1 / 7.5, 2048 6.1 / 15.9; 4096 in 64
// sequences 9.8 / 5.7, 16384 in 256 15.1 / 12.4, in 64, 256 experts, 19.6 / 23.2, in 8 17.2 / 46.8).
bool many(int64_t T, int64_t S) { return T > 640 && T > 64 * S && S <= 1024; }
// CTAs of a sequence's cluster, as log2, without chunks: by its tokens on average (64 are one
// for each warp of eight CTAs), and as many as leave two CTAs an SM (us with 1 / 2 / 4 / 8:
// 600 tokens in 100 sequences 4.6 / 4.0 / 3.7 / 5.3, in 40 5.5 / 4.2 / 3.5 / 3.9, in 20 8.1 / 5.8 /
// 4.1 / 3.6, in 10 10.6 / 6.5 / 4.8 / 5.0).
int few_log(int64_t T, int64_t S) {
  int log = T >= 64 * S ? 3 : (T >= 32 * S ? 2 : (T >= 16 * S ? 1 : 0));
  while (log < 3 && S << (log + 1) <= 2 * device_sm_count()) ++log;
  return log;
}
// CTAs that join a sequence's chunks (us with 1 / 4 / 8: 16384 tokens in 64 sequences 19.2 / 16.9 /
// 22.5, in 8 23.9 / 16.3 / 17.2; 8191 in one, 128 experts, with the gradient, 23.3 / 12.0 / 10.1).
int join_log(int64_t chunks, int64_t S) { return chunks >= 128 * S ? 3 : (chunks >= 8 * S ? 2 : 0); }

template <int VPT, typename T>
cudaError_t forward(const BalanceArgs& a, cudaStream_t s) {
  const size_t E = (size_t)a.E;
  if (!many(a.T, a.S)) {
    const int log_ctas = few_log(a.T, a.S), C = 1 << log_ctas;
    return launch_clusters<k_balance<VPT, T>>(dim3((unsigned)a.S << log_ctas), C, kThreads,
                                              E * (kWarps + C) * 8 + E * (1 + C) * 4, s, a, log_ctas);
  }
  const int chunk = (int)chunk_of(a.T), chunks = (int)ceil_div(a.T, chunk);
  const cudaError_t e =
      launch_clusters<k_balance_chunks<VPT, T>>(dim3(chunks), 1, kThreads, E * (kWarps * 8 + 4), s, a, chunk);
  if (e != cudaSuccess) return e;
  const int log_ctas = join_log(chunks, a.S), C = 1 << log_ctas;
  return launch_clusters<k_balance_join>(dim3((unsigned)a.S << log_ctas), C, kJoin, E * (1 + C) * 12, s, a, chunk,
                                         chunks, log_ctas);
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

size_t balance_bytes(int64_t T, int64_t S, int64_t E) {
  return many(T, S) ? (size_t)((ceil_div(T, chunk_of(T)) + S) * E * 12) : 0;
}

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
