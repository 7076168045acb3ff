// Routing of tokens to experts: scores and choice, their gradient, the order
// of the chosen rows by expert, and the weighted sum of the experts' results
// with its gradient.
#include <atomic>

#include "mx_internal.cuh"
#include "ptx.cuh"
#include "scores.cuh"

namespace imc {
namespace mx {
namespace {

// A float as an unsigned number in the same order; NaN below every number.
// 0 stays free for "not to be chosen".
__device__ __forceinline__ uint32_t ordered(float v) {
  if (v != v) return 1u;
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 becomes 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  if (u <= 1u) return __uint_as_float(u ? 0x7FC00000u : 0xFF800000u);
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

constexpr int kRouteWarps = 4;
// Shared-memory place of expert e: a word skipped every 32, so that lanes that
// read groups of 32 experts side by side meet different banks.
__host__ __device__ constexpr int padded(int e) { return e + (e >> 5); }

// The two highest of two pairs (a1 >= a2, b1 >= b2).
__device__ __forceinline__ void best_two(uint32_t& a1, uint32_t& a2, uint32_t b1, uint32_t b2) {
  a2 = max(min(a1, b1), max(a2, b2));
  a1 = max(a1, b1);
}

// The k rounds of a choice among 32 * R keys (lane l: keys l, l + 32, ...): the
// highest key of the warp, the lowest index that has it; lane i gets the i-th.
template <int R, int V>
__device__ __forceinline__ int choose(uint32_t (&key)[V], int k) {
  const int lane = threadIdx.x & 31;
  int id = 0;
  for (int i = 0; i < k; ++i) {
    uint32_t best = key[0], at = lane;
#pragma unroll
    for (int j = 1; j < R; ++j)
      if (key[j] > best) {
        best = key[j];
        at = lane + 32 * j;
      }
    const uint32_t top = __reduce_max_sync(kAll, best);
    const uint32_t e = __reduce_min_sync(kAll, best == top ? at : 0x7FFFFFFFu);
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (e == (uint32_t)(lane + 32 * j)) key[j] = 0;
    if (lane == i) id = (int)e;
  }
  return id;
}

// One warp per token.  Scores and keys stay in registers (VPT per lane) for the
// k rounds of the choice: the highest key of each lane, the highest of the warp
// (redux), and the lowest index that has it (redux).  The chosen scores are
// picked up from shared memory at the end.
template <int VPT, typename T>
__global__ void __launch_bounds__(kRouteWarps * 32) k_route(const RouteArgs a) {
  extern __shared__ uint32_t sm_words[];  // [warp][padded E] keys, then scores
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= a.T) return;
  float s[VPT];
  scores<VPT, T>(static_cast<const T*>(a.logits) + t * a.ld, a.E, a.sigmoid, s);
  uint32_t key[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = lane + 32 * j;
    key[j] = e < a.E ? ordered(a.bias ? s[j] + __ldg(a.bias + e) : s[j]) : 0u;
  }
  uint32_t* words = sm_words + warp * padded(a.E);
  __shared__ int groups[kRouteWarps][32];  // the groups that stay, in order
  const int size = a.size;
  constexpr int HALF = (VPT + 1) / 2;
  bool half = false;  // the candidates fill no more than half of the keys
  auto expert_of = [&](int c) {
    if (a.groups == 1) return c;
    const int g = (int)((c * a.inv_size) >> 20);
    return groups[warp][g] * size + c - g * size;
  };
  if (a.groups > 1) {
    // The sum of each group's two best; the best top_groups groups stay.
    // 2^ls lanes share a group.
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (lane + 32 * j < a.E) words[padded(lane + 32 * j)] = key[j];
    __syncwarp();
    int ls = 0;
    while ((a.groups << (ls + 1)) <= 32) ++ls;
    const int g = lane >> ls;
    uint32_t b1 = 0, b2 = 0;
    if (g < a.groups)
      for (int i = lane & ((1 << ls) - 1); i < size; i += 1 << ls)
        best_two(b1, b2, words[padded(g * size + i)], 0u);
    for (int d = 1; d < (1 << ls); d <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(kAll, b1, d), o2 = __shfl_xor_sync(kAll, b2, d);
      best_two(b1, b2, o1, o2);
    }
    uint32_t gkey = 0;
    if (g < a.groups)
      gkey = ordered(size > 1 ? from_ordered(b1) + from_ordered(b2) : from_ordered(b1));
    uint32_t kept = 0;
    for (int i = 0; i < a.top_groups; ++i) {
      const uint32_t best = __reduce_max_sync(kAll, gkey);
      const int at = (__ffs(__ballot_sync(kAll, gkey == best)) - 1) >> ls;
      kept |= 1u << at;
      if (g == at) gkey = 0;
    }
    // The rounds run over the candidates only: candidate c is the c-th expert of
    // the groups that stay.  c / size by a product, exact for c * (size - 1) < 2^20.
    const int candidates = a.top_groups * size;
    half = candidates <= 32 * HALF;
    if ((kept >> lane) & 1u) groups[warp][__popc(kept & ((1u << lane) - 1u))] = lane;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = lane + 32 * j;  // past the candidates: 0, never chosen
      if (j < HALF || !half) key[j] = c < candidates ? words[padded(expert_of(c))] : 0u;
    }
    __syncwarp();
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    if (lane + 32 * j < a.E) words[padded(lane + 32 * j)] = __float_as_uint(s[j]);
  __syncwarp();
  // (the keys past HALF are old ones then, and not looked at)
  int id = half ? choose<HALF>(key, a.k) : choose<VPT>(key, a.k);
  id = expert_of(id);
  float w = lane < a.k ? __uint_as_float(words[padded(id)]) : 0.0f;
  if (a.renorm) {
    const float total = warp_sum(w);
    w = total == 0.0f ? 0.0f : w / total;
  }
  if (lane < a.k) {
    a.weights[t * a.k + lane] = w * a.scale;
    a.experts[t * a.k + lane] = id;
  }
}

// Gradient of the weights with respect to the logits; the choice is constant.
//   w_i = scale * s_i / S (S = sum over the chosen, or 1),
//   ds_i = scale * (g_i - sum_j g_j s_j / S) / S,   or scale * g_i,
//   softmax: dx_e = s_e * (ds_e - sum_i ds_i s_i),  sigmoid: dx_e = ds_e s_e (1 - s_e).
template <int VPT, typename T>
__global__ void __launch_bounds__(kRouteWarps * 32)
    k_route_backward(const RouteArgs a, const float* __restrict__ g, T* __restrict__ grad) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= a.T) return;
  float s[VPT];
  scores<VPT, T>(static_cast<const T*>(a.logits) + t * a.ld, a.E, a.sigmoid, s);
  int id = -1;
  float gi = 0.0f;
  if (lane < a.k) {
    id = a.experts[t * a.k + lane];
    gi = g[t * a.k + lane];
    if (id < 0 || id >= a.E) id = -1;
  }
  float total = 0.0f, dot = 0.0f, si = 0.0f;
  for (int i = 0; i < a.k; ++i) {
    const int e = __shfl_sync(kAll, id, i);
    if (e < 0) continue;
    const float p = __shfl_sync(kAll, pick<VPT>(s, e >> 5), e & 31);
    total += p;
    dot += p * __shfl_sync(kAll, gi, i);
    if (lane == i) si = p;
  }
  float di = id >= 0 ? gi : 0.0f;
  const bool small = a.renorm && total < kSmallChosen;  // the whole warp
  if (a.renorm) di = total == 0.0f || id < 0 ? 0.0f : (gi - dot / total) / (small ? total * 0x1p64f : total);
  di *= a.scale;
  const float inner = a.sigmoid ? 0.0f : warp_sum(di * si);
  float d[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) d[j] = 0.0f;
  for (int i = 0; i < a.k; ++i) {
    const int e = __shfl_sync(kAll, id, i);
    const float v = __shfl_sync(kAll, di, i);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (e == lane + 32 * j) d[j] += v;
  }
  if (small) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int e = lane + 32 * j;
      if (e < a.E)
        grad[t * a.E + e] = from_f32<T>((a.sigmoid ? d[j] * s[j] * (1.0f - s[j]) : s[j] * (d[j] - inner)) * 0x1p64f);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = lane + 32 * j;
    if (e < a.E)
      grad[t * a.E + e] = from_f32<T>(a.sigmoid ? d[j] * s[j] * (1.0f - s[j]) : s[j] * (d[j] - inner));
  }
}

// ------------------------------------------------------------------ layout
// Stable counting sort of n slots by expert.  Each warp owns a contiguous run
// of slots and walks it 32 at a time: a slot's rank among its CTA's slots of the
// same expert is what lower warps and steps have counted plus the equal experts
// on lower lanes, found with one ballot per bit of the expert's number (nothing
// depends on the timing of atomics).  A slot's place is the expert's first place
// + the slots of lower CTAs + its rank.  Experts outside [0, E) fall into
// bucket E.
//
// Up to kLayoutOne slots one CTA does all of it.  More slots take two launches
// over many CTAs: k_layout_count leaves ranks in `dest` and each CTA's counts in
// `counts` [CTA][E + 1], k_layout_place sums those up (every CTA for itself, a
// bucket a thread) and places the slots.  One launch over a cluster of eight
// CTAs measured 26 us for 131072 slots of 256 experts: too few warps for the
// ~60 instructions per 32 slots.
constexpr int kLayoutThreads = 512, kLayoutWarps = kLayoutThreads / 32;
constexpr int kLayoutOne = 4096;

struct LayoutArgs {
  const int32_t* experts;
  int n, E, per;  // per: slots of a warp, a multiple of 32
  int32_t *offsets, *starts, *order, *dest, *dest224, *counts;
};

__device__ __forceinline__ int layout_bucket(const LayoutArgs& a, int64_t i, int64_t end) {
  if (i >= end) return a.E + 1;  // no slot
  const int e = __ldg(a.experts + i);
  return e < 0 || e >= a.E ? a.E : e;
}

// The slots [w0, w1) of this warp: their ranks within the warp go to `dest`,
// the warp's counts to mine [E + 1] (zero before).
__device__ __forceinline__ void layout_rank(const LayoutArgs& a, int64_t w0, int64_t w1,
                                            int32_t* mine) {
  const int lane = threadIdx.x & 31, B = a.E + 1;
  const int bits = 32 - __clz(B);  // of bucket numbers 0 .. B (B: no slot)
  constexpr int U = 4;             // steps whose loads are in flight together
  for (int64_t i0 = w0; i0 < w1; i0 += 32 * U) {
    int ids[U];
#pragma unroll
    for (int u = 0; u < U; ++u) ids[u] = layout_bucket(a, i0 + 32 * u + lane, w1);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + 32 * u >= w1) break;
      const int e = ids[u];
      uint32_t same = kAll;
      for (int b = 0; b < bits; ++b) {
        const uint32_t set = __ballot_sync(kAll, (e >> b) & 1);
        same &= (e >> b) & 1 ? set : ~set;
      }
      const int place = __popc(same & ((1u << lane) - 1u));
      const int before = e < B ? mine[e] : 0;
      __syncwarp();
      if (e < B) {
        if (place == 0) mine[e] = before + __popc(same);
        a.dest[i0 + 32 * u + lane] = before + place;
      }
      __syncwarp();
    }
  }
}

// hist [warps][B] to exclusive sums over the warps; their total of bucket e goes
// to total[e].
__device__ __forceinline__ void layout_over_warps(int32_t* hist, int B, int32_t* total) {
  for (int e = threadIdx.x; e < B; e += blockDim.x) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kLayoutWarps; ++w) {
      const int c = hist[w * B + e];
      hist[w * B + e] = sum;
      sum += c;
    }
    total[e] = sum;
  }
}

// From `all(e)`, bucket e's slots: offsets and starts (written by the CTA that
// has `write`), first[e] = the expert's first place, shift[e] = starts - offsets.
template <typename All>
__device__ __forceinline__ void layout_scan(const LayoutArgs& a, bool write, int32_t* first,
                                            int32_t* shift, All all) {
  __shared__ int32_t sums[2][32];
  const int B = a.E + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = (int)blockDim.x >> 5;
  int carry = 0, carry_pad = 0;
  for (int e0 = 0; e0 < B; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    const int n = e < B ? all(e) : 0;
    const int pad = (n + ATOM_ROWS - 1) / ATOM_ROWS * ATOM_ROWS;
    int x = n, y = pad;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int ox = __shfl_up_sync(kAll, x, d), oy = __shfl_up_sync(kAll, y, d);
      if (lane >= d) {
        x += ox;
        y += oy;
      }
    }
    __syncthreads();
    if (lane == 31) {
      sums[0][warp] = x;
      sums[1][warp] = y;
    }
    __syncthreads();
    int upto = carry + x, upto_pad = carry_pad + y;
    for (int w = 0; w < warps; ++w) {
      const int u = sums[0][w], v = sums[1][w];
      if (w < warp) {
        upto += u;
        upto_pad += v;
      }
      carry += u;
      carry_pad += v;
    }
    if (e < B) {
      const int off = upto - n, start = upto_pad - pad;
      if (write) {
        a.offsets[e] = off;
        a.starts[e] = start;
        if (e == a.E) a.offsets[e + 1] = a.n;
      }
      shift[e] = start - off;
      first[e] = off;
    }
  }
}

// Every slot of [w0, w1) to its place: first[e] + mine[e] + its rank.
__device__ __forceinline__ void layout_place(const LayoutArgs& a, int64_t w0, int64_t w1,
                                             const int32_t* first, const int32_t* mine,
                                             const int32_t* shift) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 31;
  for (int64_t i0 = w0; i0 < w1; i0 += 32 * U) {
    int ids[U], ranked[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + 32 * u + lane;
      ids[u] = layout_bucket(a, i, w1);
      ranked[u] = i < w1 ? a.dest[i] : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + 32 * u + lane;
      const int e = ids[u];
      if (i >= w1) break;
      const int pos = first[e] + mine[e] + ranked[u];
      a.order[pos] = (int32_t)i;
      const int start = first[e] + shift[e], in = pos - first[e];
      a.dest[i] = e < a.E ? start + in : -1;
      a.dest224[i] = e < a.E ? (int)sorted_at(start, TILES_224) + in : -1;
    }
  }
}

// ONE: the whole sort in one CTA; else the first of the two launches.
template <bool ONE>
__global__ void __launch_bounds__(kLayoutThreads) k_layout_count(const LayoutArgs a) {
  extern __shared__ int32_t sm[];
  const int B = a.E + 1, warp = threadIdx.x >> 5;
  int32_t *hist = sm, *total = sm + kLayoutWarps * B, *first = total + B, *shift = first + B;
  for (int i = threadIdx.x; i < kLayoutWarps * B; i += blockDim.x) hist[i] = 0;
  __syncthreads();
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int64_t w0 = ((int64_t)blockIdx.x * kLayoutWarps + warp) * a.per;
  const int64_t w1 = w0 + a.per < a.n ? w0 + a.per : a.n;
  int32_t* mine = hist + warp * B;
  layout_rank(a, w0, w1, mine);
  __syncthreads();
  layout_over_warps(hist, B, total);
  __syncthreads();
  if (ONE) {
    layout_scan(a, true, first, shift, [&](int e) { return total[e]; });
    __syncthreads();
    layout_place(a, w0, w1, first, mine, shift);
  } else {
    for (int e = threadIdx.x; e < B; e += blockDim.x)
      a.counts[(int64_t)blockIdx.x * B + e] = total[e];
    for (int64_t i = w0 + (threadIdx.x & 31); i < w1; i += 32)  // ranks within the CTA
      a.dest[i] += mine[layout_bucket(a, i, w1)];
  }
}

__global__ void __launch_bounds__(kLayoutThreads) k_layout_place(const LayoutArgs a) {
  extern __shared__ int32_t sm[];
  const int B = a.E + 1, warp = threadIdx.x >> 5;
  int32_t *first = sm, *shift = first + B, *before = shift + B;
  ptx::griddep_wait();
  ptx::griddep_launch();
  layout_scan(a, blockIdx.x == 0, first, shift, [&](int e) {
    int all = 0, low = 0;
#pragma unroll 16
    for (int c = 0; c < (int)gridDim.x; ++c) {
      const int v = __ldg(a.counts + (int64_t)c * B + e);
      all += v;
      if (c < (int)blockIdx.x) low += v;
    }
    before[e] = low;
    return all;
  });
  __syncthreads();
  const int64_t w0 = ((int64_t)blockIdx.x * kLayoutWarps + warp) * a.per;
  const int64_t w1 = w0 + a.per < a.n ? w0 + a.per : a.n;
  layout_place(a, w0, w1, first, before, shift);
}

// ------------------------------------------------------------ weighted sum
// out[t] = sum_s w[t,s] * y[t*k + s] (w null: ones), in the order of s, fp32, rounded
// once to out's type O; a thread has 8 columns of one token.
template <typename T, typename O>
__global__ void __launch_bounds__(256)
    k_combine(const T* __restrict__ y, const float* __restrict__ w, const int64_t T_, const int k,
              const int64_t N, O* __restrict__ out, const bool vec) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int64_t per = ceil_div(N, 8), items = T_ * per;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < items;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / per, c = (i - t * per) * 8;
    const int n = (int)(N - c < 8 ? N - c : 8);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const T* row = y + t * k * N + c;
    int s = 0;
    for (; s + 4 <= k; s += 4) {
      float v[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u) load8<T>(row + (s + u) * N, n, vec, v[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float ws = w ? __ldg(w + t * k + s + u) : 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = fmaf(ws, v[u][j], acc[j]);
      }
    }
    for (; s < k; ++s) {
      float v[8];
      load8<T>(row + s * N, n, vec, v);
      const float ws = w ? __ldg(w + t * k + s) : 1.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = fmaf(ws, v[j], acc[j]);
    }
    store8<O>(out + t * N + c, n, vec, acc);
  }
}

// grad_y[t*k + s] = w[t,s] * grad[t], grad_w[t,s] = <grad[t], y[t*k + s]>: one
// warp per slot (the warps of a token's slots share its gradient row in L1).
template <typename T>
__global__ void __launch_bounds__(256)
    k_combine_backward(const T* __restrict__ grad, const T* __restrict__ y,
                       const float* __restrict__ w, const int64_t slots, const int k,
                       const int64_t N, T* __restrict__ grad_y, float* __restrict__ grad_w,
                       const bool vec) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; i < slots; i += warps) {
    const float ws = w[i];
    const T *g = grad + i / k * N, *yr = y + i * N;
    float dot = 0.0f;
#pragma unroll 2
    for (int64_t c = lane * 8; c < N; c += 256) {
      const int n = (int)(N - c < 8 ? N - c : 8);
      float gv[8], yv[8];
      load8<T>(g + c, n, vec, gv);
      load8<T>(yr + c, n, vec, yv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dot = fmaf(gv[j], yv[j], dot);
        gv[j] *= ws;
      }
      store8<T>(grad_y + i * N + c, n, vec, gv);
    }
    dot = warp_sum(dot);
    if (lane == 0) grad_w[i] = dot;
  }
}

// ------------------------------------------------------------------- host
template <typename T>
cudaError_t route(const RouteArgs& a, const float* g, void* grad, cudaStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.T, kRouteWarps)), block(kRouteWarps * 32);
  const size_t smem = g ? 0 : (size_t)kRouteWarps * padded(a.E) * 4;
  cudaError_t e;
#define IMC_ROUTE(V)                                                                            \
  e = g ? launch_after_previous(k_route_backward<V, T>, grid, block, 0, s, a, g,                \
                                static_cast<T*>(grad))                                          \
        : launch_after_previous(k_route<V, T>, grid, block, smem, s, a)
  if (a.E <= 32) IMC_ROUTE(1);
  else if (a.E <= 64) IMC_ROUTE(2);
  else if (a.E <= 128) IMC_ROUTE(4);
  else if (a.E <= 256) IMC_ROUTE(8);
  else if (a.E <= 512) IMC_ROUTE(16);
  else IMC_ROUTE(32);
#undef IMC_ROUTE
  note_launch();
  return e;
}

template <typename T, typename O = T>
cudaError_t combine(const void* y, const float* w, int64_t tokens, int k, int64_t N, void* out,
                    cudaStream_t s) {
  constexpr int64_t narrow = sizeof(T) < sizeof(O) ? sizeof(T) : sizeof(O);
  const bool vec = ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0 &&
                   (N * narrow) % 16 == 0;
  const int64_t blocks = ceil_div(tokens * ceil_div(N, 8), 256), cap = (int64_t)device_sm_count() * 8;
  const cudaError_t e = launch_after_previous(
      k_combine<T, O>, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, s,
      static_cast<const T*>(y), w, tokens, k, N, static_cast<O*>(out), vec);
  note_launch();
  return e;
}

template <typename T>
cudaError_t combine_backward(const void* grad, const void* y, const float* w, int64_t tokens, int k,
                             int64_t N, void* grad_y, float* grad_w, cudaStream_t s) {
  const bool vec = ((reinterpret_cast<uintptr_t>(grad) | reinterpret_cast<uintptr_t>(y) |
                     reinterpret_cast<uintptr_t>(grad_y)) & 15u) == 0 &&
                   (N * (int64_t)sizeof(T)) % 16 == 0;
  const int64_t blocks = ceil_div(tokens * k, 8), cap = (int64_t)device_sm_count() * 8;
  const cudaError_t e = launch_after_previous(
      k_combine_backward<T>, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, s,
      static_cast<const T*>(grad), static_cast<const T*>(y), w, tokens * k, k, N,
      static_cast<T*>(grad_y), grad_w, vec);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, int dtype, cudaStream_t s) {
  note_kernel_name("k_route");
  if (dtype == IMC_F32) return route<float>(a, nullptr, nullptr, s);
  if (dtype == IMC_F16) return route<__half>(a, nullptr, nullptr, s);
  return route<__nv_bfloat16>(a, nullptr, nullptr, s);
}

cudaError_t launch_route_backward(const RouteArgs& a, int dtype, const float* g, void* grad_logits,
                                  cudaStream_t s) {
  note_kernel_name("k_route_backward");
  if (dtype == IMC_F32) return route<float>(a, g, grad_logits, s);
  if (dtype == IMC_F16) return route<__half>(a, g, grad_logits, s);
  return route<__nv_bfloat16>(a, g, grad_logits, s);
}

// CTAs of a layout: enough for four steps of 32 slots a warp, at most
// kLayoutMaxCtas (every CTA of the second launch reads all of their counts).
int layout_ctas(int64_t n) {
  if (n <= kLayoutOne) return 1;
  const int64_t c = ceil_div(n, kLayoutWarps * 128);
  return (int)(c < kLayoutMaxCtas ? c : kLayoutMaxCtas);
}

cudaError_t launch_layout(const int32_t* experts, int n, int E, int32_t* offsets, int32_t* starts,
                          int32_t* order, int32_t* dest, int32_t* dest224, int32_t* counts,
                          cudaStream_t s) {
  note_kernel_name("k_layout");
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int most = (kLayoutWarps + 3) * (1024 + 1) * 4;
  if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    for (auto k : {k_layout_count<true>, k_layout_count<false>}) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != cudaSuccess) return e;
    }
    if (dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  const int ctas = layout_ctas(n);
  LayoutArgs a = {experts, n, E, 0, offsets, starts, order, dest, dest224, counts};
  a.per = (int)(ceil_div(n, (int64_t)32 * kLayoutWarps * ctas) * 32);
  const size_t smem = (size_t)(kLayoutWarps + 3) * (E + 1) * 4;
  if (ctas == 1) {
    e = launch_after_previous(k_layout_count<true>, dim3(1), dim3(kLayoutThreads), smem, s, a);
  } else {
    e = launch_after_previous(k_layout_count<false>, dim3(ctas), dim3(kLayoutThreads), smem, s, a);
    note_launch();
    if (e == cudaSuccess)
      e = launch_after_previous(k_layout_place, dim3(ctas), dim3(kLayoutThreads),
                                (size_t)3 * (E + 1) * 4, s, a);
  }
  note_launch();
  return e;
}

cudaError_t launch_combine(const void* y, const float* w, int dtype, int64_t T, int k, int64_t N,
                           void* out, int out_dtype, cudaStream_t s) {
  note_kernel_name("k_combine");
  if (dtype == IMC_F32 && out_dtype == IMC_F16) return combine<float, __half>(y, w, T, k, N, out, s);
  if (dtype == IMC_F32 && out_dtype == IMC_BF16)
    return combine<float, __nv_bfloat16>(y, w, T, k, N, out, s);
  if (dtype == IMC_F32) return combine<float>(y, w, T, k, N, out, s);
  if (dtype == IMC_F16) return combine<__half>(y, w, T, k, N, out, s);
  return combine<__nv_bfloat16>(y, w, T, k, N, out, s);
}

cudaError_t launch_combine_backward(const void* grad, const void* y, const float* w, int dtype,
                                    int64_t T, int k, int64_t N, void* grad_y, float* grad_w,
                                    cudaStream_t s) {
  note_kernel_name("k_combine_backward");
  if (dtype == IMC_F32) return combine_backward<float>(grad, y, w, T, k, N, grad_y, grad_w, s);
  if (dtype == IMC_F16) return combine_backward<__half>(grad, y, w, T, k, N, grad_y, grad_w, s);
  return combine_backward<__nv_bfloat16>(grad, y, w, T, k, N, grad_y, grad_w, s);
}

}  // namespace mx
}  // namespace imc
