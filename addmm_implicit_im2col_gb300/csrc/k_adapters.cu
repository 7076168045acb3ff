// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = base[t] + scale[l] * (x[t] a[l]^T) b[l]^T,   l the adapter of row t,
//
// and their gradients.  The rows come in adapter order (moe_layout).
#include "adapters.cuh"
#include "ptx.cuh"
#include "scores.cuh"

namespace imc {
namespace mx {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Tile number t of the rows in adapter order, `height` rows of one adapter at most:
// the adapter, the place of its first row, its rows (0: there is no such tile).
// With `none` the rows without an adapter have tiles too (adapter L, the last ones).
struct RowTile {
  int l, p0, rows;
};
// All threads of the block.  Every thread counts the tiles of a run of buckets.
__device__ __forceinline__ RowTile find_tile(const int32_t* offsets, int L, bool none, int height,
                                             int t) {
  __shared__ int sums[kWarps];
  __shared__ RowTile found;
  const int B = L + (none ? 1 : 0), per = (B + kThreads - 1) / kThreads;
  const int e0 = threadIdx.x * per, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int tiles = 0;
  for (int e = e0; e < e0 + per && e < B; ++e)
    tiles += (__ldg(offsets + e + 1) - __ldg(offsets + e) + height - 1) / height;
  int upto = tiles;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(kAll, upto, d);
    if (lane >= d) upto += o;
  }
  if (threadIdx.x == 0) found.rows = 0;
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) upto += sums[w];
  int at = upto - tiles;
  if (t >= at && t < upto) {
    for (int e = e0; e < e0 + per && e < B; ++e) {
      const int first = __ldg(offsets + e), n = __ldg(offsets + e + 1) - first;
      const int mine = (n + height - 1) / height;
      if (t < at + mine) {
        const int in = (t - at) * height;
        found = {e, first + in, min(height, n - in)};
        break;
      }
      at += mine;
    }
  }
  __syncthreads();
  return found;
}
// At least as many tiles as any distribution of T rows over the buckets has.
int64_t most_tiles(int64_t T, int64_t L, int height) {
  const int64_t buckets = T < L + 1 ? T : L + 1;
  return (T + (height - 1) * buckets) / height;
}

// ---------------------------------------------------------------- few rows
// Up to FEW rows of one adapter per cluster of CTAs.  CTA q takes a run of K for
// h = x a^T, gives its partial sums to every CTA of the cluster (summed in the order
// of the CTAs), and then a run of the N outputs.
constexpr int FEW = 8;
constexpr int KC = 1024;  // values of K staged at once

template <typename T, int NR>
__device__ __forceinline__ void few_down(const T* a, int64_t K, int r, int64_t k0, int len, bool vec,
                                         const float* xs, float* part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j = 2 * warp; j < r; j += 2 * kWarps) {
    float acc[2][NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) acc[0][i] = acc[1][i] = 0.0f;
    const T* w = a + (int64_t)j * K + k0;
    const bool two = j + 1 < r;
#pragma unroll 2
    for (int k = lane * 8; k < len; k += 256) {
      float v[2][8];
      load8<T>(w + k, len - k, vec, v[0]);
      load8<T>(w + K + k, two ? len - k : 0, vec, v[1]);
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float4 p = *reinterpret_cast<const float4*>(xs + i * KC + k);
        const float4 q = *reinterpret_cast<const float4*>(xs + i * KC + k + 4);
        const float x[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          acc[0][i] = fmaf(x[u], v[0][u], acc[0][i]);
          acc[1][i] = fmaf(x[u], v[1][u], acc[1][i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const float s0 = warp_sum(acc[0][i]), s1 = warp_sum(acc[1][i]);
      if (lane == 0) {
        part[i * r + j] += s0;
        if (two) part[i * r + j + 1] += s1;
      }
    }
  }
}

template <typename T, int NR>
__device__ __forceinline__ void few_up(const AdapterArgs& p, const RowTile& t, int64_t n0, int64_t n1,
                                       bool vec, const float* h, const int* rows) {
  const T* b = static_cast<const T*>(p.b) + (int64_t)t.l * p.N * p.r;
  const T* base = static_cast<const T*>(p.base);
  T* out = static_cast<T*>(p.out);
  for (int64_t n = n0 + threadIdx.x; n < n1; n += kThreads) {
    float acc[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
      acc[i] = base && i < t.rows ? to_f32<T>(base[rows[i] * p.N + n]) : 0.0f;
    float sum[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) sum[i] = 0.0f;
    for (int j = 0; j < p.r; j += 8) {
      float v[8];
      load8<T>(b + n * p.r + j, p.r - j, vec, v);
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (j + u < p.r) sum[i] = fmaf(h[i * p.r + j + u], v[u], sum[i]);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (i < t.rows) out[rows[i] * p.N + n] = from_f32<T>(acc[i] + sum[i]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_adapters_few(const AdapterArgs p, const int log_ctas, const int none, const int flags) {
  extern __shared__ float4 sm4[];
  const int C = 1 << log_ctas, rank = (int)ptx::cluster_rank();
  float* xs = reinterpret_cast<float*>(sm4);  // [FEW][KC]
  float* part = xs + FEW * KC;                // [FEW][r] this CTA's sums, then h
  float* gathered = part + FEW * p.r;         // [C][FEW][r]
  __shared__ int rows[FEW];
  const bool vec_x = flags & 1, vec_a = flags & 2, vec_b = flags & 4;
  ptx::griddep_wait();
  ptx::griddep_launch();
  const RowTile t = find_tile(p.offsets, p.L, none != 0, FEW, blockIdx.x >> log_ctas);
  if (t.rows == 0) return;  // the whole cluster
  ptx::cluster_arrive();    // this CTA runs: its shared memory may be written
  if (threadIdx.x < FEW) rows[threadIdx.x] = threadIdx.x < t.rows ? p.order[t.p0 + threadIdx.x] : 0;
  for (int i = threadIdx.x; i < FEW * p.r; i += kThreads) part[i] = 0.0f;
  __syncthreads();
  const int64_t n_per = (ceil_div(p.N, C) + 7) / 8 * 8, n0 = rank * n_per < p.N ? rank * n_per : p.N;
  const int64_t n1 = n0 + n_per < p.N ? n0 + n_per : p.N;
  const T* base = static_cast<const T*>(p.base);
  T* out = static_cast<T*>(p.out);
  if (t.l == p.L) {  // no adapter
    ptx::cluster_wait();
    for (int i = 0; i < t.rows; ++i)
      for (int64_t n = n0 + threadIdx.x; n < n1; n += kThreads)
        out[rows[i] * p.N + n] = base ? base[rows[i] * p.N + n] : from_f32<T>(0.0f);
    return;
  }
  const int64_t k_per = (ceil_div(p.K, C) + 7) / 8 * 8, k0 = rank * k_per < p.K ? rank * k_per : p.K;
  const int64_t k1 = k0 + k_per < p.K ? k0 + k_per : p.K;
  const T* a = static_cast<const T*>(p.a) + (int64_t)t.l * p.r * p.K;
  const int NR = t.rows <= 1 ? 1 : (t.rows <= 2 ? 2 : (t.rows <= 4 ? 4 : 8));
  for (int64_t k = k0; k < k1; k += KC) {
    const int len = (int)(k1 - k < KC ? k1 - k : KC), units = (len + 7) / 8;
    for (int i = threadIdx.x; i < units * NR; i += kThreads) {
      const int row = i / units, u = i - row * units;
      float v[8];
      load8<T>(static_cast<const T*>(p.x) + rows[row] * p.ld + k + u * 8,
               row < t.rows ? len - u * 8 : 0, vec_x, v);
      float4* to = reinterpret_cast<float4*>(xs + row * KC + u * 8);
      to[0] = make_float4(v[0], v[1], v[2], v[3]);
      to[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    __syncthreads();
    if (NR == 1) few_down<T, 1>(a, p.K, p.r, k, len, vec_a, xs, part);
    else if (NR == 2) few_down<T, 2>(a, p.K, p.r, k, len, vec_a, xs, part);
    else if (NR == 4) few_down<T, 4>(a, p.K, p.r, k, len, vec_a, xs, part);
    else few_down<T, 8>(a, p.K, p.r, k, len, vec_a, xs, part);
    __syncthreads();
  }
  ptx::cluster_wait();
  const int sums = NR * p.r;
  for (int i = threadIdx.x; i < sums * C; i += kThreads) {
    const int q = i / sums, e = i - q * sums;
    ptx::st_cluster(ptx::cluster_addr(gathered + rank * FEW * p.r + e, q), __float_as_uint(part[e]));
  }
  ptx::cluster_sync();
  const float scale = p.scale ? p.scale[t.l] : 1.0f;
  for (int i = threadIdx.x; i < sums; i += kThreads) {
    float h = 0.0f;
    for (int q = 0; q < C; ++q) h += gathered[q * FEW * p.r + i];
    part[i] = h * scale;
  }
  __syncthreads();
  if (NR == 1) few_up<T, 1>(p, t, n0, n1, vec_b, part, rows);
  else if (NR == 2) few_up<T, 2>(p, t, n0, n1, vec_b, part, rows);
  else if (NR == 4) few_up<T, 4>(p, t, n0, n1, vec_b, part, rows);
  else few_up<T, 8>(p, t, n0, n1, vec_b, part, rows);
}

// --------------------------------------------------------------- gradients
// h[p] = scale * x[order[p]] a^T (DOWN_A) or g[p] = scale * grad[order[p]] b: a warp per
// element, p in adapter order.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_adapters_down(const AdapterGradArgs p, float* h, float* g) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const RowTile t = find_tile(p.offsets, p.L, false, 1, blockIdx.x);
  if (t.rows == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = p.order[t.p0];
  const float scale = p.scale ? p.scale[t.l] : 1.0f;
  const T* x = static_cast<const T*>(p.x) + row * p.K;
  const T* d = static_cast<const T*>(p.grad) + row * p.N;
  for (int j = warp; j < p.r; j += kWarps) {
    const T* a = static_cast<const T*>(p.a) + ((int64_t)t.l * p.r + j) * p.K;
    const T* b = static_cast<const T*>(p.b) + (int64_t)t.l * p.N * p.r + j;
    float hs = 0.0f, gs = 0.0f;
    for (int64_t k = lane; k < p.K; k += 32) hs = fmaf(to_f32<T>(x[k]), to_f32<T>(a[k]), hs);
    for (int64_t n = lane; n < p.N; n += 32) gs = fmaf(to_f32<T>(d[n]), to_f32<T>(b[n * p.r]), gs);
    hs = warp_sum(hs);
    gs = warp_sum(gs);
    if (lane == 0) {
      h[(int64_t)t.p0 * p.r + j] = hs * scale;
      g[(int64_t)t.p0 * p.r + j] = gs * scale;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_adapters_grad_x(const AdapterGradArgs p, const float* g) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const RowTile t = find_tile(p.offsets, p.L, true, 1, blockIdx.x);
  if (t.rows == 0) return;
  const int64_t row = p.order[t.p0];
  const T* base = static_cast<const T*>(p.base);
  const T* a = static_cast<const T*>(p.a) + (int64_t)t.l * p.r * p.K;
  for (int64_t k = threadIdx.x; k < p.K; k += kThreads) {
    float sum = 0.0f;
    if (t.l < p.L)
      for (int j = 0; j < p.r; ++j) sum = fmaf(g[(int64_t)t.p0 * p.r + j], to_f32<T>(a[j * p.K + k]), sum);
    const float v = base ? to_f32<T>(base[row * p.K + k]) : 0.0f;
    static_cast<T*>(p.grad_x)[row * p.K + k] = from_f32<T>(v + sum);
  }
}

// grad_a[l][j][k] = sum over l's rows of g[p][j] x[row][k]; grad_b[l][n][j] likewise.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_adapters_grad_w(const AdapterGradArgs p, const float* h, const float* g) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int l = blockIdx.x, j = blockIdx.y;
  const int64_t p0 = p.offsets[l], p1 = p.offsets[l + 1];
  if (p.grad_a)
    for (int64_t k = threadIdx.x; k < p.K; k += kThreads) {
      float sum = 0.0f;
      for (int64_t i = p0; i < p1; ++i)
        sum = fmaf(g[i * p.r + j], to_f32<T>(static_cast<const T*>(p.x)[p.order[i] * p.K + k]), sum);
      static_cast<T*>(p.grad_a)[((int64_t)l * p.r + j) * p.K + k] = from_f32<T>(sum);
    }
  if (p.grad_b)
    for (int64_t n = threadIdx.x; n < p.N; n += kThreads) {
      float sum = 0.0f;
      for (int64_t i = p0; i < p1; ++i)
        sum = fmaf(h[i * p.r + j], to_f32<T>(static_cast<const T*>(p.grad)[p.order[i] * p.N + n]), sum);
      static_cast<T*>(p.grad_b)[((int64_t)l * p.N + n) * p.r + j] = from_f32<T>(sum);
    }
}

// ------------------------------------------------------------------- host
bool aligned16(const void* p, int64_t pitch_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)pitch_bytes) & 15u) == 0;
}

template <typename T>
cudaError_t adapters_few(const AdapterArgs& a, cudaStream_t s) {
  const int log_ctas = 3;
  const int none = a.base != a.out ? 1 : 0;
  const int64_t tiles = most_tiles(a.T, a.L, FEW);
  const int64_t b = sizeof(T);
  const int flags = (aligned16(a.x, a.ld * b) ? 1 : 0) | (aligned16(a.a, a.K * b) ? 2 : 0) |
                    (aligned16(a.b, a.r * b) ? 4 : 0);
  const size_t smem = (size_t)(FEW * KC + (FEW + (FEW << log_ctas)) * a.r) * 4;
  cudaError_t e = cudaFuncSetAttribute(k_adapters_few<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles << log_ctas));
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
  e = cudaLaunchKernelEx(&cfg, k_adapters_few<T>, a, log_ctas, none, flags);
  note_launch();
  return e;
}

template <typename T>
cudaError_t backward(const AdapterGradArgs& a, cudaStream_t s) {
  float *h = static_cast<float*>(a.workspace), *g = h + a.T * a.r;
  cudaError_t e = launch_after_previous(k_adapters_down<T>, dim3((unsigned)a.T), dim3(kThreads), 0, s, a, h, g);
  note_launch();
  if (e == cudaSuccess && a.grad_x) {
    e = launch_after_previous(k_adapters_grad_x<T>, dim3((unsigned)a.T), dim3(kThreads), 0, s, a, g);
    note_launch();
  }
  if (e == cudaSuccess && (a.grad_a || a.grad_b)) {
    e = launch_after_previous(k_adapters_grad_w<T>, dim3(a.L, a.r), dim3(kThreads), 0, s, a, h, g);
    note_launch();
  }
  return e;
}

}  // namespace

cudaError_t launch_adapters(const AdapterArgs& a, int dtype, cudaStream_t s) {
  note_kernel_name("k_adapters_few");
  if (dtype == IMC_F32) return adapters_few<float>(a, s);
  if (dtype == IMC_F16) return adapters_few<__half>(a, s);
  return adapters_few<__nv_bfloat16>(a, s);
}

size_t adapters_backward_bytes(int64_t T, int64_t r) { return (size_t)(2 * T * r) * 4; }

cudaError_t launch_adapters_backward(const AdapterGradArgs& a, int dtype, cudaStream_t s) {
  note_kernel_name("k_adapters_grad_w");
  if (dtype == IMC_F32) return backward<float>(a, s);
  if (dtype == IMC_F16) return backward<__half>(a, s);
  return backward<__nv_bfloat16>(a, s);
}

}  // namespace mx
}  // namespace imc
