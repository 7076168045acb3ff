// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = base[t] + scale[l] * (x[t] a[l]^T) b[l]^T,   l the adapter of row t,
//
// and their gradients.  The rows come in adapter order (moe_layout).
#include "adapters.cuh"
#include "ptx.cuh"
#include "scores.cuh"
#include "tc_common.cuh"

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

// ------------------------------------------------------------------- tiles
// More rows: 128 rows of one adapter per cluster, on the tensor cores (tcgen05, bf16
// operands, fp32 accumulators).  CTA q of C takes a run of K for the tile's h = x a^T
// [128, r]; the cluster's sums are taken in the order of the CTAs, each CTA for 128 / C
// rows, which it gives to all of them; then every CTA takes a run of the N outputs.
// x is read once, base and out once, and h never leaves the cluster.
//
// A value is P bf16 numbers (bf16 1, fp16 2, fp32 3: exact) and an element of h PH (2 for
// the 16-bit types, 3 for fp32), one "plane" each.  The planes of the small operand lie
// one after the other along the MMA's N, so a plane of x is read once by the tensor core
// for all of them; the sums over the planes are taken in fp32 afterwards.
constexpr int TILE = 128;            // rows of a tile: the MMA's M
constexpr int KB = 64;               // values of K per stage: 128 bytes of a plane's row
constexpr int XP = TILE * KB * 2;    // bytes of a plane of a stage's x
constexpr int UP_N = 128;            // outputs of one step of the second product
constexpr int EPI_PITCH = 36;        // floats per staged row of the epilogue
constexpr int EPI_BYTES = kWarps * 32 * EPI_PITCH * 4;
// Core matrices (8 rows x 16 bytes) of the operands along r: 144 bytes apart over the
// rows, so that writes along either axis spread over the banks.
constexpr int CORE = 144;
constexpr int CORES = TILE / 8;
constexpr int CORE_K = CORE * CORES;  // apart over r

__device__ int g_watchdog_adapters;

template <typename T>
struct Planes;
template <>
struct Planes<__nv_bfloat16> {
  static constexpr int P = 1, PH = 2, DEPTH = 2, STAGES = 3;
};
template <>
struct Planes<__half> {
  static constexpr int P = 2, PH = 2, DEPTH = 2, STAGES = 2;
};
template <>
struct Planes<float> {
  static constexpr int P = 3, PH = 3, DEPTH = 1, STAGES = 1;
};

// Eight values of a row as they lie in memory.
template <typename T>
struct Raw8 {
  static constexpr int W = (int)sizeof(T) / 2;
  uint4 w[W];
  __device__ __forceinline__ void load(const T* p, int n, bool vec) {
    if (vec && n >= 8) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    } else {
      alignas(16) T t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = i < n ? p[i] : from_f32<T>(0.0f);
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint4*>(t)[i];
    }
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    alignas(16) T t[8];
#pragma unroll
    for (int i = 0; i < W; ++i) reinterpret_cast<uint4*>(t)[i] = w[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32<T>(t[i]);
  }
};

// v as the sum of Q bf16 numbers, each the nearest to what is left: 8, 16 or 24 bits.
// An infinity stays in the first.
template <int Q>
__device__ __forceinline__ void split8(float (&v)[8], uint4 (&out)[Q]) {
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
      if (q + 1 < Q) {
        const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xFFFF0000u);
        v[2 * i] = fabsf(a) == INFINITY ? 0.0f : v[2 * i] - a;
        v[2 * i + 1] = fabsf(b) == INFINITY ? 0.0f : v[2 * i + 1] - b;
      }
    }
    out[q] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <typename T>
__device__ __forceinline__ void planes_of(const Raw8<T>& raw, uint4 (&out)[Planes<T>::P]) {
  if constexpr (Planes<T>::P == 1) {
    out[0] = raw.w[0];
  } else {
    float v[8];
    raw.widen(v);
    split8<Planes<T>::P>(v, out);
  }
}
__device__ __forceinline__ uint16_t half_of(const uint4& u, int i) {
  const uint32_t w = i < 2 ? u.x : (i < 4 ? u.y : (i < 6 ? u.z : u.w));
  return (uint16_t)(i & 1 ? w >> 16 : w);
}

struct TileProblem {
  const void* x;        // [T, K], rows ld elements apart
  int64_t ld, K;
  const void* w1;       // of an adapter [r, K]; turned: [K, r]
  uint16_t* h;          // planes [PH][T][R] of h in adapter order, or null
  const void* w2;       // of an adapter [N, r]; turned: [r, N]
  const void* base;
  void* out;            // null: h alone
  int64_t N;
  int turned, vec;      // vec: 1 x, 2 w1, 4 w2, 8 base and out
};
struct TileArgs {
  TileProblem prob[2];
  const float* scale;
  const int32_t *offsets, *order;
  int64_t T;
  int L, r, R;          // R: r rounded up to 16
  int log_ctas, stages, area, cols;  // area: bytes of the stages and what follows them there
};

struct TileCtl {
  uint64_t empty[4], up, drain;
  uint32_t tmem_base;
  int abort;
  int rows[TILE];
};

template <typename T, int RU>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && RU == 1 ? 3 : 1)
    k_adapters_tile(const __grid_constant__ TileArgs g) {
  using PL = Planes<T>;
  constexpr int P = PL::P, PH = PL::PH, DEPTH = PL::DEPTH;
  extern __shared__ uint8_t sm_raw[];
  __shared__ TileCtl ctl;
  uint8_t* sm = tc::smem_align1024(sm_raw);
  const TileProblem& p = g.prob[blockIdx.y];
  const int C = 1 << g.log_ctas, rank = (int)ptx::cluster_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, R = g.R, r = g.r;
  int* wd = &g_watchdog_adapters;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) ptx::mbar_init(&ctl.empty[i], 1);
    ptx::mbar_init(&ctl.up, 1);
    ptx::mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    ptx::fence_mbar_init();
  }
  // Tensor memory before the stream's next kernel may start: a block of that one that had
  // taken it would wait for this kernel's end.
  if (warp == 0) {
    ptx::tmem_alloc(&ctl.tmem_base, g.cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  ptx::cluster_arrive();  // this CTA runs: its shared memory may be accessed
  ptx::griddep_wait();
  ptx::griddep_launch();
  const bool none = p.out && p.base != p.out;
  const RowTile t = find_tile(g.offsets, g.L, none, TILE, blockIdx.x >> g.log_ctas);
  if (tid < TILE) ctl.rows[tid] = tid < t.rows ? g.order[t.p0 + tid] : -1;
  __syncthreads();
  const int stage_bytes = P * (XP + R * 128);
  uint8_t* hp = sm + g.area;  // planes of h
  const int h_plane = (R >> 3) * CORE_K;
  const int steps = (int)ceil_div(p.N, UP_N), per = (int)ceil_div(steps, C);
  const int s0 = min(rank * per, steps), s1 = p.out ? min(s0 + per, steps) : s0;
  const T* base = static_cast<const T*>(p.base);
  T* out = static_cast<T*>(p.out);
  bool work = t.rows > 0;
  if (work && t.l == g.L) {  // rows without an adapter
    const int64_t n0 = (int64_t)s0 * UP_N, n1 = (int64_t)s1 * UP_N < p.N ? (int64_t)s1 * UP_N : p.N;
    for (int i = warp; i < t.rows; i += kWarps) {
      const int64_t at = ctl.rows[i] * p.N;
      for (int64_t n = n0 + lane * 8; n < n1; n += 256) {
        float v[8];
        const int left = (int)(n1 - n < 8 ? n1 - n : 8);
        if (base) {
          Raw8<T> raw;
          raw.load(base + at + n, left, p.vec & 8);
          if ((p.vec & 8) && left == 8) {
#pragma unroll
            for (int w = 0; w < Raw8<T>::W; ++w) reinterpret_cast<uint4*>(out + at + n)[w] = raw.w[w];
          } else {
            for (int u = 0; u < left; ++u) out[at + n + u] = base[at + n + u];
          }
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u) v[u] = 0.0f;
          store8<T>(out + at + n, left, p.vec & 8, v);
        }
      }
    }
    work = false;
  }
  ptx::cluster_wait();
  if (work) {
    // ---- h = x a^T over this CTA's run of K
    const int blocks = (int)ceil_div(p.K, KB), kper = (int)ceil_div(blocks, C);
    const int b0 = min(rank * kper, blocks), b1 = min(b0 + kper, blocks);
    const T* w1 = static_cast<const T*>(p.w1) + (int64_t)t.l * r * p.K;
    const int u = tid & 7;
    const T* xr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = ctl.rows[(tid >> 3) + 32 * i];
      xr[i] = row < 0 ? nullptr : static_cast<const T*>(p.x) + row * p.ld + u * 8;
    }
    struct Regs {
      Raw8<T> x[4], w[RU];
    };
    auto load = [&](Regs& q, int b) {
      const int64_t k = (int64_t)b * KB;
      const int left = (int)(p.K - k < KB ? p.K - k : KB);
#pragma unroll
      for (int i = 0; i < 4; ++i) q.x[i].load(xr[i] ? xr[i] + k : nullptr, xr[i] ? left - u * 8 : 0, p.vec & 1);
#pragma unroll
      for (int i = 0; i < RU; ++i) {
        if (p.turned) {  // eight j of one k
          const int idx = tid + i * kThreads, kk = idx & 63, j = (idx >> 6) * 8;
          q.w[i].load(w1 + (k + kk) * r + j, kk < left ? r - j : 0, p.vec & 2);
        } else {  // eight k of one j
          const int j = (tid >> 3) + 32 * i;
          q.w[i].load(w1 + j * p.K + k + u * 8, j < r ? left - u * 8 : 0, p.vec & 2);
        }
      }
    };
    auto stage = [&](const Regs& q, uint8_t* to) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = (tid >> 3) + 32 * i;
        uint4 v[P];
        planes_of<T>(q.x[i], v);
#pragma unroll
        for (int c = 0; c < P; ++c)
          *reinterpret_cast<uint4*>(to + c * XP + row * 128 + ((u ^ (row & 7)) << 4)) = v[c];
      }
      uint8_t* wt = to + P * XP;
#pragma unroll
      for (int i = 0; i < RU; ++i) {
        uint4 v[P];
        planes_of<T>(q.w[i], v);
        if (p.turned) {
          const int idx = tid + i * kThreads, kk = idx & 63, j = (idx >> 6) * 8;
          if (j < R) {
#pragma unroll
            for (int c = 0; c < P; ++c)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint16_t*>(wt + (c * R + j + e) * 128 + (((kk >> 3) ^ e) << 4) +
                                             (kk & 7) * 2) = half_of(v[c], e);
          }
        } else {
          const int j = (tid >> 3) + 32 * i;
          if (j < R) {
#pragma unroll
            for (int c = 0; c < P; ++c)
              *reinterpret_cast<uint4*>(wt + (c * R + j) * 128 + ((u ^ (j & 7)) << 4)) = v[c];
          }
        }
      }
    };
    Regs q[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (b0 + d < b1) load(q[d], b0 + d);
    int slot = 0, use = 0;
    for (int b = b0; b < b1; b += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        if (b + d < b1) {
          if (use > 0) tc::warp_wait_bar(&ctl.empty[slot], (use - 1) & 1, &ctl.abort, 1, wd);
          uint8_t* to = sm + slot * stage_bytes;
          stage(q[d], to);
          if (b + d + DEPTH < b1) load(q[d], b + d + DEPTH);
          ptx::fence_proxy_async_smem();
          __syncthreads();
          if (warp == 0 && ptx::elect_one()) {
            ptx::tc_fence_after();
            const uint32_t xa = ptx::smem_addr(to), wa = xa + P * XP;
#pragma unroll
            for (int c = 0; c < P; ++c) {
              const int n = (P == 3 ? 3 - c : P) * R;  // fp32: the smallest products are left out
              for (int n0 = 0; n0 < n; n0 += 256) {
                const int nn = min(256, n - n0);
                const uint32_t id = ptx::idesc_bf16(TILE, nn, false, false);
#pragma unroll
                for (int ks = 0; ks < KB / 16; ++ks)
                  ptx::mma_f16(tmem + n0, ptx::smem_desc(xa + c * XP + ks * 32, 16, 1024, ptx::kSwizzle128B),
                               ptx::smem_desc(wa + n0 * 128 + ks * 32, 16, 1024, ptx::kSwizzle128B), id,
                               b + d > b0 || c > 0 || ks > 0);
              }
            }
            ptx::mma_commit(&ctl.empty[slot]);
          }
          __syncwarp();
          if (++slot == g.stages) {
            slot = 0;
            ++use;
          }
        }
      }
    }
    // ---- this CTA's sums to its shared memory
    const int q4 = warp & 3, pitch = R * 4 + 16;
    if (b1 > b0) {
      const int done = (b1 - b0 - 1) % g.stages, uses = (b1 - b0 - 1) / g.stages;
      tc::warp_wait_bar(&ctl.empty[done], uses & 1, &ctl.abort, 2, wd);
      ptx::tc_fence_after();
    }
    for (int j = (warp >> 2) * 16; j < R; j += 32) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
      if (b1 > b0) {
#pragma unroll
        for (int c = 0; c < P; ++c) {
          uint32_t w[16];
          ptx::tmem_ld16(tmem + ((uint32_t)(q4 * 32) << 16) + c * R + j, w);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(w[i]);
        }
      }
      float4* to = reinterpret_cast<float4*>(sm + (q4 * 32 + lane) * pitch + j * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) to[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
    ptx::tc_fence_before();
  }
  ptx::cluster_sync();
  if (work) {
    // ---- h of 128 / C rows: the sums of all CTAs, in planes to all CTAs
    const int pitch = R * 4 + 16, mine = TILE >> g.log_ctas, units = mine * (R >> 3);
    const float scale = g.scale ? g.scale[t.l] : 1.0f;
    for (int i = tid; i < units; i += kThreads) {
      const int row = rank * mine + (i & (mine - 1)), ju = i >> (7 - g.log_ctas);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.0f;
      for (int c = 0; c < C; ++c) {
        const uint32_t at = ptx::cluster_addr(sm + row * pitch + ju * 32, c);
        const float4 a = ptx::ld_cluster4(at), b = ptx::ld_cluster4(at + 16);
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= scale;
      uint4 w[PH];
      split8<PH>(v, w);
      if (p.h && row < t.rows) {
#pragma unroll
        for (int c = 0; c < PH; ++c)
          *reinterpret_cast<uint4*>(p.h + ((int64_t)c * g.T + t.p0 + row) * R + ju * 8) = w[c];
      }
      if (p.out) {
        uint8_t* to = hp + ju * CORE_K + (row >> 3) * CORE + (row & 7) * 16;
        for (int d = 0; d < C; ++d)
#pragma unroll
          for (int c = 0; c < PH; ++c) ptx::st_cluster4(ptx::cluster_addr(to + c * h_plane, d), w[c]);
      }
    }
    ptx::fence_proxy_async();  // these writes are for the tensor cores
  }
  ptx::cluster_sync();
  if (work && s1 > s0) {
    // ---- out = base + h b^T, UP_N columns at a time
    ptx::fence_proxy_async();
    const T* w2 = static_cast<const T*>(p.w2) + (int64_t)t.l * r * p.N;
    const int q4 = warp & 3, half = warp >> 2;
    float* rows = reinterpret_cast<float*>(sm) + warp * 32 * EPI_PITCH;
    const int er = lane >> 2, ec = (lane & 3) * 8;
    for (int s = s0; s < s1; ++s) {
      const int64_t n0 = (int64_t)s * UP_N;
      const int left = (int)(p.N - n0 < UP_N ? p.N - n0 : UP_N);
      Raw8<T> held[2][4];  // base
      auto fetch = [&](int h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = ctl.rows[q4 * 32 + i * 8 + er], col = half * 64 + h * 32 + ec;
          const bool in = base && row >= 0;
          const T* from = in ? base + row * p.N + n0 + col : nullptr;
          if ((p.vec & 8) && in && left - col >= 8) {  // not __ldg: out may be base
#pragma unroll
            for (int w = 0; w < Raw8<T>::W; ++w)
              held[h][i].w[w] = reinterpret_cast<const uint4*>(from)[w];
          } else {
            alignas(16) T v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = in && e < left - col ? from[e] : from_f32<T>(0.0f);
#pragma unroll
            for (int w = 0; w < Raw8<T>::W; ++w) held[h][i].w[w] = reinterpret_cast<const uint4*>(v)[w];
          }
        }
      };
      fetch(0);
      if (sizeof(T) == 2) fetch(1);
      const int units = CORES * R;  // of eight values
      for (int i = tid; i < units; i += kThreads) {
        Raw8<T> raw;
        uint4 v[P];
        if (p.turned) {  // eight n of one j
          const int j = i % R, nu = i / R;
          raw.load(w2 + j * p.N + n0 + nu * 8, j < r ? left - nu * 8 : 0, p.vec & 4);
          planes_of<T>(raw, v);
#pragma unroll
          for (int c = 0; c < P; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint16_t*>(sm + c * h_plane + (j >> 3) * CORE_K + nu * CORE + e * 16 +
                                           (j & 7) * 2) = half_of(v[c], e);
        } else {  // eight j of one n
          const int n = i & (UP_N - 1), j = (i >> 7) * 8;
          raw.load(w2 + (n0 + n) * r + j, n < left ? r - j : 0, p.vec & 4);
          planes_of<T>(raw, v);
#pragma unroll
          for (int c = 0; c < P; ++c)
            *reinterpret_cast<uint4*>(sm + c * h_plane + (j >> 3) * CORE_K + (n >> 3) * CORE + (n & 7) * 16) = v[c];
        }
      }
      ptx::fence_proxy_async_smem();
      __syncthreads();
      if (warp == 0) {
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint32_t id = ptx::idesc_bf16(TILE, UP_N, false, false);
          const uint32_t ha = ptx::smem_addr(hp), wa = ptx::smem_addr(sm);
          uint32_t more = 0;
          for (int ks = 0; ks < R / 16; ++ks)
#pragma unroll
            for (int c = 0; c < PH; ++c)
#pragma unroll
              for (int d = 0; d < P; ++d) {
                if (P == 3 && c + d > 2) continue;
                ptx::mma_f16(tmem, ptx::smem_desc(ha + c * h_plane + ks * 2 * CORE_K, CORE_K, CORE, 0),
                             ptx::smem_desc(wa + d * h_plane + ks * 2 * CORE_K, CORE_K, CORE, 0), id, more);
                more = 1;
              }
          ptx::mma_commit(&ctl.up);
        }
        __syncwarp();
      }
      tc::warp_wait_bar(&ctl.up, (s - s0) & 1, &ctl.abort, 3, wd);
      ptx::tc_fence_after();
      __syncthreads();  // every warp past the wait: the operand's place is free
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (sizeof(T) == 4 && h == 1) fetch(1);
        uint32_t w[32];
        ptx::tmem_ld32(tmem + ((uint32_t)(q4 * 32) << 16) + half * 64 + h * 32, w);
        ptx::tmem_ld_wait();
        float4* to = reinterpret_cast<float4*>(rows + lane * EPI_PITCH);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          to[i] = make_float4(__uint_as_float(w[4 * i]), __uint_as_float(w[4 * i + 1]),
                              __uint_as_float(w[4 * i + 2]), __uint_as_float(w[4 * i + 3]));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = ctl.rows[q4 * 32 + i * 8 + er], col = half * 64 + h * 32 + ec;
          const float4 a = *reinterpret_cast<const float4*>(rows + (i * 8 + er) * EPI_PITCH + ec);
          const float4 b = *reinterpret_cast<const float4*>(rows + (i * 8 + er) * EPI_PITCH + ec + 4);
          float v[8];
          held[h][i].widen(v);
          v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
          v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
          if (row >= 0 && col < left) store8<T>(out + row * p.N + n0 + col, left - col, p.vec & 8, v);
        }
        __syncwarp();
      }
      ptx::tc_fence_before();
      __syncthreads();
    }
  }
  if (ctl.abort && warp == 0) {  // a wait gave up: no MMA may run on into freed memory
    if (ptx::elect_one()) ptx::mma_commit(&ctl.drain);
    __syncwarp();
    tc::drain_wait(&ctl.drain, 0);
  }
  __syncthreads();
  if (warp == 0) ptx::tmem_dealloc(tmem, g.cols);
}

// ------------------------------------------------------- weights' gradients
// grad_a[l][j][k] = sum over l's rows of g[p][j] x[row][k], and grad_b[l][n][j] with h and
// grad.  A cluster has one adapter and 128 columns of x (or grad): they are the MMA's M,
// the r columns of g its N, the rows its K.  CTA q of S takes a run of the rows; the
// cluster's sums are taken in the order of the CTAs.  A tile of x is loaded by rows, so its
// columns lie along the operand's M ("MN-major"); g's planes are turned on the way.
constexpr int GRAD_ROWS = 64;  // rows per stage
constexpr int GRAD_COLS = 128;

struct GradProblem {
  const void* x;      // [T, cols]
  int64_t cols;
  const uint16_t* h;  // planes [PH][T][R]
  void* out;          // of an adapter [r, cols]; turned: [cols, r]
  int turned, vec;
};
struct GradArgs {
  GradProblem prob[2];
  const int32_t *offsets, *order;
  int64_t T;
  int L, r, R, log_ctas, stages, cols;
};
struct GradCtl {
  uint64_t empty[4], drain;
  uint32_t tmem_base;
  int abort;
};

template <typename T, int RU>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && RU == 1 ? 3 : 1)
    k_adapters_grad(const __grid_constant__ GradArgs g) {
  using PL = Planes<T>;
  constexpr int P = PL::P, PH = PL::PH;
  extern __shared__ uint8_t sm_raw[];
  __shared__ GradCtl ctl;
  uint8_t* sm = tc::smem_align1024(sm_raw);
  const GradProblem& p = g.prob[blockIdx.z];
  const int C = 1 << g.log_ctas, rank = (int)ptx::cluster_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, R = g.R, r = g.r;
  const int64_t col0 = (int64_t)(blockIdx.x >> g.log_ctas) * GRAD_COLS;
  const int l = blockIdx.y;
  int* wd = &g_watchdog_adapters;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) ptx::mbar_init(&ctl.empty[i], 1);
    ptx::mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0) {
    ptx::tmem_alloc(&ctl.tmem_base, g.cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  ptx::griddep_wait();
  ptx::griddep_launch();
  // (the problems may have different numbers of columns)
  const bool work = col0 < p.cols;
  const int first = __ldg(g.offsets + l), rows = __ldg(g.offsets + l + 1) - first;
  const int blocks = (rows + GRAD_ROWS - 1) / GRAD_ROWS, per = (blocks + C - 1) >> g.log_ctas;
  const int b0 = min(rank * per, blocks), b1 = work ? min(b0 + per, blocks) : b0;
  constexpr int XG = GRAD_ROWS * GRAD_COLS * 2;  // bytes of a plane of a stage's x
  const int core_k = (PH * R / 8) * 128 + 16;     // 16 bytes more: writes spread over the banks
  const int stage_bytes = (P * XG + 8 * core_k + 1023) & ~1023;
  const int left = (int)(p.cols - col0 < GRAD_COLS ? p.cols - col0 : GRAD_COLS);
  const int u = tid & 15, xrow = tid >> 4;
  const T* x = static_cast<const T*>(p.x) + col0 + u * 8;
  struct Regs {
    Raw8<T> x[4];
    uint4 h[RU][PH];
  };
  int at[4];  // rows of the next block to be loaded
  auto rows_of = [&](int b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int in = b * GRAD_ROWS + xrow + 16 * i;
      at[i] = b < b1 && in < rows ? __ldg(g.order + first + in) : -1;
    }
  };
  auto load = [&](Regs& q, int b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q.x[i].load(x + at[i] * p.cols, at[i] >= 0 ? left - u * 8 : 0, p.vec);
#pragma unroll
    for (int i = 0; i < RU; ++i) {
      const int idx = tid + i * kThreads, t = idx & 63, j = (idx >> 6) * 8, in = b * GRAD_ROWS + t;
#pragma unroll
      for (int c = 0; c < PH; ++c)
        q.h[i][c] = j < R && in < rows
                        ? __ldg(reinterpret_cast<const uint4*>(p.h + ((int64_t)c * g.T + first + in) * R + j))
                        : make_uint4(0, 0, 0, 0);
    }
  };
  Regs q;
  rows_of(b0);
  if (b0 < b1) load(q, b0);
  rows_of(b0 + 1);
  int slot = 0, use = 0;
  for (int b = b0; b < b1; ++b) {
    if (use > 0) tc::warp_wait_bar(&ctl.empty[slot], (use - 1) & 1, &ctl.abort, 4, wd);
    uint8_t* to = sm + slot * stage_bytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = xrow + 16 * i;
      uint4 v[P];
      planes_of<T>(q.x[i], v);
#pragma unroll
      for (int c = 0; c < P; ++c)
        *reinterpret_cast<uint4*>(to + c * XG + (u >> 3) * (GRAD_ROWS * 128) + row * 128 +
                                  (((u & 7) ^ (row & 7)) << 4)) = v[c];
    }
    uint8_t* ht = to + P * XG;
#pragma unroll
    for (int i = 0; i < RU; ++i) {
      const int idx = tid + i * kThreads, t = idx & 63, j = (idx >> 6) * 8;
      if (j < R) {
#pragma unroll
        for (int c = 0; c < PH; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint16_t*>(ht + (t >> 3) * core_k + ((c * R + j) >> 3) * 128 + e * 16 +
                                         (t & 7) * 2) = half_of(q.h[i][c], e);
      }
    }
    if (b + 1 < b1) {
      load(q, b + 1);
      rows_of(b + 2);
    }
    ptx::fence_proxy_async_smem();
    __syncthreads();
    if (warp == 0) {
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        const uint32_t xa = ptx::smem_addr(to), ha = xa + P * XG;
#pragma unroll
        for (int c = 0; c < P; ++c) {
          const int n = (P == 3 ? 3 - c : PH) * R;
          for (int n0 = 0; n0 < n; n0 += 256) {
            const int nn = min(256, n - n0);
            const uint32_t id = ptx::idesc_bf16(GRAD_COLS, nn, true, false);
#pragma unroll
            for (int ks = 0; ks < GRAD_ROWS / 16; ++ks)
              ptx::mma_f16(tmem + n0,
                           ptx::smem_desc(xa + c * XG + ks * 2048, GRAD_ROWS * 128, 1024, ptx::kSwizzle128B),
                           ptx::smem_desc(ha + (n0 >> 3) * 128 + ks * 2 * core_k, core_k, 128, 0), id,
                           b > b0 || c > 0 || ks > 0);
          }
        }
        ptx::mma_commit(&ctl.empty[slot]);
      }
      __syncwarp();
    }
    if (++slot == g.stages) {
      slot = 0;
      ++use;
    }
  }
  const int pitch = R + 1;  // words of a column's sums
  float* part = reinterpret_cast<float*>(sm);
  if (b1 > b0) {
    const int done = (b1 - b0 - 1) % g.stages, uses = (b1 - b0 - 1) / g.stages;
    tc::warp_wait_bar(&ctl.empty[done], uses & 1, &ctl.abort, 5, wd);
    ptx::tc_fence_after();
  }
  __syncthreads();
  if (work) {
    const int q4 = warp & 3;
    for (int j = (warp >> 2) * 16; j < R; j += 32) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
      if (b1 > b0) {
#pragma unroll
        for (int c = 0; c < PH; ++c) {
          uint32_t w[16];
          ptx::tmem_ld16(tmem + ((uint32_t)(q4 * 32) << 16) + c * R + j, w);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(w[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) part[(q4 * 32 + lane) * pitch + j + i] = v[i];
    }
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  if (work) {
    const int n = left * r, share = (n + C - 1) >> g.log_ctas;
    const int e0 = rank * share, e1 = min(e0 + share, n);
    T* out = static_cast<T*>(p.out) + (int64_t)l * r * p.cols;
    for (int e = e0 + tid; e < e1; e += kThreads) {
      const int col = p.turned ? e / r : e % left, j = p.turned ? e - col * r : e / left;
      float sum = 0.0f;
      for (int c = 0; c < C; ++c)
        sum += __uint_as_float(ptx::ld_cluster(ptx::cluster_addr(part + col * pitch + j, c)));
      out[p.turned ? (col0 + col) * r + j : (int64_t)j * p.cols + col0 + col] = from_f32<T>(sum);
    }
  }
  ptx::cluster_sync();  // no CTA ends while another reads its sums
  if (ctl.abort && warp == 0) {
    if (ptx::elect_one()) ptx::mma_commit(&ctl.drain);
    __syncwarp();
    tc::drain_wait(&ctl.drain, 0);
  }
  __syncthreads();
  if (warp == 0) ptx::tmem_dealloc(tmem, g.cols);
}

// ------------------------------------------------------------------- host
bool aligned16(const void* p, int64_t pitch_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)pitch_bytes) & 15u) == 0;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 grid, int ctas, size_t smem, cudaStream_t s,
                            Args... args) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, args...);
  note_launch();
  return e;
}

// Tensor-memory columns of a block: a power of two that holds `need`.
int tmem_cols(int need) {
  int c = 32;
  while (c < need) c *= 2;
  return c;
}
// Shared memory of a block that takes `cols` of an SM's 512 tensor-memory columns: at least
// that share of the SM's 228 KB.  Blocks that fit on an SM together then find their tensor
// memory too, so none waits for it inside a cluster whose other blocks hold theirs on an SM
// where another cluster's block waits.
size_t smem_for(size_t bytes, int cols) {
  const size_t share = (size_t)(228 << 10) * cols / 512 - 1024, most = 232448 - 2048;
  bytes = bytes > share ? bytes : share;
  return bytes < most ? bytes : most;
}

template <typename T>
cudaError_t adapters_few(const AdapterArgs& a, cudaStream_t s) {
  note_kernel_name("k_adapters_few");
  const int log_ctas = 3;
  const int none = a.base != a.out ? 1 : 0;
  const int64_t tiles = most_tiles(a.T, a.L, FEW);
  const int64_t b = sizeof(T);
  const int flags = (aligned16(a.x, a.ld * b) ? 1 : 0) | (aligned16(a.a, a.K * b) ? 2 : 0) |
                    (aligned16(a.b, a.r * b) ? 4 : 0);
  const size_t smem = (size_t)(FEW * KC + (FEW + (FEW << log_ctas)) * a.r) * 4;
  return launch_clusters(k_adapters_few<T>, dim3((unsigned)(tiles << log_ctas)), 1 << log_ctas, smem, s, a,
                         log_ctas, none, flags);
}

// The kernel form by r rounded up to 16.
#define IMC_BY_RANK(R, CALL) \
  do {                       \
    if ((R) <= 32) CALL(1);  \
    if ((R) <= 64) CALL(2);  \
    CALL(4);                 \
  } while (0)

int log2_up(int64_t v) {
  int n = 0;
  while (((int64_t)1 << n) < v) ++n;
  return n;
}

template <typename T>
cudaError_t run_tiles(TileArgs g, int problems, cudaStream_t s) {
  using PL = Planes<T>;
  g.R = (g.r + 15) / 16 * 16;
  const int64_t tiles = most_tiles(g.T, g.L, TILE);
  // about three blocks per SM
  const int64_t want = 3 * (int64_t)device_sm_count() / (ceil_div(g.T, TILE) * problems);
  g.log_ctas = want >= 8 ? 3 : log2_up(want < 1 ? 1 : want);
  const int stage = PL::P * (XP + g.R * 128), h_plane = g.R / 8 * CORE_K;
  g.stages = g.R > 64 && PL::STAGES > 2 ? 2 : PL::STAGES;
  if (PL::P == 2 && g.R > 64) g.stages = 1;
  int area = g.stages * stage;
  const int others[3] = {TILE * (g.R * 4 + 16), PL::P * h_plane, EPI_BYTES};
  for (int o : others) area = area > o ? area : o;
  g.area = (area + 1023) / 1024 * 1024;
  g.cols = tmem_cols(PL::P * g.R > UP_N ? PL::P * g.R : UP_N);
  const size_t smem = smem_for((size_t)g.area + PL::PH * h_plane + 1024, g.cols);
  const dim3 grid((unsigned)(tiles << g.log_ctas), problems);
#define IMC_TILES(RU) return launch_clusters(k_adapters_tile<T, RU>, grid, 1 << g.log_ctas, smem, s, g)
  IMC_BY_RANK(g.R, IMC_TILES);
#undef IMC_TILES
}

// Alignment for 16-byte accesses of each operand of a problem.
template <typename T>
int tile_vec(const TileProblem& p, int r) {
  const int64_t b = sizeof(T);
  return (aligned16(p.x, p.ld * b) ? 1 : 0) | (aligned16(p.w1, (p.turned ? r : p.K) * b) ? 2 : 0) |
         (aligned16(p.w2, (p.turned ? p.N : r) * b) ? 4 : 0) |
         (aligned16(p.out, p.N * b) && aligned16(p.base, 0) ? 8 : 0);
}

template <typename T>
cudaError_t adapters(const AdapterArgs& a, cudaStream_t s) {
  if (a.T <= 64) return adapters_few<T>(a, s);
  note_kernel_name("k_adapters_tile");
  TileArgs g = {};
  TileProblem& p = g.prob[0];
  p.x = a.x;
  p.ld = a.ld;
  p.K = a.K;
  p.w1 = a.a;
  p.w2 = a.b;
  p.base = a.base;
  p.out = a.out;
  p.N = a.N;
  p.vec = tile_vec<T>(p, a.r);
  g.scale = a.scale;
  g.offsets = a.offsets;
  g.order = a.order;
  g.T = a.T;
  g.L = a.L;
  g.r = a.r;
  return run_tiles<T>(g, 1, s);
}

size_t planes_bytes(int64_t T, int64_t r) {  // of h or g, whatever their type
  return (size_t)(3 * T * ((r + 15) / 16 * 16) * 2);
}

template <typename T>
cudaError_t backward(const AdapterGradArgs& a, cudaStream_t s) {
  using PL = Planes<T>;
  note_kernel_name("k_adapters_grad");
  uint16_t* h = static_cast<uint16_t*>(a.workspace);
  uint16_t* d = h + planes_bytes(a.T, a.r) / 2;
  TileArgs g = {};
  g.scale = a.scale;
  g.offsets = a.offsets;
  g.order = a.order;
  g.T = a.T;
  g.L = a.L;
  g.r = a.r;
  int problems = 0;
  if (a.grad_x || a.grad_a) {  // g = scale * grad b, and grad_x = base + g a
    TileProblem& p = g.prob[problems++];
    p.x = a.grad;
    p.ld = p.K = a.N;
    p.w1 = a.b;
    p.w2 = a.a;
    p.h = a.grad_a ? d : nullptr;
    p.base = a.base;
    p.out = a.grad_x;
    p.N = a.grad_x ? a.K : 0;
    p.turned = 1;
    p.vec = tile_vec<T>(p, a.r);
  }
  if (a.grad_b) {  // h = scale * x a^T
    TileProblem& p = g.prob[problems++];
    p.x = a.x;
    p.ld = p.K = a.K;
    p.w1 = a.a;
    p.h = h;
    p.vec = tile_vec<T>(p, a.r);
  }
  cudaError_t e = run_tiles<T>(g, problems, s);
  if (e != cudaSuccess || (!a.grad_a && !a.grad_b)) return e;
  GradArgs w = {};
  w.offsets = a.offsets;
  w.order = a.order;
  w.T = a.T;
  w.L = a.L;
  w.r = a.r;
  w.R = (a.r + 15) / 16 * 16;
  int parts = 0;
  int64_t chunks = 0, all = 0;
  auto add = [&](const void* x, int64_t cols, const uint16_t* planes, void* out, int turned) {
    GradProblem& p = w.prob[parts++];
    p.x = x;
    p.cols = cols;
    p.h = planes;
    p.out = out;
    p.turned = turned;
    p.vec = aligned16(x, cols * (int64_t)sizeof(T)) ? 1 : 0;
    const int64_t n = ceil_div(cols, GRAD_COLS);
    chunks = chunks > n ? chunks : n;
    all += n;
  };
  if (a.grad_a) add(a.x, a.K, d, a.grad_a, 0);
  if (a.grad_b) add(a.grad, a.N, h, a.grad_b, 1);
  // about three blocks per SM, of four stages of rows on average at least
  int64_t want = 3 * (int64_t)device_sm_count() / (all * a.L);
  const int64_t most = a.T / a.L / (4 * GRAD_ROWS);
  want = want < most ? want : most;
  w.log_ctas = want >= 8 ? 3 : log2_up(want < 1 ? 1 : want);
  const int stage = (PL::P * GRAD_ROWS * GRAD_COLS * 2 + 8 * (PL::PH * w.R / 8 * 128 + 16) + 1023) / 1024 * 1024;
  w.stages = PL::P == 1 && w.R <= 64 ? 3 : (PL::P == 3 || w.R > 64 ? 1 : 2);
  size_t bytes = (size_t)w.stages * stage, sums = (size_t)GRAD_COLS * (w.R + 1) * 4;
  bytes = bytes > sums ? bytes : sums;
  w.cols = tmem_cols(PL::PH * w.R);
  const size_t smem = smem_for(bytes + 1024, w.cols);
  const dim3 grid((unsigned)(chunks << w.log_ctas), a.L, parts);
#define IMC_GRADS(RU) return launch_clusters(k_adapters_grad<T, RU>, grid, 1 << w.log_ctas, smem, s, w)
  IMC_BY_RANK(w.R, IMC_GRADS);
#undef IMC_GRADS
}

}  // namespace

cudaError_t launch_adapters(const AdapterArgs& a, int dtype, cudaStream_t s) {
  if (dtype == IMC_F32) return adapters<float>(a, s);
  if (dtype == IMC_F16) return adapters<__half>(a, s);
  return adapters<__nv_bfloat16>(a, s);
}

size_t adapters_backward_bytes(int64_t T, int64_t r) { return 2 * planes_bytes(T, r); }

cudaError_t launch_adapters_backward(const AdapterGradArgs& a, int dtype, cudaStream_t s) {
  if (dtype == IMC_F32) return backward<float>(a, s);
  if (dtype == IMC_F16) return backward<__half>(a, s);
  return backward<__nv_bfloat16>(a, s);
}

cudaError_t adapters_take_watchdog(int* value) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_watchdog_adapters, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_watchdog_adapters, &zero, sizeof(int));
}

}  // namespace mx
}  // namespace imc
