// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = base[t] + scale[l] * (x[t] a[l]^T) b[l]^T,   l the adapter of row t,
//
// and their gradients.  The rows come in adapter order (moe_layout).  Forms: few rows, one
// launch (k_adapters_few); tiles of 128 rows, two (k_adapters_down or _down_tma, then _up);
// the gradient of x the same two with the weights' roles exchanged; the weights' gradients
// k_adapters_grad, _grad_runs or, for a handful of rows each, _grad_fma.
#include <mutex>
#include <type_traits>

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
template <int THREADS = kThreads>
__device__ __forceinline__ RowTile find_tile(const int32_t* offsets, int L, bool none, int height,
                                             int t) {
  __shared__ int sums[THREADS / 32];
  __shared__ RowTile found;
  const int B = L + (none ? 1 : 0), per = (B + THREADS - 1) / THREADS;
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
  for (int w = 0; w < THREADS / 32; ++w)
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
// All tiles of the buckets 0 .. B - 1: first [B + 1] (or null), the buckets' first places, and
// before [B + 1], the tiles before each.  All threads of the block; ends with a barrier.
template <int THREADS>
__device__ __forceinline__ void count_tiles(const int32_t* offsets, int B, int height, int* first, int* before,
                                            int* sums) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (B + THREADS - 1) / THREADS, e0 = tid * per;
  int tiles = 0;
  for (int e = e0; e < e0 + per && e < B; ++e) {
    const int at = __ldg(offsets + e);
    if (first) first[e] = at;
    tiles += (__ldg(offsets + e + 1) - at + height - 1) / height;
  }
  if (tid == 0 && first) first[B] = __ldg(offsets + B);
  int upto = tiles;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(kAll, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += sums[w];
  int at = upto - tiles;
  for (int e = e0; e < e0 + per && e < B; ++e) {
    before[e] = at;
    at += (__ldg(offsets + e + 1) - __ldg(offsets + e) + height - 1) / height;
  }
  if (tid == THREADS - 1) before[B] = upto;
  __syncthreads();
}
// At least as many tiles as any distribution of T rows over the buckets has.
int64_t most_tiles(int64_t T, int64_t L, int height) {
  const int64_t buckets = T < L + 1 ? T : L + 1;
  return (T + (height - 1) * buckets) / height;
}

template <typename T>
struct Planes;
// P: planes of a value where it has to be bf16 (gradients of the weights); PD and FD: planes
// and format (0 fp16, 1 bf16) of one in the two products with a and b, which take fp16 as
// it is; PH: planes of an element of h; stages of the rings.
template <>
struct Planes<__nv_bfloat16> {
  static constexpr int P = 1, PD = 1, FD = 1, PH = 2, STAGES = 4, GRAD_STAGES = 3;
};
template <>
struct Planes<__half> {
  static constexpr int P = 2, PD = 1, FD = 0, PH = 2, STAGES = 4, GRAD_STAGES = 2;
};
template <>
struct Planes<float> {
  static constexpr int P = 3, PD = 3, FD = 1, PH = 3, STAGES = 2, GRAD_STAGES = 2;
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
  // The same from rows aligned to `piece` bytes; 16-bit values at odd places by the words that
  // hold them, the halves that are not theirs dropped.
  __device__ __forceinline__ void load_by(const T* p, int n, int piece) {
    if (sizeof(T) == 2 && n >= 8 && piece == 2) {
      const uint32_t odd = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 2);
      const uint32_t* from = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(p) - odd);
      uint32_t v[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) v[i] = i < 4 || odd ? __ldg(from + i) : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(w)[i] = __funnelshift_r(v[i], v[i + 1], odd * 8);
    } else if (n >= 8 && piece == 8) {
#pragma unroll
      for (int i = 0; i < 2 * W; ++i) reinterpret_cast<uint2*>(w)[i] = __ldg(reinterpret_cast<const uint2*>(p) + i);
    } else if (n >= 8 && piece == 4) {
#pragma unroll
      for (int i = 0; i < 4 * W; ++i) reinterpret_cast<uint32_t*>(w)[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
    } else {
      load(p, n, piece == 16);
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

// ---------------------------------------------------------------- few rows
// Up to FEW rows of one adapter per cluster of CTAs, in one launch.  CTA q takes a run of K
// for h = x a^T, gives its partial sums to every CTA of the cluster (summed in the order of
// the CTAs), and then a run of the N outputs.  Such a call is bound by latency: of the loads
// that wait for one another, and of fetching instructions that run once.  So the loops are
// short: both products use mma.sync (a warp's small tiles need no shared memory and no
// barriers, unlike tcgen05's), whose operands come straight from global memory, sixteen
// bytes a lane: the order of the values along the summed axis is the same for both operands,
// whatever it is.  One row of 8 adapters, r 16, 4096 x 4096, bf16, takes 5.8 us, 64 rows of 64
// adapters, 4096 x 1024, 7.2 (10.5 MB of weights: 1.5 TB/s).
constexpr int FEW = 8;
constexpr int FEW_ROWS = 1024;  // rows whose numbers are asked for before the tile is known
constexpr int FEW_N = 512;      // outputs staged at once
constexpr int FEW_PITCH = FEW_N + 8;

// Four values of a row.
template <typename T>
struct Raw4 {
  uint32_t w[sizeof(T)];
  __device__ __forceinline__ void load(const T* p, int n, bool vec) {
    if (vec && n >= 4) {
      if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(w) = __ldg(reinterpret_cast<const uint2*>(p));
      else *reinterpret_cast<uint4*>(w) = __ldg(reinterpret_cast<const uint4*>(p));
    } else {
      T t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = i < n ? p[i] : from_f32<T>(0.0f);
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w[i] = *reinterpret_cast<const uint16_t*>(t + 2 * i) | (uint32_t)*reinterpret_cast<const uint16_t*>(t + 2 * i + 1) << 16;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(t + i);
      }
    }
  }
  __device__ __forceinline__ void widen(float (&v)[4]) const {
    alignas(16) T t[4];
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) reinterpret_cast<uint32_t*>(t)[i] = w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = to_f32<T>(t[i]);
  }
};
// d += A B of a warp: sixteen rows of A (this lane's words of row lane / 4 in a, of the eighth
// after it in a8) and eight columns of B (of column lane / 4 in b).  16-bit types: K = 16, two
// words of two values; fp32: K = 8, two words, as three products of TF32 parts, the small ones
// summed apart (e): the tensor core truncates its sums.
__device__ __forceinline__ void few_mma(__nv_bfloat16, float (&d)[4], float (&)[4], const uint32_t* a, const uint32_t* a8, const uint32_t* b) {
  ptx::mma_sync_bf16(d, a[0], a8[0], a[1], a8[1], b[0], b[1]);
}
__device__ __forceinline__ void few_mma(__half, float (&d)[4], float (&)[4], const uint32_t* a, const uint32_t* a8, const uint32_t* b) {
  ptx::mma_sync_f16(d, a[0], a8[0], a[1], a8[1], b[0], b[1]);
}
__device__ __forceinline__ void few_mma(float, float (&d)[4], float (&e)[4], const uint32_t* a, const uint32_t* a8, const uint32_t* b) {
  auto hi = [](uint32_t v) { return __float_as_uint(tc::tf32_hi(__uint_as_float(v))); };
  auto lo = [](uint32_t v) { return __float_as_uint(tc::tf32_lo(__uint_as_float(v))); };
  ptx::mma_sync_tf32(e, lo(a[0]), lo(a8[0]), lo(a[1]), lo(a8[1]), hi(b[0]), hi(b[1]));
  ptx::mma_sync_tf32(e, hi(a[0]), hi(a8[0]), hi(a[1]), hi(a8[1]), lo(b[0]), lo(b[1]));
  ptx::mma_sync_tf32(d, hi(a[0]), hi(a8[0]), hi(a[1]), hi(a8[1]), hi(b[0]), hi(b[1]));
}

struct FewArgs {
  AdapterArgs a;
  int log_ctas, none, vec;  // vec: 1 x, 2 a (16 bytes), 4 b (four values)
  int R, blocks, parts;     // r rounded up to 16; blocks of 16 of it; warps that share one
};

// (fp32 with three blocks an SM spills registers: 512 rows of 4 adapters, r 16, 1024 x 1024, 11.4 us for 8.5)
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : 3) k_adapters_few(const __grid_constant__ FewArgs g) {
  extern __shared__ uint8_t sm_raw[];
  __shared__ int order[FEW_ROWS], rows[FEW];
  __shared__ float row_scale[FEW];
  uint8_t* sm = sm_raw;
  using O = std::conditional_t<sizeof(T) == 4, float, T>;  // of h's two parts
  const AdapterArgs& p = g.a;
  const int rank = (int)ptx::cluster_rank(), C = 1 << g.log_ctas, R = g.R, r = p.r;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row8 = lane >> 2, quad = lane & 3;
  float* part = reinterpret_cast<float*>(sm);     // [parts][FEW][R]
  float* gathered = part + g.parts * FEW * R;     // [C][FEW][R]
  const int h_pitch = R + 16 / (int)sizeof(O);
  O* hs = reinterpret_cast<O*>(gathered + C * FEW * R);                   // two parts of [FEW][h_pitch]
  float* outs = reinterpret_cast<float*>(hs + 2 * FEW * h_pitch);         // [FEW][FEW_PITCH]
  ptx::griddep_wait();
  ptx::griddep_launch();
#pragma unroll
  for (int i = 0; i < FEW_ROWS / kThreads; ++i) {
    const int at = tid + i * kThreads;
    if (at < p.T) order[at] = __ldg(p.order + at);
  }
  const RowTile t = find_tile(p.offsets, p.L, g.none != 0, FEW, blockIdx.x >> g.log_ctas);
  if (t.rows == 0) return;  // the whole cluster
  ptx::cluster_arrive();    // this CTA runs: its shared memory may be written
  if (tid < FEW) {          // past the tile's end the last one again
    const int at = t.p0 + min(tid, t.rows - 1);
    rows[tid] = at < FEW_ROWS ? order[at] : __ldg(p.order + at);
  }
  __syncthreads();
  const T* base = static_cast<const T*>(p.base);
  T* out = static_cast<T*>(p.out);
  const int64_t n_per = (((p.N + C - 1) >> g.log_ctas) + 15) & ~15ll, n0 = rank * n_per < p.N ? rank * n_per : p.N;
  const int64_t n1 = n0 + n_per < p.N ? n0 + n_per : p.N;
  const bool product = t.l < p.L;
  if (product) {
    const T* a = static_cast<const T*>(p.a) + (int64_t)t.l * r * p.K;
    const T* b = static_cast<const T*>(p.b) + (int64_t)t.l * p.N * r;
    // The second product's units, sixteen outputs by sixteen j each, four at a time: the
    // first four are asked for here, as well as the first of base.  The rest of b is on its
    // way to L2.
    const int live0 = (int)(n1 - n0 < FEW_N ? n1 - n0 : FEW_N);
    constexpr int Q = 4;
    Raw4<T> w[Q], w8[Q];
    const T* from;  // this lane's values of the next unit to be asked for
    int ask_nb, ask_j;
    auto start_b = [&](int64_t n) {
      ask_nb = warp * 16;
      ask_j = 0;
      from = b + (n + ask_nb + row8) * r + quad * 4;
    };
    // (`full`: sixteen outputs, sixteen j, aligned; a third of the other's instructions)
    auto load_b = [&](auto full, int64_t n, int live) {
#pragma unroll
      for (int u = 0; u < Q; ++u) {
        if (ask_nb < live) {
          if constexpr (full) {
            w[u].load(from, 4, true);
            w8[u].load(from + 8 * r, 4, true);
          } else {
            const int64_t row = n + ask_nb + row8;
            const int left = r - ask_j - quad * 4;
            w[u].load(from, row < n1 ? left : 0, g.vec & 4);
            w8[u].load(from + 8 * r, row + 8 < n1 ? left : 0, g.vec & 4);
          }
          from += 16;
          ask_j += 16;
          if (ask_j == R) {
            ask_j = 0;
            ask_nb += kWarps * 16;
            from += (int64_t)kWarps * 16 * r - R;
          }
        }
      }
    };
    const bool whole_b = (g.vec & 4) && r == R;
    auto any_b = [&](int64_t n, int live) {
      if (whole_b && live % 16 == 0) load_b(std::true_type{}, n, live);
      else load_b(std::false_type{}, n, live);
    };
    start_b(n0);
    any_b(n0, live0);
    T was[Q];
#pragma unroll
    for (int u = 0; u < Q; ++u) {
      const int i = tid + u * kThreads, row = live0 ? i / live0 : FEW;
      was[u] = base && row < t.rows ? base[rows[row & (FEW - 1)] * p.N + n0 + i - row * live0] : from_f32<T>(0.0f);
    }
    const int64_t bytes = (n1 - n0) * r * (int64_t)sizeof(T);
    for (int64_t i = tid * 128; i < bytes; i += kThreads * 128)
      ptx::prefetch_l2(reinterpret_cast<const uint8_t*>(b + n0 * r) + i);
    // ---- h = x a^T over this CTA's run of K: a warp has sixteen j and a part of the run
    const int64_t k_per = (((p.K + C - 1) >> g.log_ctas) + 31) & ~31ll, k0 = rank * k_per < p.K ? rank * k_per : p.K;
    const int64_t k1 = k0 + k_per < p.K ? k0 + k_per : p.K;
    if (warp < g.blocks * g.parts) {
      const int block = warp % g.blocks, share = warp / g.blocks, j = block * 16 + row8;
      const T *wa = a + j * p.K, *wa8 = wa + 8 * p.K, *x = static_cast<const T*>(p.x) + rows[row8] * p.ld;
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f}, e[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      auto step = [&](const Raw8<T>& u, const Raw8<T>& u8, const Raw8<T>& v) {
        const uint32_t *aw = reinterpret_cast<const uint32_t*>(u.w), *aw8 = reinterpret_cast<const uint32_t*>(u8.w),
                       *bw = reinterpret_cast<const uint32_t*>(v.w);
#pragma unroll
        for (int i = 0; i < 2 * (int)sizeof(T); i += 2) few_mma(T(), d, e, aw + i, aw8 + i, bw + i);
      };
      const int first = share * 32, len = (int)(k1 - k0), stride = g.parts * 32;
      int at = first;
      wa += k0 + quad * 8, wa8 += k0 + quad * 8, x += k0 + quad * 8;
      if ((g.vec & 3) == 3 && r == R) {  // whole units
#pragma unroll 4
        for (; at + 32 <= len; at += stride) {
          Raw8<T> u, u8, v;
          u.load(wa + at, 8, true);
          u8.load(wa8 + at, 8, true);
          v.load(x + at, 8, true);
          step(u, u8, v);
        }
      }
#pragma unroll 1
      for (; at < len; at += stride) {
        const int left = len - at - quad * 8;
        Raw8<T> u, u8, v;
        u.load(wa + at, j < r ? left : 0, g.vec & 2);
        u8.load(wa8 + at, j + 8 < r ? left : 0, g.vec & 2);
        v.load(x + at, left, g.vec & 1);
        step(u, u8, v);
      }
      float* to = part + (share * FEW + quad * 2) * R + j;
      to[0] = d[0] + e[0], to[R] = d[1] + e[1], to[8] = d[2] + e[2], to[R + 8] = d[3] + e[3];
    }
    const float scale = p.scale ? p.scale[t.l] : 1.0f;
    __syncthreads();
    ptx::cluster_wait();
    const int units = FEW * R / 4;
    for (int i = tid; i < units * C; i += kThreads) {
      const int q = i / units, e = (i - q * units) * 4;
      float4 s = *reinterpret_cast<const float4*>(part + e);
      for (int u = 1; u < g.parts; ++u) {
        const float4 v = *reinterpret_cast<const float4*>(part + u * FEW * R + e);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
      }
      ptx::st_cluster4(ptx::cluster_addr(gathered + rank * FEW * R + e, q),
                       make_uint4(__float_as_uint(s.x), __float_as_uint(s.y), __float_as_uint(s.z), __float_as_uint(s.w)));
    }
    ptx::cluster_sync();
    // ---- h in two parts (fp16: the row's largest value brought to 2^14 .. 2^15); a warp a row
    {
      float top = 0.0f;
      float* mine = gathered + warp * R;
      for (int i = lane; i < R; i += 32) {
        float s = 0.0f;
        for (int q = 0; q < C; ++q) s += mine[q * FEW * R + i];
        s = i < r ? s * scale : 0.0f;  // past r: zeros times x, which may be infinite
        mine[i] = s;
        top = fmaxf(top, fabsf(s));
      }
      float up = 1.0f;
      if (Planes<T>::FD == 0) {
        top = warp_max(top);
        uint32_t e8 = __float_as_uint(top) >> 23;
        e8 = e8 == 255u || top == 0.0f ? 141u : max(e8, 15u);
        up = __uint_as_float((268u - e8) << 23);
        if (lane == 0) row_scale[warp] = __uint_as_float((e8 - 14u) << 23);
      } else if (lane == 0) {
        row_scale[warp] = 1.0f;
      }
      for (int i = lane; i < R; i += 32) {
        const float s = mine[i] * up;
        if constexpr (sizeof(T) == 4) {  // few_mma takes it apart
          hs[warp * h_pitch + i] = s;
        } else {
          const O hi = from_f32<O>(s);
          const float f = to_f32<O>(hi);
          hs[warp * h_pitch + i] = hi;
          hs[(FEW + warp) * h_pitch + i] = from_f32<O>(fabsf(f) == INFINITY ? 0.0f : s - f);
        }
      }
    }
    __syncthreads();
    for (int64_t n = n0; n < n1; n += FEW_N) {
      const int live = (int)(n1 - n < FEW_N ? n1 - n : FEW_N);
      if (n > n0) {
        start_b(n);
        any_b(n, live);
      }
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f}, e[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      int nb = warp * 16, j = 0;
#pragma unroll 1
      while (nb < live) {
#pragma unroll
        for (int u = 0; u < Q; ++u) {
          if (nb < live) {  // the whole warp
            const O* h = hs + row8 * h_pitch + j + quad * 4;
            const uint32_t* hw = reinterpret_cast<const uint32_t*>(h);
            few_mma(T(), d, e, w[u].w, w8[u].w, hw);
            if constexpr (sizeof(T) == 2) few_mma(T(), d, e, w[u].w, w8[u].w, reinterpret_cast<const uint32_t*>(h + FEW * h_pitch));
            else few_mma(T(), d, e, w[u].w + 2, w8[u].w + 2, hw + 2);
            j += 16;
            if (j == R) {
              float* to = outs + quad * 2 * FEW_PITCH + nb + row8;
              to[0] = d[0] + e[0], to[FEW_PITCH] = d[1] + e[1], to[8] = d[2] + e[2], to[FEW_PITCH + 8] = d[3] + e[3];
              d[0] = d[1] = d[2] = d[3] = 0.0f;
              e[0] = e[1] = e[2] = e[3] = 0.0f;
              j = 0;
              nb += kWarps * 16;
            }
          }
        }
        any_b(n, live);
      }
      __syncthreads();
      auto put = [&](int i, int row, int64_t at, T base_value) {
        out[at] = from_f32<T>(fmaf(outs[row * FEW_PITCH + i - row * live], row_scale[row], to_f32<T>(base_value)));
      };
      int i = tid;
      if (n == n0) {
#pragma unroll
        for (int u = 0; u < Q; ++u, i += kThreads) {
          const int row = i / live;
          if (row < t.rows) put(i, row, rows[row] * p.N + n + i - row * live, was[u]);
        }
      }
      for (; i < live * t.rows; i += kThreads) {
        const int row = i / live;
        const int64_t at = rows[row] * p.N + n + i - row * live;
        put(i, row, at, base ? base[at] : from_f32<T>(0.0f));
      }
      __syncthreads();
    }
  } else {  // no adapter
    ptx::cluster_wait();
    for (int i = 0; i < t.rows; ++i)
      for (int64_t n = n0 + tid; n < n1; n += kThreads)
        out[rows[i] * p.N + n] = base ? base[rows[i] * p.N + n] : from_f32<T>(0.0f);
  }
}

// ------------------------------------------------------------------- tiles
// More rows: tiles of 128 rows of one adapter on the tensor cores (tcgen05, fp32
// accumulators), in two launches.  The first computes h = x a^T, a cluster of C CTAs for
// each tile: CTA q takes a run of K, and the cluster's sums are taken in the order of the
// CTAs.  The second adds h b^T to base, a CTA for each 128 x 128 outputs.  Both stream
// (x; base and out), and many small CTAs on an SM hide the memory's latency.  One launch
// for both (h stayed in the cluster) took 66 us for 8192 rows, 8 adapters, r 32, 4096 x
// 4096, bf16, where these take 44.9: 18 for the first (3.7 TB/s of x; all but 10 us of it are
// the launch, the two loads that wait for one another before x can be asked for, and the
// cluster's sums), 27 for the second (5 TB/s of base and out).
//
// A value is a sum of bf16 numbers ("planes"): bf16 1, fp16 2, fp32 3, exactly; an element
// of h is kept as PH of them (2 for the 16-bit types: to 2^-17 of its value; 3 for fp32).
// Beside fp16 b, h is two fp16 numbers instead, its row scaled by a power of two that
// brings its largest value to 2^14 .. 2^15: to 2^-22 of that, whatever its size.
// The planes of the operand that lies along the MMA's N follow one another there, so
// that the tensor core reads a plane of the other operand once for all of them.  fp32: what
// plane c of one and plane d of the other give goes to the sums of order c + d, so that the
// largest are added to once for sixteen terms (the tensor core's sums are truncated; with all
// orders in one sum gradients were off by 1.6e-6, now by 4.4e-7, 2047 rows of 4 adapters,
// r 8, 1000 x 2048).  The orders are added in
// fp32 afterwards, the second product takes them from the smallest on.
constexpr int TILE = 128;            // rows of a tile: the MMA's M
constexpr int KB = 64;               // values of K per stage: 128 bytes of a plane's row
constexpr int XP = TILE * KB * 2;    // bytes of a plane of a stage's x
constexpr int UP_N = 128;            // outputs of one step of the second product
__device__ int g_watchdog_adapters;

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
// Eight values in Q planes; one: as they are.
template <typename T, int Q>
__device__ __forceinline__ void planes_of(const Raw8<T>& raw, uint4 (&out)[Q]) {
  if constexpr (Q == 1) {
    out[0] = raw.w[0];
  } else {
    float v[8];
    raw.widen(v);
    split8<Q>(v, out);
  }
}
// An asynchronous copy of the first n (whole pieces) of eight 16-bit values of a row that is
// aligned to `piece` bytes; zeros for the others.  (`any`: some address as aligned as that; a copy
// asks for it even where it reads nothing.)
template <typename T>
__device__ __forceinline__ void copy_unit(uint8_t* to, const T* from, int n, int piece, const void* any) {
  if (piece == 16) {
    ptx::copy16(to, n > 0 ? from : any, n > 0);
  } else if (piece == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) ptx::copy_small<8>(to + 8 * i, 4 * i < n ? from + 4 * i : any, 4 * i < n);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) ptx::copy_small<4>(to + 4 * i, 2 * i < n ? from + 2 * i : any, 2 * i < n);
  }
}
struct DownProblem {
  const void* x;   // [T, K], rows ld elements apart
  int64_t ld, K;
  const void* w;   // of an adapter [r, K]; turned: [K, r]
  uint16_t* h;     // [T][PH][R], its planes, in adapter order; or null
  uint16_t* h16;   // [T][2][R] of scaled fp16 rows, and what they are to be multiplied by
  float* row_scale;  // [T]; or null
  int turned, x_piece, w_piece;  // alignment of the rows of x and w, up to 16 bytes
};
struct DownArgs {
  DownProblem prob[2];
  const float* scale;
  const int32_t *offsets, *order;
  int64_t T;
  int L, r, R, log_ctas, cols, stages, w_bytes;  // R: r rounded up to 16; w_bytes: of w in a stage
};
struct RingCtl {
  uint64_t empty[4], drain;
  uint32_t tmem_base;
  int abort;
};

// This CTA's sums of h, from tensor memory to its shared memory; the P planes' sums are
// added.  Warps in groups of four: group `part` of `parts` takes every parts-th 16 columns.
template <int P>
__device__ __forceinline__ void own_sums(uint8_t* sm, uint32_t tmem, int R, bool any, int part, int parts) {
  const int row = (threadIdx.x >> 5 & 3) * 32 + (threadIdx.x & 31), pitch = R * 4 + 16;
  for (int j = part * 16; j < R; j += parts * 16) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    if (any) {
#pragma unroll
      for (int c = P - 1; c >= 0; --c) {
        uint32_t s[16];
        ptx::tmem_ld16(tmem + ((uint32_t)(row & ~31) << 16) + c * R + j, s);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(s[i]);
      }
    }
    float4* to = reinterpret_cast<float4*>(sm + row * pitch + j * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}
// h of this CTA's 128 / C rows of the tile: the sums of all CTAs in their order, scaled,
// in planes.  All threads of the block.
template <typename T, int THREADS>
__device__ __forceinline__ void all_sums(uint8_t* sm, const DownArgs& g, const DownProblem& p,
                                         const RowTile& t, int rank) {
  constexpr int PH = Planes<T>::PH;
  __shared__ uint32_t top[sizeof(T) == 2 ? TILE : 1];  // a row's largest magnitude
  const int R = g.R, C = 1 << g.log_ctas, pitch = R * 4 + 16;
  const int mine = TILE >> g.log_ctas, units = mine * (R >> 3);
  const float scale = g.scale ? g.scale[t.l] : 1.0f;
  auto sums = [&](int row, int ju, float (&v)[8]) {
    // (loads of up to eight CTAs in flight together; the sum in their order)
    float4 a[8], b[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < C) {
        const uint32_t at = ptx::cluster_addr(sm + row * pitch + ju * 32, c);
        a[c] = ptx::ld_cluster4(at);
        b[c] = ptx::ld_cluster4(at + 16);
      }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < C) {
        v[0] += a[c].x, v[1] += a[c].y, v[2] += a[c].z, v[3] += a[c].w;
        v[4] += b[c].x, v[5] += b[c].y, v[6] += b[c].z, v[7] += b[c].w;
      }
    // (past r: zeros times x, which may be infinite)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ju * 8 + e < g.r ? v[e] * scale : 0.0f;
  };
  const bool scaled = sizeof(T) == 2 && Planes<T>::FD == 0 && p.h16;
  float held[Planes<T>::FD == 0 ? 8 : 1];  // the first unit's, which is all that most threads have
  if (scaled) {
    for (int i = threadIdx.x; i < mine; i += THREADS) top[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < units; i += THREADS) {
      const int row = i / (R >> 3);
      float v[8];
      sums(rank * mine + row, i % (R >> 3), v);
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        if (Planes<T>::FD == 0 && i == (int)threadIdx.x) held[Planes<T>::FD == 0 ? e : 0] = v[e];
      }
      atomicMax(top + row, m);  // whatever the order
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < units; i += THREADS) {
    const int row = rank * mine + i / (R >> 3), ju = i % (R >> 3);
    if (row >= t.rows) break;
    float v[8];
    if (Planes<T>::FD == 0 && scaled && i == (int)threadIdx.x) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = held[Planes<T>::FD == 0 ? e : 0];
    } else {
      sums(row, ju, v);
    }
    if (scaled) {
      // 2^14 over the largest value's power of two; rows of zeros, and those with
      // infinities or NaN, as they are
      uint32_t e8 = top[row - rank * mine] >> 23;
      e8 = e8 == 255u || top[row - rank * mine] == 0 ? 141u : max(e8, 15u);
      const float up = __uint_as_float((268u - e8) << 23);
      alignas(16) __half hi[8], lo[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hi[e] = __float2half_rn(v[e] * up);
        const float f = __half2float(hi[e]);
        lo[e] = __float2half_rn(fabsf(f) == INFINITY ? 0.0f : v[e] * up - f);
      }
      uint4* to = reinterpret_cast<uint4*>(p.h16 + (int64_t)(t.p0 + row) * 2 * R + ju * 8);
      to[0] = *reinterpret_cast<const uint4*>(hi);
      to[R / 8] = *reinterpret_cast<const uint4*>(lo);
      if (ju == 0) p.row_scale[t.p0 + row] = __uint_as_float((e8 - 14u) << 23);
    }
    if (p.h) {
      uint4 w[PH];
      split8<PH>(v, w);
#pragma unroll
      for (int c = 0; c < PH; ++c)
        *reinterpret_cast<uint4*>(p.h + ((int64_t)(t.p0 + row) * PH + c) * R + ju * 8) = w[c];
    }
  }
}

// A place in a ring and the parity of its current round.
struct Slot {
  int i = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      ++round;
    }
  }
};

// After a wait that gave up: the copies that a warp has under way, one use of its ring's
// barriers after the other, `asked` in all, land before the block ends.
__device__ __forceinline__ void drain_ring(uint64_t* full, int S, int asked) {
  for (int i = asked > S ? asked - S : 0; i < asked; ++i) tc::drain_wait(full + i % S, (i / S) & 1);
}

// Barriers and tensor memory of a block.  The memory is taken before the stream's next
// kernel may start: a block of that one that had it would wait for this kernel's end.
// The first `loaded` barriers take that many arrivals a phase, the others one.
template <typename Ctl>
__device__ __forceinline__ uint32_t set_up(Ctl& ctl, int barriers, uint64_t* bars, int cols, int loaded = 0,
                                           int arrivals = 1) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < barriers; ++i) ptx::mbar_init(bars + i, i < loaded ? arrivals : 1);
    ctl.abort = 0;
    ptx::fence_mbar_init();
  }
  if (threadIdx.x < 32) {
    ptx::tmem_alloc(&ctl.tmem_base, cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  return ctl.tmem_base;
}
// After a wait that gave up, no MMA may run on into freed memory.
template <typename Ctl>
__device__ __forceinline__ void tear_down(Ctl& ctl, uint32_t tmem, int cols) {
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x >= 32) return;
  ptx::tc_fence_after();
  if (ctl.abort) {
    if (ptx::elect_one()) ptx::mma_commit(&ctl.drain);
    __syncwarp();
    tc::drain_wait(&ctl.drain, 0);
  }
  ptx::tmem_dealloc(tmem, cols);
}

// Bytes of w in a stage: n rows of 128 bytes, or units of 64 of them turned.
__host__ __device__ constexpr int down_w_bytes(int n) { return (n + 63) / 64 * (KB * 128); }

template <typename T, int RU>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2)
    k_adapters_down(const __grid_constant__ DownArgs g) {
  using PL = Planes<T>;
  constexpr int P = PL::PD, S = PL::STAGES;
  constexpr bool ASYNC = sizeof(T) == 2;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ RingCtl ctl;
  __shared__ int rows[TILE];
  const DownProblem& p = g.prob[blockIdx.y];
  const int C = 1 << g.log_ctas, rank = (int)ptx::cluster_rank();
  const int tid = threadIdx.x, warp = tid >> 5, R = g.R, r = g.r;
  int* wd = &g_watchdog_adapters;
  if (ptx::smem_addr(sm) & 1023u) {  // (no room to align it: two blocks fill an SM)
    if (tid == 0) atomicCAS(wd, 0, 15);
    return;
  }
  const uint32_t tmem = set_up(ctl, 5, ctl.empty, g.cols);
  ptx::griddep_wait();
  ptx::griddep_launch();
  const RowTile t = find_tile(g.offsets, g.L, false, TILE, blockIdx.x >> g.log_ctas);
  if (t.rows > 0) {  // else the whole cluster has no tile
    if (tid < TILE) rows[tid] = tid < t.rows ? g.order[t.p0 + tid] : -1;
    __syncthreads();
    const int stage_bytes = P * XP + down_w_bytes(P * R);
    // every C-th block of K is this CTA's: what the cluster reads at one time lies together
    const int blocks = (int)((p.K + KB - 1) / KB), b0 = 0, b1 = (blocks - rank + C - 1) >> g.log_ctas;
    auto k_of = [&](int b) { return ((b << g.log_ctas) + rank) * KB; };
    const T* w = static_cast<const T*>(p.w) + (int64_t)t.l * r * p.K;
    const int u = tid & 7;
    const T* xr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = rows[(tid >> 3) + 32 * i];
      xr[i] = row < 0 ? nullptr : static_cast<const T*>(p.x) + row * p.ld + u * 8;
    }
    // x and w of a block go straight to shared memory, or (fp32, and rows that copies of 4
    // bytes cannot reach) through registers.  w lies by its rows j with 64 k each, or
    // turned (r contiguous) by k with the planes' j in units of 64, as the MMA's "MN-major"
    // operand.
    const bool copy_x = ASYNC && p.x_piece >= 4, copy_w = ASYNC && p.w_piece >= 4;
    Raw8<T> held_w[RU], held_x[ASYNC ? 1 : 4];
    const int ru = R >> 3;
    int wj[RU], wk[RU];  // this thread's units of w
#pragma unroll
    for (int i = 0; i < RU; ++i) {
      const int idx = tid + i * kThreads;
      wk[i] = p.turned ? idx / ru : u * 8;
      wj[i] = p.turned ? (idx - wk[i] * ru) * 8 : idx >> 3;
    }
    auto w_unit = [&](int i, int64_t k, int left, int& n) {
      const bool in = wj[i] < r && wk[i] < left;
      n = !in ? 0 : (p.turned ? r - wj[i] : left - wk[i]);
      return p.turned ? w + (k + wk[i]) * r + wj[i] : w + wj[i] * p.K + k + wk[i];
    };
    auto fetch = [&](int b) {
      const int64_t k = k_of(b);
      const int left = (int)(p.K - k < KB ? p.K - k : KB);
      if (!ASYNC) {
#pragma unroll
        for (int i = 0; i < 4; ++i) held_x[ASYNC ? 0 : i].load_by(xr[i] + k, xr[i] ? left - u * 8 : 0, p.x_piece);
      }
      if (!copy_w) {
#pragma unroll
        for (int i = 0; i < RU; ++i) {
          int n;
          const T* from = w_unit(i, k, left, n);
          held_w[i].load_by(from, n, p.w_piece);
        }
      }
    };
    auto put = [&](int b, uint8_t* to) {
      const int64_t k = k_of(b);
      const int left = (int)(p.K - k < KB ? p.K - k : KB);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = (tid >> 3) + 32 * i, at = row * 128 + ((u ^ (row & 7)) << 4);
        if (copy_x) {
          copy_unit(to + at, xr[i] + k, xr[i] ? left - u * 8 : 0, p.x_piece, p.x);
        } else {
          Raw8<T> raw;
          if (ASYNC) raw.load_by(xr[i] + k, xr[i] ? left - u * 8 : 0, 2);
          else raw = held_x[ASYNC ? 0 : i];
          uint4 v[P];
          planes_of<T, P>(raw, v);
#pragma unroll
          for (int c = 0; c < P; ++c) *reinterpret_cast<uint4*>(to + c * XP + at) = v[c];
        }
      }
      uint8_t* wt = to + P * XP;
#pragma unroll
      for (int i = 0; i < RU; ++i) {
        if (wj[i] >= R || wk[i] >= KB) continue;
        uint4 v[P];
        if (!copy_w) planes_of<T, P>(held_w[i], v);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          const int j = c * R + wj[i];
          uint8_t* at = wt + (p.turned ? (j >> 6) * (KB * 128) + wk[i] * 128 + ((((j >> 3) ^ wk[i]) & 7) << 4)
                                       : j * 128 + ((u ^ (j & 7)) << 4));
          if (copy_w) {
            int n;
            const T* from = w_unit(i, k, left, n);
            copy_unit(at, from, n, p.w_piece, w);
          } else {
            *reinterpret_cast<uint4*>(at) = v[c];
          }
        }
      }
    };
    if (b0 < b1) fetch(b0);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (b0 + i < b1) {
        put(b0 + i, sm + i * stage_bytes);
        if (b0 + i + 1 < b1) fetch(b0 + i + 1);
      }
      ptx::copy_commit();
    }
    int slot = 0, use = 0;  // of block b
    for (int b = b0; b < b1; ++b) {
      ptx::copy_wait<S - 2>();
      ptx::fence_proxy_async_smem();
      __syncthreads();
      if (warp == 0) {
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint32_t xa = ptx::smem_addr(sm + slot * stage_bytes), wa = xa + P * XP;
#pragma unroll
          for (int c = 0; c < P; ++c) {
            const int n = (P - c) * R;  // fp32: the smallest products are left out
            for (int n0 = 0; n0 < n; n0 += 256) {
              const int nn = min(256, n - n0);
              const uint32_t id = ptx::idesc_f16(PL::FD, TILE, nn, false, p.turned);
              // (n0 is a multiple of 64; 64 rows of j and 64 k by 64 j both take 8 KB)
#pragma unroll
              for (int ks = 0; ks < KB / 16; ++ks)
                ptx::mma_f16(tmem + c * R + n0, ptx::smem_desc(xa + c * XP + ks * 32, 16, 1024, ptx::kSwizzle128B),
                             ptx::smem_desc(wa + n0 * 128 + ks * (p.turned ? 2048 : 32), KB * 128, 1024,
                                            ptx::kSwizzle128B),
                             id, b > b0 || c > 0 || ks > 0);
            }
          }
          ptx::mma_commit(&ctl.empty[slot]);
        }
        __syncwarp();
      }
      // the next block to load goes where the block before this one was
      if (b + S - 1 < b1) {
        const int last = slot ? slot - 1 : S - 1;
        if (b > b0) tc::warp_wait_bar(&ctl.empty[last], (slot ? use : use - 1) & 1, &ctl.abort, 1, wd);
        put(b + S - 1, sm + last * stage_bytes);
        if (b + S < b1) fetch(b + S);
      }
      ptx::copy_commit();
      if (++slot == S) {
        slot = 0;
        ++use;
      }
    }
    ptx::copy_wait<0>();
    const bool any = b1 > b0;
    if (any) {
      const int done = (b1 - b0 - 1) % S, uses = (b1 - b0 - 1) / S;
      tc::warp_wait_bar(&ctl.empty[done], uses & 1, &ctl.abort, 2, wd);
      ptx::tc_fence_after();
    }
    __syncthreads();
    own_sums<P>(sm, tmem, R, any, warp >> 2, kWarps / 4);
    ptx::cluster_sync();
    all_sums<T, kThreads>(sm, g, p, t, rank);
    ptx::cluster_sync_reads();  // no CTA ends while another reads its sums
  }
  tear_down(ctl, tmem, g.cols);
}

// The same for 16-bit rows that 16-byte copies can reach, without a barrier of the whole block
// in the loop: four warps load 32 rows of x each, by TMA where they lie one after the other
// and by asynchronous copies where they do not (TMA takes ~130 cycles to issue four rows as
// well as a box), one has TMA load w, one issues the MMAs, and nothing passes through registers.
constexpr int DOWN_THREADS = 192, DOWN_STAGES = 8;
struct DownMaps {
  CUtensorMap x[2], w[2];  // of each problem, x by 32 rows
};
// A warp's asynchronous copies to a ring of S stages: each stage's barrier gets the warp's
// arrival when its copies have landed, AHEAD stages later.
struct Landing {
  Slot late;
  int behind = 0;
  const int ahead;
  __device__ explicit Landing(int S) : ahead(S > 3 ? 3 : 2) {}
  __device__ __forceinline__ void arrive(uint64_t* full, int S) {
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(full + late.i);
    late.next(S);
  }
  // after the copies to one more stage
  __device__ __forceinline__ void next(uint64_t* full, int S) {
    ptx::copy_commit();
    if (behind < ahead) {
      ++behind;
      return;
    }
    if (ahead == 3) ptx::copy_wait<3>();
    else ptx::copy_wait<2>();
    arrive(full, S);
  }
  __device__ __forceinline__ void finish(uint64_t* full, int S) {
    ptx::copy_wait<0>();
    for (; behind > 0; --behind) arrive(full, S);
  }
  // a stage that the warp arrives at by itself
  __device__ __forceinline__ void skip(uint64_t* full, int S) {
    if (behind) finish(full, S);
    late.next(S);
  }
};
struct DownCtl {
  uint64_t full[DOWN_STAGES], empty[DOWN_STAGES], accf, drain;
  uint32_t tmem_base;
  int abort;
};

template <typename T>
__global__ void __launch_bounds__(DOWN_THREADS)
    k_adapters_down_tma(const __grid_constant__ DownMaps maps, const __grid_constant__ DownArgs g) {
  using PL = Planes<T>;
  extern __shared__ uint8_t sm_raw[];
  __shared__ DownCtl ctl;
  __shared__ int rows[TILE];
  uint8_t* sm = tc::smem_align1024(sm_raw);
  const DownProblem& p = g.prob[blockIdx.y];
  const int C = 1 << g.log_ctas, rank = (int)ptx::cluster_rank(), S = g.stages;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, R = g.R;
  int* wd = &g_watchdog_adapters;
  const uint32_t tmem = set_up(ctl, 2 * DOWN_STAGES + 2, ctl.full, g.cols, DOWN_STAGES, 5);
  if (tid == 32) {
    ptx::tma_prefetch_desc(&maps.x[blockIdx.y]);
    ptx::tma_prefetch_desc(&maps.w[blockIdx.y]);
  }
  ptx::griddep_wait();
  ptx::griddep_launch();
  const RowTile t = find_tile<DOWN_THREADS>(g.offsets, g.L, false, TILE, blockIdx.x >> g.log_ctas);
  if (t.rows > 0) {  // else the whole cluster has no tile
    // rows of the tile; past its end the last one again (their sums are not used)
    if (tid < TILE) rows[tid] = g.order[t.p0 + min(tid, t.rows - 1)];
    __syncthreads();
    const int wb = p.turned ? down_w_bytes(R) : R * 128, stage_bytes = XP + g.w_bytes;
    // every C-th block of K is this CTA's: what the cluster reads at one time lies together
    const int blocks = (int)((p.K + KB - 1) / KB), b0 = 0, b1 = (blocks - rank + C - 1) >> g.log_ctas;
    auto k_of = [&](int b) { return ((b << g.log_ctas) + rank) * KB; };
    if (warp == 0) {
      const void* mw = &maps.w[blockIdx.y];
      Slot ring;
      int b = b0;
      for (; b < b1; ++b, ring.next(S)) {
        const int slot = ring.i;
        if (ring.round > 0 && !tc::warp_wait_bar(&ctl.empty[slot], (ring.round - 1) & 1, &ctl.abort, 1, wd)) break;
        if (lane == 0) {
          uint8_t* to = sm + slot * stage_bytes + XP;
          ptx::mbar_arrive_expect_tx(&ctl.full[slot], wb);
          if (p.turned) {
            for (int j = 0; j < R; j += 64) ptx::tma_load_3d(to + j * 128, mw, &ctl.full[slot], j, k_of(b), t.l);
          } else {
            ptx::tma_load_3d(to, mw, &ctl.full[slot], k_of(b), 0, t.l);
          }
        }
        __syncwarp();
      }
      if (ctl.abort) drain_ring(ctl.full, S, b - b0);
    } else if (warp == 1) {
      Slot ring;
      for (int b = b0; b < b1; ++b, ring.next(S)) {
        const int slot = ring.i;
        if (!tc::warp_wait_bar(&ctl.full[slot], ring.round & 1, &ctl.abort, 12, wd)) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint32_t xa = ptx::smem_addr(sm + slot * stage_bytes), wa = xa + XP;
          const uint32_t id = ptx::idesc_f16(PL::FD, TILE, R, false, p.turned);
#pragma unroll
          for (int ks = 0; ks < KB / 16; ++ks)
            ptx::mma_f16(tmem, ptx::smem_desc(xa + ks * 32, 16, 1024, ptx::kSwizzle128B),
                         ptx::smem_desc(wa + ks * (p.turned ? 2048 : 32), KB * 128, 1024, ptx::kSwizzle128B),
                         id, b > b0 || ks > 0);
          ptx::mma_commit(&ctl.empty[slot]);
          if (b + 1 == b1) ptx::mma_commit(&ctl.accf);
        }
        __syncwarp();
      }
    } else {
      const int first = (warp - 2) * 32 + (lane >> 3), unit = lane & 7;
      const T* from[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) from[i] = static_cast<const T*>(p.x) + rows[first + i * 4] * p.ld + unit * 8;
      const int some = min(32, t.rows - (warp - 2) * 32);  // of these rows
      const int head = rows[(warp - 2) * 32];
      const bool run = some > 0 && __all_sync(kAll, lane >= some || rows[(warp - 2) * 32 + lane] == head + lane);
      const void* mx = &maps.x[blockIdx.y];
      Slot ring;
      Landing land(S);
      int b = b0;
      for (; b < b1; ++b, ring.next(S)) {
        const int slot = ring.i;
        if (ring.round > 0 && !tc::warp_wait_bar(&ctl.empty[slot], (ring.round - 1) & 1, &ctl.abort, 16, wd)) break;
        const int k = k_of(b);
        uint8_t* to = sm + slot * stage_bytes + first * 128;
        if (run) {  // one box
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(&ctl.full[slot], 4096);
            ptx::tma_load_2d(sm + slot * stage_bytes + (warp - 2) * 4096, mx, &ctl.full[slot], k, head);
          }
          __syncwarp();
          continue;
        }
        const bool in = k + unit * 8 < p.K;  // K is a multiple of 8
        if (some > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = first + i * 4;
            ptx::copy16(to + i * 512 + ((unit ^ (row & 7)) << 4), in ? from[i] + k : from[i] - unit * 8, in);
          }
        }
        land.next(ctl.full, S);
      }
      if (!run) land.finish(ctl.full, S);
      if (b1 > b0) tc::warp_wait_bar(&ctl.accf, 0, &ctl.abort, 2, wd);
      if (ctl.abort && run) drain_ring(ctl.full, S, b - b0);
      ptx::tc_fence_after();
      own_sums<1>(sm, tmem, R, b1 > b0, 0, 1);
    }
    __syncwarp();
    ptx::cluster_sync();
    all_sums<T, DOWN_THREADS>(sm, g, p, t, rank);
    ptx::cluster_sync_reads();  // no CTA ends while another reads its sums
  }
  tear_down(ctl, tmem, g.cols);
}

// Rows of an operand along r in shared memory: r rounded up to 16, 32 or 64 values, swizzled
// accordingly, or two such blocks of 64.
struct Along {
  int bytes, blocks;  // of a row; of 64 values
  __host__ __device__ explicit Along(int R)
      : bytes(R <= 16 ? 32 : (R <= 32 ? 64 : 128)), blocks(R > 64 ? 2 : 1) {}
  __host__ __device__ int plane() const { return TILE * bytes * blocks; }
  // 16-byte unit u of row n
  __device__ __forceinline__ int at(int n, int u) const {
    if (bytes == 32) return n * 32 + ((u ^ (n >> 2 & 1)) << 4);
    if (bytes == 64) return n * 64 + ((u ^ (n >> 1 & 3)) << 4);
    return (u >> 3) * (TILE * 128) + n * 128 + (((u ^ n) & 7) << 4);
  }
  // the matrix descriptor of sixteen values from 16 ks on
  __device__ __forceinline__ uint64_t desc(uint32_t base, int ks) const {
    const int in = ks * 32, block = in / bytes;
    return ptx::smem_desc(base + block * (TILE * bytes) + in - block * bytes, 16, 8 * bytes,
                          bytes == 32 ? 6 : (bytes == 64 ? ptx::kSwizzle64B : ptx::kSwizzle128B));
  }
};

struct UpArgs {
  const float* row_scale;  // of scaled h, else null
  const void* w;      // of an adapter [N, r]; turned: [r, N]
  const void* base;
  void* out;
  const int32_t *offsets, *order;
  int64_t T, N;
  int L, r, R, steps, turned, vec;  // vec: w by TMA
  int w_piece, piece;  // alignment of the rows of w, and of base and out, up to 16 bytes
  int group;                              // items that a block takes at once
  int jump, jump_tiles, jump_steps;       // from the last of them to its next: items, the same as tiles and steps
  int slots, h_slots, b_slots, w_bytes, h_bytes;  // of the rings of w, h and base; bytes of one
  int buckets;                                    // where the table of the buckets is
};
struct UpMaps {
  CUtensorMap base, out;  // by 32 rows, 128 bytes of columns
  CUtensorMap h, w;             // a plane of 128 rows; 128 outputs (turned: 64) and r
};
constexpr int UP_EPI = 8;  // warps; beside them loaders and one for the MMAs
template <typename T>
constexpr int UP_LOAD = sizeof(T) == 2 ? 1 : 4;
template <typename T>
constexpr int UP_THREADS = (UP_EPI + UP_LOAD<T> + 1) * 32;
constexpr int UP_SLOTS = 4, BASE_SLOTS = 4;
constexpr int kAdapters = 1024;  // the most that a layout has
struct UpCtl {
  uint64_t wfull[UP_SLOTS], wempty[UP_SLOTS], hfull[2], hempty[2], accf[2], acce[2], drain;
  uint64_t bfull[UP_EPI][BASE_SLOTS];
  uint32_t tmem_base;
  int abort;
  int sums[16];
};

// A block's items, each 128 outputs (`step`) of a tile's rows: runs of `group` items, the
// blocks' runs interleaved, so that what all blocks read and write at one time lies
// together.  Walked by counting, in 32 bits (T N < 2^40, with sixteen rows a tile on average at
// least, makes fewer than 2^31 items), with the divisions on the host: a 64-bit one takes half
// a microsecond here.
struct Walk {
  int tile, step, in;
  uint32_t at, items;
  __device__ __forceinline__ Walk(const UpArgs& g, uint32_t items_) : in(0), at(blockIdx.x * g.group), items(items_) {
    tile = (int)(at / (uint32_t)g.steps);
    step = (int)at - tile * g.steps;
  }
  __device__ __forceinline__ bool more() const { return at < items; }
  __device__ __forceinline__ void next(const UpArgs& g) {
    const bool jump = ++in == g.group;
    if (jump) in = 0;
    at += jump ? g.jump : 1;
    tile += jump ? g.jump_tiles : 0;
    step += jump ? g.jump_steps : 1;
    if (step >= g.steps) {
      step -= g.steps;
      ++tile;
    }
  }
};

// Tiles before each bucket, and its first row: in shared memory behind the rings.
struct Buckets {
  int *before, *first;
  __device__ __forceinline__ Buckets(uint8_t* at, int L) : before(reinterpret_cast<int*>(at)), first(before + L + 2) {}
};
constexpr int buckets_bytes(int L) { return (L + 2) * 8; }
// Tile t of the counted buckets.
__device__ __forceinline__ RowTile tile_of(const Buckets& in, int B, int t) {
  int low = 0, high = B;  // before[low] <= t < before[high]
  while (high - low > 1) {
    const int mid = (low + high) >> 1;
    if (in.before[mid] <= t) low = mid;
    else high = mid;
  }
  const int p0 = in.first[low] + (t - in.before[low]) * TILE;
  return {low, p0, min(TILE, in.first[low + 1] - p0)};
}

// Two values of base and of the product (fp16: times its row's scale).
__device__ __forceinline__ uint32_t add_pair(__nv_bfloat16, uint32_t base, float a, float b, float) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(base << 16) + a,
                                                 __uint_as_float(base & 0xFFFF0000u) + b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t add_pair(__half, uint32_t base, float a, float b, float scale) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&base));
  const __half2 v = __floats2half2_rn(fmaf(a, scale, f.x), fmaf(b, scale, f.y));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Bytes of a warp's part of base: 32 rows of 64 columns, in boxes of 128 bytes a row.  Without
// TMA a row of 16-bit values may start in the middle of a word: one more word for each.
template <typename T, bool TMA>
constexpr int UP_PART = 32 * 64 * (int)sizeof(T) + (!TMA && sizeof(T) == 2 ? 128 : 0);
// Columns that a warp stages at once where there is no room for that.
constexpr int STAGED_COLS = 16;

// Persistent blocks, each with an equal run of the (tile, 128 outputs) items:
//   warps 0-7   epilogue: a warp has 32 rows and half of an item's columns: it asks for
//               its part of base some items ahead (a TMA box, or asynchronous copies where the
//               rows do not lie one after the other), adds the product from tensor memory in
//               place, rounds once, and has TMA store it (row by row itself where the box
//               would reach other rows).  Form TMA: rows aligned to 16 bytes; the other
//               copies by 8 or 4 bytes (16-bit rows at odd elements: by the words that hold
//               them), or, with no room for parts of base (fp32, ranks above 64), adds column by
//               column through shared memory
//   then        one warp (fp32: four, which cut w into its planes) that loads h of a tile
//               and w of an item, and one for tensor memory and the MMAs (two accumulators
//               of 128 columns)
template <typename T, bool TMA>
__global__ void __launch_bounds__(UP_THREADS<T>, sizeof(T) == 2 ? 2 : 1)
    k_adapters_up(const __grid_constant__ UpMaps maps, const __grid_constant__ UpArgs g) {
  using PL = Planes<T>;
  constexpr int P = PL::PD, PH = PL::PH, LOAD = UP_LOAD<T>, THREADS = UP_THREADS<T>;
  extern __shared__ uint8_t sm_raw[];
  __shared__ UpCtl ctl;
  uint8_t* sm = tc::smem_align1024(sm_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, R = g.R, r = g.r;
  int* wd = &g_watchdog_adapters;
  if (tid == 0) {
    for (int i = 0; i < UP_SLOTS; ++i) {
      ptx::mbar_init(&ctl.wfull[i], g.vec ? 1 : LOAD * 32);
      ptx::mbar_init(&ctl.wempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ctl.hfull[i], 1);
      ptx::mbar_init(&ctl.hempty[i], 1);
      ptx::mbar_init(&ctl.accf[i], 1);
      ptx::mbar_init(&ctl.acce[i], UP_EPI * 32);
    }
    ptx::mbar_init(&ctl.drain, 1);
    for (int i = 0; i < UP_EPI * BASE_SLOTS; ++i) ptx::mbar_init(&ctl.bfull[0][0] + i, 1);
    ctl.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == UP_EPI + LOAD) {
    ptx::tmem_alloc(&ctl.tmem_base, 2 * UP_N);
    ptx::tmem_relinquish();
  }
  if (tid == 32) {
    ptx::tma_prefetch_desc(&maps.h);
    if (g.vec) ptx::tma_prefetch_desc(&maps.w);
    if (TMA) {
      if (g.base) ptx::tma_prefetch_desc(&maps.base);
      ptx::tma_prefetch_desc(&maps.out);
    }
  }
  // The call's inputs are there already (the first launch has waited for them); h is not.  Every
  // role waits for the launch before this one by itself: what it then waits for with a limit is
  // this block's work alone, however long that launch still ran.
  const T* base = static_cast<const T*>(g.base);
  T* out = static_cast<T*>(g.out);
  const int B = g.L + (g.base != g.out ? 1 : 0);  // rows without an adapter: copied, or left
  const Buckets buckets(sm + g.buckets, g.L);
  count_tiles<THREADS>(g.offsets, B, TILE, buckets.first, buckets.before, ctl.sums);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  ptx::griddep_launch();
  const Walk walk(g, (uint32_t)buckets.before[B] * (uint32_t)g.steps);
  constexpr int SB = UP_PART<T, TMA>;
  uint8_t* ws = sm + UP_EPI * g.b_slots * SB;
  uint8_t* hs = ws + g.slots * g.w_bytes;
  const Along along(R);
  const int plane = along.plane();

  if (warp >= UP_EPI && warp < UP_EPI + LOAD) {
    // ------------------------------------------------------------- loaders
    ptx::griddep_wait();
    const int lt = tid - UP_EPI * 32, ru = R >> 3;
    constexpr int LT = LOAD * 32;
    const int row_by = LT / ru, ju_by = LT - row_by * ru;  // from one of a thread's units to its next
    int last = -1;
    Slot hslot, wslot;
    RowTile t = {0, 0, 0};
    for (Walk item = walk; item.more(); item.next(g)) {
      const int64_t n0 = (int64_t)item.step * UP_N;
      const bool other = item.tile != last;
      if (other) t = tile_of(buckets, B, item.tile);
      last = item.tile;
      if (t.l == g.L) continue;
      if (other) {
        const int hb = hslot.i;
        if (hslot.round > 0 && !tc::warp_wait_bar(&ctl.hempty[hb], (hslot.round - 1) & 1, &ctl.abort, 6, wd)) break;
        if (lt == 0) {
          uint8_t* to = hs + hb * g.h_bytes;
          ptx::mbar_arrive_expect_tx(&ctl.hfull[hb], PH * plane);
#pragma unroll
          for (int c = 0; c < PH; ++c)
            for (int k = 0; k < along.blocks; ++k)
              ptx::tma_load_3d(to + c * plane + k * (TILE * 128), &maps.h, &ctl.hfull[hb], k * 64, c, t.p0);
        }
        hslot.next(g.h_slots);
      }
      const int slot = wslot.i;
      if (wslot.round > 0 && !tc::warp_wait_bar(&ctl.wempty[slot], (wslot.round - 1) & 1, &ctl.abort, 7, wd)) break;
      uint8_t* to = ws + slot * g.w_bytes;
      if (P == 1 && g.vec) {
        if (lt == 0) {
          uint64_t* bar = &ctl.wfull[slot];
          ptx::mbar_arrive_expect_tx(bar, g.turned ? R * 256 : plane);
          if (g.turned) {
            const int boxes = 2;
            for (int k = 0; k < boxes; ++k) ptx::tma_load_3d(to + k * (R * 128), &maps.w, bar, (int)n0 + k * 64, 0, t.l);
          } else {
            for (int k = 0; k < along.blocks; ++k)
              ptx::tma_load_3d(to + k * (TILE * 128), &maps.w, bar, k * 64, (int)n0, t.l);
          }
        }
        __syncwarp();
      } else {
        const T* w = static_cast<const T*>(g.w) + (int64_t)t.l * r * g.N;
        const int left = (int)(g.N - n0 < UP_N ? g.N - n0 : UP_N);
        const int un0 = lt / ru, uj0 = lt - un0 * ru;
        int un = un0, uj = uj0;
        // unit i of this thread: where it is, how many of its values, where it goes
        auto unit = [&](int i, const T*& from, int& have, uint8_t*& at) {
          if (uj >= ru) {
            uj -= ru;
            ++un;
          }
          if (g.turned) {  // eight n of one j; n lies along the operand's N
            const int nu = i & 15, j = i >> 4;
            from = w + j * g.N + n0 + nu * 8;
            have = j < r ? left - nu * 8 : 0;
            at = to + (nu >> 3) * (R * 128) + j * 128 + (((nu ^ j) & 7) << 4);
          } else {  // eight j of one n
            from = w + (n0 + un) * r + uj * 8;
            have = un < left ? r - uj * 8 : 0;
            at = to + along.at(un, uj);
          }
          un += row_by;
          uj += ju_by;
        };
        const T* from;
        int have;
        uint8_t* at;
        if (P == 1 && g.w_piece >= 4) {  // all of it under way at once
          for (int i = lt; i < TILE / 8 * R; i += LT) {
            unit(i, from, have, at);
            copy_unit(at, from, have, g.w_piece, w);
          }
          ptx::copy_commit();
          ptx::copy_wait<0>();
        } else {
          const int pitch = g.turned ? R * 256 : plane;
#pragma unroll 4
          for (int i = lt; i < TILE / 8 * R; i += LT) {
            unit(i, from, have, at);
            Raw8<T> raw;
            raw.load(from, have, g.w_piece == 16);
            uint4 v[P];
            planes_of<T, P>(raw, v);
#pragma unroll
            for (int c = 0; c < P; ++c) *reinterpret_cast<uint4*>(at + c * pitch) = v[c];
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&ctl.wfull[slot]);
      }
      wslot.next(g.slots);
    }
    if (ctl.abort && lt == 0) {  // the copies under way land before the block ends
      auto drain = [](uint64_t* bars, const Slot& next, int n) {
        for (int i = 0; i < n; ++i)
          if (i < next.i || next.round > 0) tc::drain_wait(bars + i, (i < next.i ? next.round : next.round - 1) & 1);
      };
      drain(ctl.hfull, hslot, g.h_slots);
      if (g.vec) drain(ctl.wfull, wslot, g.slots);
    }
  } else if (warp == UP_EPI + LOAD) {
    // ---------------------------------------------------------------- MMAs
    ptx::griddep_wait();
    int last = -1, hb = 0;
    Slot hslot, wslot, aslot;
    bool product = false;
    const uint32_t id = ptx::idesc_f16(PL::FD, TILE, UP_N, false, g.turned);
    for (Walk item = walk; item.more();) {
      const bool other = item.tile != last;
      if (other) product = tile_of(buckets, B, item.tile).l < g.L;
      last = item.tile;
      item.next(g);
      if (!product) continue;
      if (other) {
        hb = hslot.i;
        if (!tc::warp_wait_bar(&ctl.hfull[hb], hslot.round & 1, &ctl.abort, 8, wd)) break;
        hslot.next(g.h_slots);
      }
      const int slot = wslot.i, buf = aslot.i;
      if (!tc::warp_wait_bar(&ctl.wfull[slot], wslot.round & 1, &ctl.abort, 9, wd)) break;
      if (aslot.round > 0 && !tc::warp_wait_bar(&ctl.acce[buf], (aslot.round - 1) & 1, &ctl.abort, 10, wd)) break;
      wslot.next(g.slots);
      aslot.next(2);
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        const uint32_t ha = ptx::smem_addr(hs + hb * g.h_bytes), wa = ptx::smem_addr(ws + slot * g.w_bytes);
        uint32_t more = 0;
#pragma unroll
        for (int order = P == 3 ? 2 : PH - 1; order >= 0; --order)
#pragma unroll
          for (int d = 0; d < P; ++d) {
            const int c = order - d;
            if (c < 0 || c >= PH) continue;
            for (int ks = 0; ks < R / 16; ++ks) {
              const uint64_t wdesc =
                  g.turned ? ptx::smem_desc(wa + d * (R * 256) + ks * 2048, R * 128, 1024, ptx::kSwizzle128B)
                           : along.desc(wa + d * plane, ks);
              ptx::mma_f16(tmem + buf * UP_N, along.desc(ha + c * plane, ks), wdesc, id, more);
              more = 1;
            }
          }
        ptx::mma_commit(&ctl.wempty[slot]);
        ptx::mma_commit(&ctl.accf[buf]);
        if (!item.more() || item.tile != last) ptx::mma_commit(&ctl.hempty[hb]);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q4 = warp & 3, half = warp >> 2, NS = g.b_slots;
    uint8_t* ring = sm + warp * NS * SB;
    constexpr int BOX = 128 / (int)sizeof(T);  // columns of a box
    // An item's tile, the row of this lane in it, its columns.  For loads and for stores:
    // the first run ahead.
    struct Place {
      int tile = -1, row = 0, rows = 0, l = 0, place = 0;
      bool run = false;  // the warp's rows lie one after the other
      int64_t col = 0;
    };
    auto place = [&](Place& q, const Walk& item) {
      q.col = (int64_t)item.step * UP_N + half * 64;
      if (item.tile == q.tile) return;
      q.tile = item.tile;
      const RowTile t = tile_of(buckets, B, item.tile);
      q.l = t.l;
      q.rows = t.rows - q4 * 32 < 0 ? 0 : min(32, t.rows - q4 * 32);  // of this warp
      if (q.rows == 0) return;
      q.place = t.p0 + q4 * 32 + min(lane, q.rows - 1);
      q.row = __ldg(g.order + q.place);
      const int first = __shfl_sync(kAll, q.row, 0);
      q.run = TMA && __all_sync(kAll, lane >= q.rows || q.row == first + lane);
    };
    // without TMA: lanes of a row of 128 bytes, by 8 or 4 bytes
    const int piece = g.piece, lanes_log = piece == 8 ? 4 : 5, rows_by = 32 >> lanes_log;
    const int sub_row = lane >> lanes_log, sub = (lane - (sub_row << lanes_log)) * (piece == 8 ? 8 : 4);
    // does a row's part start in the middle of a word
    auto odd = [&](int64_t row, int64_t col) {
      return sizeof(T) == 2 && !TMA ? (int)((reinterpret_cast<uintptr_t>(base) >> 1) + row * g.N + col) & 1 : 0;
    };
    Place ahead, now;
    Walk item = walk, next = walk;
    Slot nslot;
    auto load = [&] {  // base of the next item to its place in the ring
      if (!next.more()) {
        ptx::copy_commit();
        return;
      }
      place(ahead, next);
      next.next(g);
      const int slot = nslot.i;
      nslot.next(NS);
      if (base && ahead.rows > 0 && ahead.col < g.N) {
        uint8_t* to = ring + slot * SB;
        const int boxes = ahead.col + BOX < g.N ? 64 / BOX : 1;
        if (ahead.run) {
          uint64_t* bar = &ctl.bfull[warp][slot];
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(bar, boxes * 4096);
            for (int b = 0; b < boxes; ++b)
              ptx::tma_load_2d(to + b * 4096, &maps.base, bar, (int)ahead.col + b * BOX, ahead.row);
          }
        } else if (!TMA) {  // one or two rows at a time
          // (A word that holds an element of base is within its allocation; what else it holds
          // is dropped.)
          for (int b = 0; b < boxes; ++b) {
            const int64_t c = ahead.col + b * BOX + sub / (int)sizeof(T);
#pragma unroll 4
            for (int i = 0; i < 32; i += rows_by) {
              const int at = i + sub_row;
              const int64_t row = __shfl_sync(kAll, ahead.row, at), first = c - odd(row, ahead.col);
              uint8_t* place = to + b * 4096 + at * 128 + ((((sub >> 4) ^ at) & 7) << 4) + (sub & 15);
              const bool in = first < g.N;
              const T* from = base + row * g.N + first;
              if (piece == 8) ptx::copy_small<8>(place, in ? from : base, in);
              else ptx::copy_small<4>(place, in ? static_cast<const void*>(from) : g.order, in);
            }
          }
          if (sizeof(T) == 2 && odd(ahead.row, ahead.col)) {  // the last element's word
            const bool in = ahead.col + 63 < g.N;
            ptx::copy_small<4>(to + 4096 + lane * 4, in ? static_cast<const void*>(base + (int64_t)ahead.row * g.N + ahead.col + 63) : g.order, in);
          }
        } else {  // four rows at a time, eight lanes each
          const int unit = lane & 7;
          for (int b = 0; b < boxes; ++b) {
            const int64_t c = ahead.col + b * BOX + unit * (16 / (int)sizeof(T));
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const int at = i + (lane >> 3);
              const int64_t row = __shfl_sync(kAll, ahead.row, at);
              ptx::copy16(to + b * 4096 + at * 128 + ((unit ^ (at & 7)) << 4), c < g.N ? base + row * g.N + c : base, c < g.N);
            }
          }
        }
      }
      ptx::copy_commit();  // (of every item, so that they can be counted)
    };
    const bool wide = TMA || sizeof(T) == 2 || NS > 0;
    float scale = 1.0f;  // of this lane's row of h; there once an accumulator is
    int scale_of = -1, n = 0;
    auto scale_it = [&] {
      if (PL::FD == 1 || now.tile == scale_of) return;
      scale_of = now.tile;
      scale = now.rows > 0 ? __ldcg(g.row_scale + now.place) : 1.0f;
    };
    uint32_t phases = 0;  // of the ring's barriers
    if (wide)
      for (int i = 0; i < NS - 1; ++i) load();
    Slot slot_of;
    for (; item.more(); item.next(g), slot_of.next(NS)) {
      place(now, item);
      const bool product = now.l < g.L, live = now.rows > 0 && now.col < g.N;
      const uint32_t acc = tmem + ((uint32_t)(q4 * 32) << 16) + (n & 1) * UP_N + half * 64;
      if (wide) {
        const int slot = slot_of.i;
        uint8_t* mine = ring + slot * SB;
        if (base && live) {
          if (now.run) {
            if (!tc::warp_wait_bar(&ctl.bfull[warp][slot], phases >> slot & 1, &ctl.abort, 13, wd)) break;
            phases ^= 1u << slot;
          } else if (NS == 4) {  // NS - 2 items have been asked for since
            ptx::copy_wait<2>();
          } else if (NS == 3) {
            ptx::copy_wait<1>();
          } else {
            ptx::copy_wait<0>();
          }
          __syncwarp();
        }
        if (product) {
          if (n == 0) ptx::griddep_wait();
          if (!tc::warp_wait_bar(&ctl.accf[n & 1], (n >> 1) & 1, &ctl.abort, 11, wd)) break;
          ptx::tc_fence_after();
          scale_it();
        }
        // the item before this one has been stored: its place takes the next one to load
        if (lane == 0) ptx::bulk_wait_read0();
        __syncwarp();
        load();
        const int shift = base ? odd(now.row, now.col) * 16 : 0;
        if (live && (product || !base || (!TMA && sizeof(T) == 2))) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint32_t s[32];
            if (product) {
              ptx::tmem_ld32(acc + b * 32, s);
              ptx::tmem_ld_wait();
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) s[e] = 0;
            }
            constexpr int V = 16 / (int)sizeof(T);  // values of 16 bytes
#pragma unroll
            for (int i = 0; i < 32 / V; ++i) {
              const int unit = (b * 32 / V + i) & 7, box = (b * 32 / V + i) >> 3;
              uint4* at = reinterpret_cast<uint4*>(mine + box * 4096 + lane * 128 + ((unit ^ (lane & 7)) << 4));
              uint4 h = base ? *at : make_uint4(0, 0, 0, 0);
              uint32_t* hw = reinterpret_cast<uint32_t*>(&h);
              if (!TMA && sizeof(T) == 2) {
                const uint8_t* next = i + b * (32 / V) == 7 ? mine + 4096 + lane * 4 : mine + lane * 128 + (((unit + 1) ^ (lane & 7)) << 4);
                const uint32_t after = base ? *reinterpret_cast<const uint32_t*>(next) : 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) hw[e] = __funnelshift_r(hw[e], e < 3 ? hw[e + 1] : after, shift);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if constexpr (sizeof(T) == 2)
                  hw[e] = add_pair(T(), hw[e], __uint_as_float(s[i * 8 + 2 * e]), __uint_as_float(s[i * 8 + 2 * e + 1]),
                                   scale);
                else
                  hw[e] = __float_as_uint(__uint_as_float(hw[e]) + __uint_as_float(s[i * 4 + e]));
              }
              *at = h;
            }
          }
        }
        if (product) {
          ptx::tc_fence_before();
          ptx::mbar_arrive(&ctl.acce[n & 1]);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (live) {
          if (now.run && now.rows == 32) {
            if (lane == 0)
              for (int b = 0; b < 64 / BOX && now.col + b * BOX < g.N; ++b)
                ptx::tma_store_2d(&maps.out, mine + b * 4096, (int)now.col + b * BOX, now.row);
          } else if (!TMA) {
            const int64_t width = g.N - now.col < 64 ? g.N - now.col : 64;
#pragma unroll
            for (int b = 0; b < 64 / BOX; ++b) {
              const int c = b * BOX + sub / (int)sizeof(T);
#pragma unroll 4
              for (int i = 0; i < 32; i += rows_by) {
                const int at = i + sub_row;
                const int64_t to_row = __shfl_sync(kAll, now.row, at);
                const uint8_t* from = mine + b * 4096 + at * 128 + ((((sub >> 4) ^ at) & 7) << 4) + (sub & 15);
                T* to = out + to_row * g.N + now.col + c;
                if (at < now.rows && c < width) {
                  if (sizeof(T) == 2 && piece == 2) {
                    to[0] = reinterpret_cast<const T*>(from)[0];
                    if (c + 1 < width) to[1] = reinterpret_cast<const T*>(from)[1];
                  } else if (piece == 8) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(from);
                  else *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(from);
                }
              }
            }
            __syncwarp();
          } else {  // four rows at a time, eight lanes each
            const int64_t width = g.N - now.col < 64 ? g.N - now.col : 64;
#pragma unroll
            for (int b = 0; b < 64 / BOX; ++b)
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const int from = i + (lane >> 3), unit = lane & 7, c = b * BOX + unit * (16 / (int)sizeof(T));
                const int64_t to_row = __shfl_sync(kAll, now.row, from);
                if (from < now.rows && c < width)
                  *reinterpret_cast<uint4*>(out + to_row * g.N + now.col + c) = *reinterpret_cast<const uint4*>(
                      mine + b * 4096 + from * 128 + ((unit ^ (from & 7)) << 4));
              }
            ptx::fence_proxy_async_smem();  // read before TMA writes there again
            __syncwarp();
          }
        }
        if (lane == 0) ptx::bulk_commit();
      } else if constexpr (!TMA && sizeof(T) == 4) {
        if (product) {
          if (n == 0) ptx::griddep_wait();
          if (!tc::warp_wait_bar(&ctl.accf[n & 1], (n >> 1) & 1, &ctl.abort, 11, wd)) break;
          ptx::tc_fence_after();
          scale_it();
        }
        constexpr int SC = STAGED_COLS, ROWS = 32 / SC;  // columns, and rows at once
        float* mine = reinterpret_cast<float*>(hs + g.h_slots * g.h_bytes) + warp * 32 * (SC + 1);
        const int to_row = lane < now.rows ? now.row : -1;
#pragma unroll 1
        for (int b = 0; b < 64 / SC; ++b) {
          if (product) {
            uint32_t s[SC];
            ptx::tmem_ld16(acc + b * SC, s);
            ptx::tmem_ld_wait();
            if (b + 1 == 64 / SC) {
              ptx::tc_fence_before();
              ptx::mbar_arrive(&ctl.acce[n & 1]);
            }
#pragma unroll
            for (int e = 0; e < SC; ++e) mine[lane * (SC + 1) + e] = __uint_as_float(s[e]) * scale;
            __syncwarp();
          }
          const int64_t c = now.col + b * SC + lane % SC;  // a lane has a column of its rows
          const bool in = c < g.N;
#pragma unroll 1
          for (int i0 = lane / SC; i0 < 32; i0 += 8 * ROWS) {
            int64_t at[8];
            T v[8];  // (out may be base: all eight are read before one is written)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int64_t to = __shfl_sync(kAll, to_row, i0 + k * ROWS);
              at[k] = in && to >= 0 ? to * g.N + c : -1;
              v[k] = base && at[k] >= 0 ? base[at[k]] : from_f32<T>(0.0f);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (at[k] < 0) continue;
              out[at[k]] = product ? from_f32<T>(to_f32<T>(v[k]) + mine[(i0 + k * ROWS) * (SC + 1) + lane % SC]) : v[k];
            }
          }
          __syncwarp();
        }
      }
      if (product) ++n;
    }
    if (wide) {
      if (ctl.abort) {  // the copies under way land before the block ends
        for (; item.at < next.at && base; item.next(g), slot_of.next(NS)) {
          place(now, item);
          if (now.rows == 0 || now.col >= g.N || !now.run) continue;
          tc::drain_wait(&ctl.bfull[warp][slot_of.i], phases >> slot_of.i & 1);
        }
      }
      ptx::copy_wait<0>();
      if (lane == 0) ptx::bulk_wait_all();
      __syncwarp();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp != UP_EPI + LOAD) return;
  ptx::tc_fence_after();
  if (ctl.abort) {  // after a wait that gave up, no MMA may run on into freed memory
    if (ptx::elect_one()) ptx::mma_commit(&ctl.drain);
    __syncwarp();
    tc::drain_wait(&ctl.drain, 0);
  }
  ptx::tmem_dealloc(tmem, 2 * UP_N);
}

// ------------------------------------------------------- weights' gradients
// grad_a[l][j][k] = sum over l's rows of g[p][j] x[row][k], and grad_b[l][n][j] with h and
// grad.  A cluster has one adapter and 128 columns of x (or grad): they are the MMA's M,
// the r columns of g its N, the rows its K.  CTA q of C takes a run of the rows; the
// cluster's sums are taken in the order of the CTAs.  Tiles of x and of g's planes are
// loaded by rows, so their columns lie along the operands' M and N ("MN-major").  fp32 and
// fp16, whose planes pass through registers, and bf16 rows not aligned to 16 bytes: fp32
// 2047 rows of 4 adapters, r 8, 1000 x 2048, all gradients 37.7 us.
constexpr int GRAD_ROWS = 64;  // rows per stage
constexpr int GRAD_COLS = 128;

struct GradProblem {
  const void* x;      // [T, cols]
  int64_t cols;
  const uint16_t* h;  // [T][PH][R]
  void* out;          // of an adapter [r, cols]; turned: [cols, r]
  int turned, piece;  // alignment of x's rows, up to 16 bytes
};
struct GradArgs {
  GradProblem prob[2];
  const int32_t *offsets, *order;
  int64_t T;
  int L, r, R, log_ctas, cols, stages, blocks;  // blocks of 16 of R
};
// A CTA's sums, from tensor memory to its shared memory: a column's r sums after another's,
// one word apart.
template <int PH>
__device__ __forceinline__ void grad_sums(uint8_t* sm, uint32_t tmem, int R, bool any, int part, int parts) {
  float* to = reinterpret_cast<float*>(sm);
  const int col = (threadIdx.x >> 5 & 3) * 32 + (threadIdx.x & 31);
  for (int j = part * 16; j < R; j += parts * 16) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    if (any) {
#pragma unroll
      for (int c = PH - 1; c >= 0; --c) {
        uint32_t w[16];
        ptx::tmem_ld16(tmem + ((uint32_t)(col & ~31) << 16) + c * R + j, w);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(w[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) to[col * (R + 1) + j + i] = v[i];
  }
}
// This CTA's share of the gradient: the sums of all CTAs in their order.
template <typename T, int THREADS>
__device__ __forceinline__ void grad_out(uint8_t* sm, const GradArgs& g, const GradProblem& p, int l,
                                         int rank, int64_t col0) {
  const int C = 1 << g.log_ctas, r = g.r, pitch = g.R + 1;
  const int left = (int)(p.cols - col0 < GRAD_COLS ? p.cols - col0 : GRAD_COLS);
  const int n = left * r, share = (n + C - 1) >> g.log_ctas;
  const int e0 = rank * share, e1 = min(e0 + share, n);
  const float* part = reinterpret_cast<const float*>(sm);
  T* out = static_cast<T*>(p.out) + (int64_t)l * r * p.cols;
  for (int e = e0 + threadIdx.x; e < e1; e += THREADS) {
    const int col = p.turned ? e / r : e % left, j = p.turned ? e - col * r : e / left;
    float sum = 0.0f;
    for (int c = 0; c < C; ++c)
      sum += __uint_as_float(ptx::ld_cluster(ptx::cluster_addr(part + col * pitch + j, c)));
    out[p.turned ? (col0 + col) * r + j : (int64_t)j * p.cols + col0 + col] = from_f32<T>(sum);
  }
}

// Bytes of h's n columns in a stage: GRAD_ROWS rows in units of 64 columns.
__host__ __device__ constexpr int grad_h_bytes(int n) { return (n + 63) / 64 * (GRAD_ROWS * 128); }

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1)
    k_adapters_grad(const __grid_constant__ GradArgs g) {
  using PL = Planes<T>;
  constexpr int P = PL::P, PH = PL::PH, S = PL::GRAD_STAGES;
  constexpr bool HELD = P > 1;  // x goes through registers, a block ahead
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ RingCtl ctl;
  const GradProblem& p = g.prob[blockIdx.z];
  const int C = 1 << g.log_ctas, rank = (int)ptx::cluster_rank();
  const int tid = threadIdx.x, warp = tid >> 5, R = g.R;
  const int64_t col0 = (int64_t)(blockIdx.x >> g.log_ctas) * GRAD_COLS;
  const int l = blockIdx.y;
  int* wd = &g_watchdog_adapters;
  if (col0 >= p.cols) return;  // the whole cluster (the problems may have different numbers of columns)
  if (ptx::smem_addr(sm) & 1023u) {  // (no room to align it: two blocks fill an SM)
    if (tid == 0) atomicCAS(wd, 0, 15);
    return;
  }
  const uint32_t tmem = set_up(ctl, 5, ctl.empty, g.cols);
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int first = __ldg(g.offsets + l), rows = __ldg(g.offsets + l + 1) - first;
  const int blocks = (rows + GRAD_ROWS - 1) / GRAD_ROWS, per = (blocks + C - 1) >> g.log_ctas;
  const int b0 = min(rank * per, blocks), b1 = min(b0 + per, blocks);
  constexpr int XG = GRAD_ROWS * GRAD_COLS * 2;  // bytes of a plane of a stage's x
  const int stage_bytes = P * XG + grad_h_bytes(PH * R);
  const int left = (int)(p.cols - col0 < GRAD_COLS ? p.cols - col0 : GRAD_COLS);
  const int u = tid & 15, xrow = tid >> 4, ru = R >> 3;
  const T* x = static_cast<const T*>(p.x) + col0 + u * 8;
  const bool copy = !HELD && p.piece >= 4;
  int next[4];  // rows of the next block whose x is asked for
  auto rows_of = [&](int b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int in = b * GRAD_ROWS + xrow + 16 * i;
      next[i] = b < b1 && in < rows ? __ldg(g.order + first + in) : -1;
    }
  };
  Raw8<T> held[HELD ? 4 : 1];
  auto fetch = [&](int b) {  // block b's x, then the rows of the next one
    if (HELD) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        held[HELD ? i : 0].load_by(x + next[i] * p.cols, next[i] >= 0 ? left - u * 8 : 0, p.piece);
      rows_of(b + 1);
    }
  };
  auto put = [&](int b, uint8_t* to) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = xrow + 16 * i;
      uint8_t* at = to + (u >> 3) * (GRAD_ROWS * 128) + row * 128 + (((u & 7) ^ (row & 7)) << 4);
      if (copy) {
        copy_unit(at, x + next[i] * p.cols, next[i] >= 0 ? left - u * 8 : 0, p.piece, p.x);
      } else {
        Raw8<T> raw;
        if (HELD) raw = held[HELD ? i : 0];
        else raw.load_by(x + next[i] * p.cols, next[i] >= 0 ? left - u * 8 : 0, 2);
        uint4 v[P];
        planes_of<T, P>(raw, v);
#pragma unroll
        for (int c = 0; c < P; ++c) *reinterpret_cast<uint4*>(at + c * XG) = v[c];
      }
    }
    uint8_t* ht = to + P * XG;
    for (int i = tid; i < GRAD_ROWS * ru; i += kThreads) {
      const int t = i / ru, ju = i - t * ru, in = b * GRAD_ROWS + t;
#pragma unroll
      for (int c = 0; c < PH; ++c) {
        const int j = c * ru + ju;  // unit of the planes one after the other
        ptx::copy16(ht + (j >> 3) * (GRAD_ROWS * 128) + t * 128 + (((j ^ t) & 7) << 4),
                    in < rows ? p.h + ((int64_t)(first + in) * PH + c) * R + ju * 8 : p.h, in < rows);
      }
    }
    if (!HELD) rows_of(b + 1);
  };
  rows_of(b0);
  if (b0 < b1) fetch(b0);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    if (b0 + i < b1) {
      put(b0 + i, sm + i * stage_bytes);
      if (b0 + i + 1 < b1) fetch(b0 + i + 1);
    }
    ptx::copy_commit();
  }
  int slot = 0, use = 0;  // of block b
  for (int b = b0; b < b1; ++b) {
    ptx::copy_wait<S - 2>();
    ptx::fence_proxy_async_smem();
    __syncthreads();
    if (warp == 0) {
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        const uint32_t xa = ptx::smem_addr(sm + slot * stage_bytes), ha = xa + P * XG;
#pragma unroll
        for (int c = 0; c < P; ++c) {
          const int n = (P == 3 ? 3 - c : PH) * R;  // fp32: the smallest products are left out
          for (int n0 = 0; n0 < n; n0 += 256) {
            const int nn = min(256, n - n0);
            const uint32_t id = ptx::idesc_f16(1, GRAD_COLS, nn, true, true);
#pragma unroll
            for (int ks = 0; ks < GRAD_ROWS / 16; ++ks)
              ptx::mma_f16(tmem + (P == 3 ? c * R : 0) + n0,
                           ptx::smem_desc(xa + c * XG + ks * 2048, GRAD_ROWS * 128, 1024, ptx::kSwizzle128B),
                           ptx::smem_desc(ha + n0 * 128 + ks * 2048, GRAD_ROWS * 128, 1024, ptx::kSwizzle128B), id,
                           b > b0 || c > 0 || ks > 0);
          }
        }
        ptx::mma_commit(&ctl.empty[slot]);
      }
      __syncwarp();
    }
    // the next block to load goes where the block before this one was
    if (b + S - 1 < b1) {
      const int last = slot ? slot - 1 : S - 1;
      if (b > b0) tc::warp_wait_bar(&ctl.empty[last], (slot ? use : use - 1) & 1, &ctl.abort, 4, wd);
      put(b + S - 1, sm + last * stage_bytes);
      if (b + S < b1) fetch(b + S);
    }
    ptx::copy_commit();
    if (++slot == S) {
      slot = 0;
      ++use;
    }
  }
  ptx::copy_wait<0>();
  if (b1 > b0) {
    const int done = (b1 - b0 - 1) % S, uses = (b1 - b0 - 1) / S;
    tc::warp_wait_bar(&ctl.empty[done], uses & 1, &ctl.abort, 5, wd);
    ptx::tc_fence_after();
  }
  __syncthreads();
  grad_sums<PH>(sm, tmem, R, b1 > b0, warp >> 2, kWarps / 4);
  ptx::cluster_sync();
  grad_out<T, kThreads>(sm, g, p, l, rank, col0);
  ptx::cluster_sync_reads();  // no CTA ends while another reads its sums
  tear_down(ctl, tmem, g.cols);
}

// The same by fp32 FMAs, for adapters with few rows: nothing is staged but h, no tensor memory
// is set up, and a block has sixteen j's of 256 columns of one adapter, four by four for each
// thread, with all its rows in their order.  (The rule and its figures: run_grads.)
constexpr int FMA_J = 16, FMA_COLS = 256, FMA_ROWS = 64, FMA_THREADS = 256;
template <typename T>
__global__ void __launch_bounds__(FMA_THREADS) k_adapters_grad_fma(const __grid_constant__ GradArgs g) {
  constexpr int PH = Planes<T>::PH, U = 8;
  __shared__ __align__(16) float hs[FMA_ROWS][FMA_J];
  __shared__ int rows[FMA_ROWS];
  const int problem = blockIdx.z / g.blocks;
  const GradProblem& p = g.prob[problem];
  const int R = g.R, r = g.r;
  const int tid = threadIdx.x, lane = tid & 63, l = blockIdx.y;
  const int j0 = (blockIdx.z - problem * g.blocks) * FMA_J, j4 = (tid >> 6) * 4;
  const int64_t col0 = (int64_t)blockIdx.x * FMA_COLS;
  ptx::griddep_wait();
  ptx::griddep_launch();
  if (col0 >= p.cols) return;  // (the problems may have different numbers of columns)
  const int left = (int)(p.cols - col0 < FMA_COLS ? p.cols - col0 : FMA_COLS);
  const int first = __ldg(g.offsets + l), n = __ldg(g.offsets + l + 1) - first;
  const T* x = static_cast<const T*>(p.x) + col0 + lane * 4;
  const int mine = left - lane * 4;
  const bool vec = p.piece >= 4 * (int)sizeof(T);
  float acc[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
  for (int t = 0; t < n; t += FMA_ROWS) {
    const int live = min(FMA_ROWS, n - t);
    if (tid < FMA_ROWS) rows[tid] = tid < live ? __ldg(g.order + first + t + tid) : 0;
    for (int i = tid; i < FMA_ROWS * (FMA_J / 2); i += FMA_THREADS) {  // two j's; zeros past the end
      const int row = i / (FMA_J / 2), j = i % (FMA_J / 2) * 2;
      float a = 0.0f, b = 0.0f;
      if (row < live) {
        const uint32_t* h = reinterpret_cast<const uint32_t*>(p.h + (int64_t)(first + t + row) * PH * R + j0 + j);
#pragma unroll
        for (int c = 0; c < PH; ++c) {
          const uint32_t w = __ldcg(h + c * (R / 2));
          a += __uint_as_float(w << 16);
          b += __uint_as_float(w & 0xFFFF0000u);
        }
      }
      hs[row][j] = a;
      hs[row][j + 1] = b;
    }
    __syncthreads();
    if (mine > 0) {
#pragma unroll 1
      for (int i = 0; i < live; i += U) {
        Raw4<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u].load(x + rows[i + u] * p.cols, i + u < live ? mine : 0, vec);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float4 h = *reinterpret_cast<const float4*>(&hs[i + u][j4]);
          float v[4];
          raw[u].widen(v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[0][e] = fmaf(h.x, v[e], acc[0][e]);
            acc[1][e] = fmaf(h.y, v[e], acc[1][e]);
            acc[2][e] = fmaf(h.z, v[e], acc[2][e]);
            acc[3][e] = fmaf(h.w, v[e], acc[3][e]);
          }
        }
      }
    }
    __syncthreads();
  }
  if (mine <= 0) return;
  T* out = static_cast<T*>(p.out) + (int64_t)l * r * p.cols;
  const int64_t col = col0 + lane * 4;
  auto put = [&](T* to, const float (&v)[4], int have, bool whole) {
    if (whole && have >= 4) {
      alignas(16) T t[4] = {from_f32<T>(v[0]), from_f32<T>(v[1]), from_f32<T>(v[2]), from_f32<T>(v[3])};
      if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(t);
      else *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(t);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < have) to[i] = from_f32<T>(v[i]);
    }
  };
  const bool units = (reinterpret_cast<uintptr_t>(p.out) & (4 * sizeof(T) - 1)) == 0 &&
                     ((p.turned ? (int64_t)r : p.cols) & 3) == 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (p.turned) {  // four j's of a column
      const float v[4] = {acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
      if (i < mine) put(out + (col + i) * r + j0 + j4, v, r - j0 - j4, units);
    } else if (j0 + j4 + i < r) {  // four columns of a j
      put(out + (int64_t)(j0 + j4 + i) * p.cols + col, acc[i], mine, units);
    }
  }
}

// The same for bf16 rows that 16-byte copies can reach, with equal shares however the rows are spread
// over the adapters: a cluster has 128 columns for all adapters, and its CTAs equal runs of
// the blocks of 64 rows, counted over the adapters one after the other.  Two accumulators:
// the next adapter's MMAs run while one's sums are written.  An adapter that lies within a
// run is that CTA's to write; one that several runs share (a run has two such at most) is
// summed at the end, in the order of the CTAs, each taking a part of its gradient.  All
// gradients of 8192 rows of 8 adapters, r 16, 4096 x 4096: 105 us, 113 with an adapter's rows to
// each cluster (one adapter: 90, 85).  This launch takes 31 of the 90 (134 MB, a third of them
// from L2): 0.75 us for each block of a CTA, whatever the number of stages beyond three.
struct GradMaps {
  CUtensorMap x[2], h[2];  // of each problem, by 64 rows
};
constexpr int GRAD_LOAD = 4, GRAD_EPI = 4, GRAD_THREADS = (GRAD_LOAD + 1 + GRAD_EPI) * 32;  // loaders, MMAs, epilogue
struct GradCtl {
  // (full and acce take an arrival of each of four warps, the others one)
  uint64_t full[DOWN_STAGES], acce[2], empty[DOWN_STAGES], accf[2], drain;
  uint32_t tmem_base;
  int abort;
  int sums[16];
  int before[kAdapters + 2];  // row blocks before an adapter
};

__global__ void __launch_bounds__(GRAD_THREADS) k_adapters_grad_runs(const __grid_constant__ GradMaps maps,
                                                                          const __grid_constant__ GradArgs g) {
  using T = __nv_bfloat16;
  constexpr int PH = Planes<T>::PH, XG = GRAD_ROWS * GRAD_COLS * 2;
  extern __shared__ uint8_t sm_raw[];
  __shared__ GradCtl ctl;
  uint8_t* sm = tc::smem_align1024(sm_raw);
  const GradProblem& p = g.prob[blockIdx.y];
  const int C = 1 << g.log_ctas, rank = (int)ptx::cluster_rank(), S = g.stages;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, R = g.R, r = g.r, L = g.L;
  const int64_t col0 = (int64_t)(blockIdx.x >> g.log_ctas) * GRAD_COLS;
  const int left = (int)(p.cols - col0 < GRAD_COLS ? p.cols - col0 : GRAD_COLS);
  int* wd = &g_watchdog_adapters;
  if (left <= 0) return;  // the whole cluster (the problems may have different numbers of columns)
  static_assert(GRAD_LOAD == GRAD_EPI, "arrivals");
  const uint32_t tmem = set_up(ctl, 2 * DOWN_STAGES + 5, ctl.full, g.cols, DOWN_STAGES + 2, GRAD_LOAD);
  if (tid == 32) {
    ptx::tma_prefetch_desc(&maps.x[blockIdx.y]);
    ptx::tma_prefetch_desc(&maps.h[blockIdx.y]);
  }
  ptx::griddep_wait();
  ptx::griddep_launch();
  count_tiles<GRAD_THREADS>(g.offsets, L, GRAD_ROWS, nullptr, ctl.before, ctl.sums);
  const int blocks = ctl.before[L];
  auto run_of = [&](int q) { return (int)((int64_t)blocks * q >> g.log_ctas); };
  const int b0 = run_of(rank), b1 = run_of(rank + 1);
  const int hb = grad_h_bytes(PH * R), stage_bytes = XG + hb;
  const int pitch = R + 1;
  float* head = reinterpret_cast<float*>(sm + S * stage_bytes);  // sums of the run's first adapter
  float* tail = reinterpret_cast<float*>(sm);                    // of its last, when the ring is done
  // the adapter of row block b
  auto adapter_of = [&](int b) {
    int low = 0, high = L;  // before[low] <= b < before[high]
    while (high - low > 1) {
      const int mid = (low + high) >> 1;
      if (ctl.before[mid] <= b) low = mid;
      else high = mid;
    }
    return low;
  };
  T* out = static_cast<T*>(p.out);
  if (warp < GRAD_LOAD) {
    // A full block of rows that lie one after the other: a box of 64 columns of x by each of
    // the first two warps, h by the third.  Else sixteen rows and their h by each warp, x two
    // rows at a time; zeros past the adapter's end.  The rows' numbers (a lane has two) are
    // asked for two blocks early.
    const void *mx = &maps.x[blockIdx.y], *mh = &maps.h[blockIdx.y];
    const int unit = lane & 15, hu = PH * R / 8, mine = warp * 16;
    const int h_row = lane / hu, h_by = 32 / hu;
    const T* x = static_cast<const T*>(p.x) + col0 + unit * 8;
    const bool in_x = unit * 8 < left;
    int l = b0 < b1 ? adapter_of(b0) : 0;
    struct Rows {
      int place, have, lo, hi;  // first place, rows, this lane's rows of the two halves
    };
    auto rows_of = [&](int b) {
      Rows q = {0, 0, -1, -1};
      if (b >= b1) return q;
      while (ctl.before[l + 1] <= b) ++l;
      q.place = __ldg(g.offsets + l) + (b - ctl.before[l]) * GRAD_ROWS;
      q.have = min(GRAD_ROWS, __ldg(g.offsets + l + 1) - q.place);
      if (lane < q.have) q.lo = __ldg(g.order + q.place + lane);
      if (lane + 32 < q.have) q.hi = __ldg(g.order + q.place + lane + 32);
      return q;
    };
    Rows now = rows_of(b0), next = rows_of(b0 + 1);
    Slot ring;
    Landing land(S);
    int b = b0;
    for (; b < b1; ++b, ring.next(S)) {
      const int slot = ring.i;
      const Rows after = rows_of(b + 2);
      if (ring.round > 0 && !tc::warp_wait_bar(&ctl.empty[slot], (ring.round - 1) & 1, &ctl.abort, 4, wd)) break;
      uint8_t* to = sm + slot * stage_bytes;
      uint64_t* bar = &ctl.full[slot];
      const int head = __shfl_sync(kAll, now.lo, 0);
      if (now.have == GRAD_ROWS && __all_sync(kAll, now.lo == head + lane && now.hi == head + 32 + lane)) {
        land.skip(ctl.full, S);
        if (lane == 0) {
          if (warp < 2 && warp * 64 < left) {
            ptx::mbar_arrive_expect_tx(bar, XG / 2);
            ptx::tma_load_2d(to + warp * (XG / 2), mx, bar, (int)col0 + warp * 64, head);
          } else if (warp == 2) {
            ptx::mbar_arrive_expect_tx(bar, hb);
            for (int j = 0; j < PH * R; j += 64) ptx::tma_load_2d(to + XG + j * 128, mh, bar, j, now.place);
          } else {
            ptx::mbar_arrive(bar);
          }
        }
        __syncwarp();
      } else {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const int at = mine + i + (lane >> 4);
          const int lo = __shfl_sync(kAll, now.lo, at & 31), hi = __shfl_sync(kAll, now.hi, at & 31);
          const int64_t row = at & 32 ? hi : lo;
          const bool have = row >= 0 && in_x;
          ptx::copy16(to + (unit >> 3) * (GRAD_ROWS * 128) + at * 128 + (((unit ^ at) & 7) << 4),
                      have ? x + row * p.cols : static_cast<const T*>(p.x), have);
        }
        if (h_row < h_by) {
          const int u = lane - h_row * hu;
          for (int i = h_row; i < 16; i += h_by) {
            const int at = mine + i;
            const bool have = at < now.have;
            ptx::copy16(to + XG + (u >> 3) * (GRAD_ROWS * 128) + at * 128 + (((u ^ at) & 7) << 4),
                        have ? p.h + (int64_t)(now.place + at) * PH * R + u * 8 : p.h, have);
          }
        }
        land.next(ctl.full, S);
      }
      now = next;
      next = after;
    }
    land.finish(ctl.full, S);
    if (ctl.abort) drain_ring(ctl.full, S, b - b0);
  } else if (warp == GRAD_LOAD) {
    const uint32_t id = ptx::idesc_f16(1, GRAD_COLS, PH * R, true, true);
    Slot ring, acc;
    int l = b0 < b1 ? adapter_of(b0) : 0, end = 0;
    for (int b = b0; b < b1; ++b, ring.next(S)) {
      const int slot = ring.i;
      const bool fresh = b >= end;  // the first block of an adapter's segment
      if (fresh) {
        while (ctl.before[l + 1] <= b) ++l;
        end = min(ctl.before[l + 1], b1);
        if (acc.round > 0 && !tc::warp_wait_bar(&ctl.acce[acc.i], (acc.round - 1) & 1, &ctl.abort, 15, wd)) break;
      }
      if (!tc::warp_wait_bar(&ctl.full[slot], ring.round & 1, &ctl.abort, 14, wd)) break;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        const uint32_t xa = ptx::smem_addr(sm + slot * stage_bytes), ha = xa + XG;
#pragma unroll
        for (int ks = 0; ks < GRAD_ROWS / 16; ++ks)
          ptx::mma_f16(tmem + acc.i * PH * R, ptx::smem_desc(xa + ks * 2048, GRAD_ROWS * 128, 1024, ptx::kSwizzle128B),
                       ptx::smem_desc(ha + ks * 2048, GRAD_ROWS * 128, 1024, ptx::kSwizzle128B), id,
                       !fresh || ks > 0);
        ptx::mma_commit(&ctl.empty[slot]);
        if (b + 1 == end) ptx::mma_commit(&ctl.accf[acc.i]);
      }
      __syncwarp();
      if (b + 1 == end) acc.next(2);
    }
  } else {
    // a thread has a column's sums
    const int col = (warp & 3) * 32 + lane;
    const bool vec = r == R && (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
    Slot acc;
    int l = b0 < b1 ? adapter_of(b0) : 0;
    for (int b = b0; b < b1;) {
      while (ctl.before[l + 1] <= b) ++l;
      const int end = min(ctl.before[l + 1], b1);
      const bool begins = ctl.before[l] >= b0, ends = ctl.before[l + 1] <= b1;
      if (!tc::warp_wait_bar(&ctl.accf[acc.i], acc.round & 1, &ctl.abort, 5, wd)) break;
      ptx::tc_fence_after();
      const uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16) + acc.i * PH * R;
      T* to = out + (int64_t)l * r * p.cols;
      for (int j = 0; j < R; j += 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < PH; ++c) {
          uint32_t w[16];
          ptx::tmem_ld16(from + c * R + j, w);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(w[i]);
        }
        if (!begins || !ends) {
          float* part = (begins ? tail : head) + col * pitch + j;
#pragma unroll
          for (int i = 0; i < 16; ++i) part[i] = v[i];
        } else if (col < left) {
          if (!p.turned) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (j + i < r) to[(int64_t)(j + i) * p.cols + col0 + col] = from_f32<T>(v[i]);
          } else {
            float lo[8], hi[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) lo[i] = v[i], hi[i] = v[8 + i];
            T* at = to + (col0 + col) * r + j;
            store8<T>(at, r - j, vec, lo);
            store8<T>(at + 8, r - j - 8, vec, hi);
          }
        }
      }
      // Each warp arrives for itself: one may leave this loop (its wait gave up) while another
      // goes on, so nothing here may wait for all of them.
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ctl.acce[acc.i]);
      acc.next(2);
      b = end;
    }
  }
  __syncwarp();
  ptx::cluster_sync();
  // ---- the shared adapters: the run's first, if it began before; its last, if it goes on
  if (b0 < b1) {
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const int l = adapter_of(which ? b1 - 1 : b0);
      const int begin = ctl.before[l], end = ctl.before[l + 1];
      const bool begins = begin >= b0, ends = end <= b1;
      if (which ? !begins || ends : begins) continue;
      int ra = rank, rb = rank;  // the CTAs that share it
      while (ra > 0 && run_of(ra) > begin) --ra;
      while (rb + 1 < C && run_of(rb + 1) < end) ++rb;
      int sharers = 0, before = 0;  // without those that have no row blocks
      for (int q = ra; q <= rb; ++q)
        if (run_of(q) < run_of(q + 1)) {
          ++sharers;
          before += q < rank ? 1 : 0;
        }
      const int n = left * r, share = (n + sharers - 1) / sharers, e0 = before * share, e1 = min(e0 + share, n);
      for (int e = e0 + tid; e < e1; e += GRAD_THREADS) {
        const int col = p.turned ? e / r : e % left, j = p.turned ? e - col * r : e / left;
        float sum = 0.0f;
        for (int q = ra; q <= rb; ++q) {
          if (run_of(q) == run_of(q + 1)) continue;  // (no row blocks)
          sum += __uint_as_float(ptx::ld_cluster(ptx::cluster_addr((q == ra ? tail : head) + col * pitch + j, q)));
        }
        out[(int64_t)l * r * p.cols + (p.turned ? (col0 + col) * r + j : (int64_t)j * p.cols + col0 + col)] =
            from_f32<T>(sum);
      }
    }
  }
  // ---- adapters without rows: zeros
  for (int l = rank; l < L; l += C) {
    if (ctl.before[l + 1] > ctl.before[l]) continue;
    for (int e = tid; e < left * r; e += GRAD_THREADS) {
      const int col = p.turned ? e / r : e % left, j = p.turned ? e - col * r : e / left;
      out[(int64_t)l * r * p.cols + (p.turned ? (col0 + col) * r + j : (int64_t)j * p.cols + col0 + col)] =
          from_f32<T>(0.0f);
    }
  }
  ptx::cluster_sync_reads();  // no CTA ends while another reads its sums
  tear_down(ctl, tmem, g.cols);
}

// ------------------------------------------------------------------- host
// What rows at p, `pitch` bytes apart, are aligned to: 16, 8, 4 or 2 bytes.
int piece_of(const void* p, int64_t pitch) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p) | (uintptr_t)pitch;
  return bits & 3 ? 2 : (bits & 7 ? 4 : (bits & 15 ? 8 : 16));
}
bool aligned16(const void* p, int64_t pitch) { return piece_of(p, pitch) == 16; }

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
size_t smem_for(size_t bytes, int cols, size_t fixed = 2048) {  // fixed: static shared memory, at most
  const size_t share = (size_t)(228 << 10) * cols / 512 - 1024, most = kBlockSharedMemory - fixed;
  bytes = bytes > share ? bytes : share;
  return bytes < most ? bytes : most;
}

int round16(int r) { return (r + 15) / 16 * 16; }

template <typename T>
cudaError_t adapters_few(const AdapterArgs& a, cudaStream_t s) {
  note_kernel_name("k_adapters_few");
  const int64_t tiles = most_tiles(a.T, a.L, FEW), b = sizeof(T);
  FewArgs g = {};
  g.a = a;
  // Eight CTAs a tile; four where those are more than 3.5 an SM (us with 8 / 4, bf16, r 16, 4096 x
  // 4096: 64 rows of 64 adapters 9.5 / 11.7, 512 rows of 8 22.2 / 19.0, 1000 rows of 64 34.0 / 31.8).
  // fp32, two CTAs an SM: four where eight do not run at once (64 rows of 64, 4096 x 1024: 13.2 / 8.7).
  g.log_ctas = tiles * 16 <= (sizeof(T) == 4 ? 4 : 7) * device_sm_count() ? 3 : 2;
  g.none = a.base != a.out ? 1 : 0;
  g.vec = (aligned16(a.x, a.ld * b) ? 1 : 0) | (aligned16(a.a, a.K * b) ? 2 : 0) |
          (a.r % 4 == 0 && reinterpret_cast<uintptr_t>(a.b) % (4 * b) == 0 ? 4 : 0);
  g.R = round16(a.r);
  g.blocks = g.R / 16;
  g.parts = kWarps / g.blocks;
  const int C = 1 << g.log_ctas;
  const size_t smem = (size_t)((g.parts + C) * FEW * g.R + FEW * FEW_PITCH) * 4 + (size_t)2 * FEW * (g.R * b + 16);
  return launch_clusters<k_adapters_few<T>>(dim3((unsigned)(tiles << g.log_ctas)), C, kThreads, smem, s, g);
}

// The kernel form by r rounded up to 16.
#define IMC_BY_RANK(R, CALL) \
  do {                       \
    if ((R) <= 32) CALL(1);  \
    if ((R) <= 64) CALL(2);  \
    CALL(4);                 \
  } while (0)

// Tensor maps.  TMA reads rows that are 16-byte aligned.
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
    else
      cudaGetLastError();
  });
  return fn;
}
// [batch][rows][cols], rows ld elements apart (batch 0: two dimensions), in boxes of box_rows
// x box_bytes (32, 64 or 128) of columns, swizzled by as much.
template <typename T>
bool encode(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_rows,
            int64_t batch = 0, int box_bytes = 128) {
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
  const cuuint64_t strides[2] = {(cuuint64_t)(ld * sizeof(T)), (cuuint64_t)(rows * ld * sizeof(T))};
  const cuuint32_t box[3] = {box_bytes / (cuuint32_t)sizeof(T), (cuuint32_t)box_rows, 1}, es[3] = {1, 1, 1};
  const CUtensorMapDataType type = sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  const CUtensorMapSwizzle swizzle =
      box_bytes == 32 ? CU_TENSOR_MAP_SWIZZLE_32B : (box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  return encode_fn()(m, type, batch ? 3 : 2, const_cast<void*>(base), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// h: a box is one plane of 128 rows, 128 bytes at most.
bool encode_h(CUtensorMap* m, const uint16_t* h, int64_t T, int R, int planes) {
  const Along along(R);
  const cuuint64_t dims[3] = {(cuuint64_t)R, (cuuint64_t)planes, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)R * 2, (cuuint64_t)planes * R * 2};
  const cuuint32_t box[3] = {(cuuint32_t)along.bytes / 2, 1, TILE}, es[3] = {1, 1, 1};
  const CUtensorMapSwizzle swizzle = along.bytes == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                       : (along.bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<uint16_t*>(h), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks of `smem` bytes (and under 1 KB of static shared memory) that an SM holds.
int64_t resident(size_t smem) { return (228 << 10) / (int64_t)((smem + 1023) / 1024 * 1024 + 2048); }
// CTAs of a cluster, as log2: as many as keep the tiles' clusters, about T / 128 and half a
// tile for each adapter, resident at once.
int cluster_log(int64_t room, int64_t T, int64_t L, int problems) {
  const int64_t tiles = ceil_div(T, TILE) + (T < L ? T : L) / 2, want = room / (tiles * problems);
  return want >= 8 ? 3 : (want >= 4 ? 2 : (want >= 2 ? 1 : 0));
}

template <typename T>
cudaError_t run_down_tma(DownArgs& g, int problems, cudaStream_t s) {
  DownMaps maps = {};
  for (int i = 0; i < problems; ++i) {
    const DownProblem& p = g.prob[i];
    const bool w = p.turned ? encode<T>(&maps.w[i], p.w, g.r, p.K, g.r, KB, g.L)
                            : encode<T>(&maps.w[i], p.w, p.K, g.r, p.K, g.R, g.L);
    if (!w || !encode<T>(&maps.x[i], p.x, p.K, g.T, p.ld, 32)) return cudaErrorInvalidValue;
  }
  const int64_t tiles = most_tiles(g.T, g.L, TILE);
  // Two blocks per SM, with a ring of up to 104 KB each (what is under way decides: 8192 rows of
  // 8 adapters, r 32, 4096 x 4096, bf16, take 44.9 us, 48.2 with 60 KB); three stages at least,
  // as Landing needs.
  g.log_ctas = cluster_log(2 * (int64_t)device_sm_count(), g.T, g.L, problems);
  g.w_bytes = g.R * 128;
  for (int i = 0; i < problems; ++i)
    if (g.prob[i].turned) g.w_bytes = down_w_bytes(g.R);
  const int stage = XP + g.w_bytes, sums = TILE * (g.R * 4 + 16);
  g.stages = (104 << 10) / stage < DOWN_STAGES ? (104 << 10) / stage : DOWN_STAGES;
  const int bytes = g.stages * stage > sums ? g.stages * stage : sums;
  g.cols = tmem_cols(g.R);
  return launch_clusters<k_adapters_down_tma<T>>(dim3((unsigned)(tiles << g.log_ctas), problems), 1 << g.log_ctas,
                                                 DOWN_THREADS, smem_for((size_t)bytes + 1024, g.cols), s, maps, g);
}

template <typename T>
cudaError_t run_down(DownArgs& g, int problems, cudaStream_t s) {
  using PL = Planes<T>;
  if constexpr (sizeof(T) == 2) {
    bool tma = encode_fn() != nullptr;
    for (int i = 0; i < problems; ++i) tma = tma && g.prob[i].x_piece == 16 && g.prob[i].w_piece == 16;
    if (tma) return run_down_tma<T>(g, problems, s);
  }
  const int64_t tiles = most_tiles(g.T, g.L, TILE);
  const int ring = PL::STAGES * (PL::PD * XP + down_w_bytes(PL::PD * g.R)), sums = TILE * (g.R * 4 + 16);
  g.cols = tmem_cols(PL::PD * g.R);
  const size_t smem = smem_for((size_t)(ring > sums ? ring : sums), g.cols);
  g.log_ctas = cluster_log(resident(smem) * device_sm_count(), g.T, g.L, problems);
  const dim3 grid((unsigned)(tiles << g.log_ctas), problems);
#define IMC_DOWN(RU) return launch_clusters<k_adapters_down<T, RU>>(grid, 1 << g.log_ctas, kThreads, smem, s, g)
  IMC_BY_RANK(g.R, IMC_DOWN);
#undef IMC_DOWN
}

// Shared memory of a second product's block: what the kernel declares (in whole KB, since the
// rings behind it are aligned to one), and a KB to align them by itself.
constexpr int UP_STATIC = ((int)sizeof(UpCtl) + 1023) / 1024 * 1024, UP_ROOM = kBlockSharedMemory - UP_STATIC - 1024;

template <typename T, bool TMA>
cudaError_t run_up_as(UpArgs& g, const uint16_t* h, cudaStream_t s) {
  using PL = Planes<T>;
  const Along along(g.R);
  constexpr int part = UP_EPI * UP_PART<T, TMA>, staged = UP_EPI * 32 * (STAGED_COLS + 1) * 4;
  // rings: at least two parts of base, one h, one w; then more parts, w, h
  const int table = buckets_bytes(g.L), most = UP_ROOM - table;
  const bool ring = 2 * part + g.h_bytes + g.w_bytes <= most;
  g.slots = g.h_slots = 1;
  g.b_slots = ring ? 2 : 0;
  auto bytes = [&] { return g.b_slots * part + g.slots * g.w_bytes + g.h_slots * g.h_bytes + (ring ? 0 : staged); };
  // two blocks on an SM where both find room with two slots for w
  int limit = most, blocks = 1;
  if (sizeof(T) == 2) {
    const int half = (228 << 9) - 1024 - UP_STATIC - 1024 - table;
    g.slots = 2;
    if (bytes() <= half) {
      limit = half;
      blocks = 2;
    }
    g.slots = 1;
  }
  auto grow = [&](int& n, int to) {
    while (n < to) {
      ++n;
      if (bytes() <= limit) continue;
      --n;
      break;
    }
  };
  if (bytes() > most || (TMA && !ring)) return cudaErrorInvalidValue;
  grow(g.slots, 2);
  if (ring) grow(g.b_slots, BASE_SLOTS);
  grow(g.h_slots, 2);
  grow(g.slots, UP_SLOTS);
  g.buckets = bytes();
  UpMaps maps = {};
  bool ok = encode_h(&maps.h, h, g.T, g.R, PL::PH);
  if (TMA && g.base) ok = ok && encode<T>(&maps.base, g.base, g.N, g.T, g.N, 32);
  if (TMA) ok = ok && encode<T>(&maps.out, g.out, g.N, g.T, g.N, 32);
  if (g.vec)
    ok = ok && (g.turned ? encode<T>(&maps.w, g.w, g.N, g.r, g.N, g.R, g.L)
                         : encode<T>(&maps.w, g.w, g.r, g.N, g.r, UP_N, g.L, along.bytes));
  if (!ok) return cudaErrorInvalidValue;
  const int64_t items = most_tiles(g.T, g.L, TILE) * g.steps, most_blocks = (int64_t)device_sm_count() * blocks;
  // (us with one item at a time / two: 8192 rows of 8 adapters, r 32, 4096 x 4096, bf16: 47.0 / 45.4;
  // 4096 rows of 8, r 16, 1024 x 1024, fp16, no more items than blocks: 14.9 / 17.1)
  g.group = items > 4 * most_blocks ? 2 : 1;
  const int grid = (int)(items < most_blocks ? items : most_blocks);
  g.jump = (grid - 1) * g.group + 1;
  g.jump_tiles = g.jump / g.steps;
  g.jump_steps = g.jump % g.steps;
  return launch_clusters<k_adapters_up<T, TMA>>(dim3(grid), 1, UP_THREADS<T>, (size_t)bytes() + table + 1024, s, maps, g);
}

template <typename T>
cudaError_t run_up(UpArgs& g, const uint16_t* h, cudaStream_t s) {
  using PL = Planes<T>;
  const int64_t b = sizeof(T);
  const Along along(g.R);
  if (!encode_fn()) return cudaErrorNotSupported;
  g.steps = (int)ceil_div(g.N, UP_N);
  g.w_bytes = PL::PD * (g.turned ? g.R * 256 : along.plane());
  g.h_bytes = PL::PH * along.plane();
  g.piece = piece_of(g.out, g.N * b | (int64_t)(reinterpret_cast<uintptr_t>(g.base) & 15));
  g.w_piece = piece_of(g.w, (g.turned ? g.N : g.r) * b);
  g.vec = g.w_piece == 16 && PL::PD == 1 ? 1 : 0;
  // TMA: two parts of base have to fit beside h and w (fp32: up to rank 32, or 64 and 126 adapters)
  const bool fits = 2 * UP_EPI * UP_PART<T, true> + g.h_bytes + g.w_bytes <= UP_ROOM - buckets_bytes(g.L);
  return g.piece == 16 && fits ? run_up_as<T, true>(g, h, s) : run_up_as<T, false>(g, h, s);
}

// The form for few rows: an adapter has sixteen on average at most, whose tiles of 128 would
// be nearly empty, or there are few altogether, and one launch is over sooner than two; but not
// more tiles of eight than 256, whose clusters run one after the other.  us with it / in tiles
// (bf16, 4096 x 4096 where nothing else is said): 64 rows of 64 adapters, r 16, 9.1 / 27.0; 1000
// of 64 30.5 / 34.5; 2000 of 64 50.0 / 35.2; 8000 of 600, r 8, 512 x 512 78.9 / 41.1; 600 of 60,
// 1024 x 2048 11.6 / 26.7; 128 of 1 9.7 / 11.9; 512 of 1 21.9 / 12.8, 1024 x 1024 10.6 / 10.2;
// 256 of 1, r 32, 1024 x 1024 7.5 / 10.4; 256 of 8, r 64, 19.2 / 19.4; fp32 777 of 5, r 9, 1100 x
// 1001 12.6 / 17.4.
bool few_rows(int64_t T, int64_t L, int64_t r) {
  return (T <= 16 * L || T * r <= 8192) && most_tiles(T, L, FEW) <= 256;
}

// The workspace of one h (of g): its planes, its scaled fp16 rows, their scales.
size_t room_bytes(int64_t T, int64_t R) { return (size_t)(T * R * (6 + 4) + (T + 3) / 4 * 16); }
struct Room {
  uint16_t *h, *h16;
  float* row_scale;
};
Room room_of(void* workspace, int i, int64_t T, int64_t R) {
  uint16_t* h = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + i * room_bytes(T, R));
  return {h, h + 3 * T * R, reinterpret_cast<float*>(h + 5 * T * R)};
}

template <typename T>
cudaError_t adapters(const AdapterArgs& a, cudaStream_t s) {
  if (few_rows(a.T, a.L, a.r)) return adapters_few<T>(a, s);
  note_kernel_name("k_adapters_up");
  const int64_t b = sizeof(T);
  DownArgs g = {};
  g.scale = a.scale;
  g.offsets = a.offsets;
  g.order = a.order;
  g.T = a.T;
  g.L = a.L;
  g.r = a.r;
  g.R = round16(a.r);
  const Room room = room_of(a.workspace, 0, a.T, g.R);
  constexpr bool F16 = Planes<T>::FD == 0;
  g.prob[0] = {a.x, a.ld, a.K, a.a, F16 ? nullptr : room.h, F16 ? room.h16 : nullptr, F16 ? room.row_scale : nullptr, 0,
               piece_of(a.x, a.ld * b | a.K * b), piece_of(a.a, a.K * b)};
  const cudaError_t e = run_down<T>(g, 1, s);
  if (e != cudaSuccess) return e;
  UpArgs up = {g.prob[0].row_scale, a.b, a.base, a.out, a.offsets, a.order, a.T, a.N, a.L, a.r, g.R};
  return run_up<T>(up, F16 ? room.h16 : room.h, s);
}

template <typename T>
cudaError_t run_grads(const AdapterGradArgs& a, int R, const uint16_t* h, const uint16_t* d, cudaStream_t s) {
  using PL = Planes<T>;
  GradArgs w = {};
  w.offsets = a.offsets;
  w.order = a.order;
  w.T = a.T;
  w.L = a.L;
  w.r = a.r;
  w.R = R;
  int parts = 0;
  int64_t chunks = 0, all = 0;
  auto add = [&](const void* x, int64_t cols, const uint16_t* planes, void* out, int turned) {
    GradProblem& p = w.prob[parts++];
    p.x = x;
    p.cols = cols;
    p.h = planes;
    p.out = out;
    p.turned = turned;
    p.piece = piece_of(x, cols * (int64_t)sizeof(T));
    const int64_t n = ceil_div(cols, GRAD_COLS);
    chunks = chunks > n ? chunks : n;
    all += n;
  };
  if (a.grad_a) add(a.x, a.K, d, a.grad_a, 0);
  if (a.grad_b) add(a.grad, a.N, h, a.grad_b, 1);
  w.blocks = R / FMA_J;
  // Adapters of up to 48 rows on average (16 where x cannot be read by four values): FMAs (all
  // gradients, us with them / in tiles, r 16: bf16 318 rows of 61 adapters, 344 x 120, 21.2 / 55.2;
  // bf16 1200 of 42, 1024 x 1024, 30.6 / 38.3; fp32 1636 of 42, 448 x 3232, 56.9 / 69.7; but bf16 512
  // of 8, 4096 x 4096, 45.1 / 34.1, fp16 2048 of 32, 1024 x 1024, 44.1 / 32.7, and fp32 308 of 15, 1045
  // x 439, 33.0 / 28.7).
  bool units = true;
  for (int i = 0; i < parts; ++i) units = units && w.prob[i].piece >= 4 * (int)sizeof(T);
  if (a.T <= (units ? 48 : 16) * a.L) {
    int64_t most_chunks = 0;
    for (int i = 0; i < parts; ++i) {
      const int64_t n = ceil_div(w.prob[i].cols, FMA_COLS);
      most_chunks = most_chunks > n ? most_chunks : n;
    }
    return launch_clusters<k_adapters_grad_fma<T>>(dim3((unsigned)most_chunks, a.L, parts * w.blocks), 1, FMA_THREADS, 0,
                                                   s, w);
  }
  // About four blocks per SM, of a stage of rows on average at least (fp32 2047 rows of 4 adapters,
  // r 8, 1000 x 2048: 41.4 us for 52.8 with four stages at least; fp32 4096 of 8, r 16, 2048 x
  // 2048: 79 for 95 with three blocks).
  int64_t want = 4 * (int64_t)device_sm_count() / (all * a.L);
  const int64_t most = a.T / a.L / GRAD_ROWS;
  want = want < most ? want : most;
  w.log_ctas = want >= 8 ? 3 : (want >= 4 ? 2 : (want >= 2 ? 1 : 0));
  if constexpr (PL::P == 1) {
    bool copies = encode_fn() != nullptr;
    for (int i = 0; i < parts; ++i) copies = copies && w.prob[i].piece == 16;
    if (copies) {
      GradMaps maps = {};
      for (int i = 0; i < parts; ++i)
        if (!encode<T>(&maps.x[i], w.prob[i].x, w.prob[i].cols, a.T, w.prob[i].cols, GRAD_ROWS) ||
            !encode<T>(&maps.h[i], w.prob[i].h, PL::PH * w.R, a.T, PL::PH * w.R, GRAD_ROWS))
          return cudaErrorInvalidValue;
      const int stage = GRAD_ROWS * GRAD_COLS * 2 + grad_h_bytes(PL::PH * w.R), sums = GRAD_COLS * (w.R + 1) * 4;
      // two blocks per SM where three stages and a set of sums fit in half of it
      const int fixed = (int)(sizeof(GradCtl) + 1023) / 1024 * 1024 + 256;  // static shared memory
      const int half = (114 << 10) - 1024 - fixed - 1024, most = kBlockSharedMemory - fixed - 1024;
      const int room = 3 * stage + sums <= half ? half : most;
      w.stages = (room - sums) / stage < DOWN_STAGES ? (room - sums) / stage : DOWN_STAGES;
      while (w.stages * stage < sums) ++w.stages;  // (the ring holds a set of sums, too, in the end)
      w.cols = tmem_cols(2 * PL::PH * w.R);
      const int64_t blocks = ceil_div(a.T, GRAD_ROWS), per_chunk = (room == half ? 2 : 1) * (int64_t)device_sm_count() / all;
      const int64_t ctas = per_chunk < blocks ? per_chunk : blocks;
      w.log_ctas = ctas >= 8 ? 3 : (ctas >= 4 ? 2 : (ctas >= 2 ? 1 : 0));
      return launch_clusters<k_adapters_grad_runs>(dim3((unsigned)(chunks << w.log_ctas), parts), 1 << w.log_ctas, GRAD_THREADS,
                                                  smem_for((size_t)w.stages * stage + sums + 1024, w.cols, fixed), s, maps, w);
    }
  }
  const size_t ring = (size_t)PL::GRAD_STAGES * (PL::P * GRAD_ROWS * GRAD_COLS * 2 + grad_h_bytes(PL::PH * w.R));
  const size_t sums = (size_t)GRAD_COLS * (w.R + 1) * 4;
  w.cols = tmem_cols(PL::PH * w.R);
  const size_t smem = smem_for(ring > sums ? ring : sums, w.cols);
  return launch_clusters<k_adapters_grad<T>>(dim3((unsigned)(chunks << w.log_ctas), a.L, parts), 1 << w.log_ctas,
                                             kThreads, smem, s, w);
}

template <typename T>
cudaError_t backward(const AdapterGradArgs& a, cudaStream_t s) {
  using PL = Planes<T>;
  note_kernel_name("k_adapters_grad");
  constexpr bool F16 = PL::FD == 0;
  DownArgs g = {};
  g.scale = a.scale;
  g.offsets = a.offsets;
  g.order = a.order;
  g.T = a.T;
  g.L = a.L;
  g.r = a.r;
  g.R = round16(a.r);
  const int64_t size = sizeof(T);
  const Room h = room_of(a.workspace, 0, a.T, g.R), d = room_of(a.workspace, 1, a.T, g.R);
  const bool scaled = F16 && a.grad_x;
  int problems = 0;
  if (a.grad_x || a.grad_a)  // g = scale * grad b
    g.prob[problems++] = {a.grad, a.N, a.N, a.b, F16 && !a.grad_a ? nullptr : d.h, scaled ? d.h16 : nullptr,
                          scaled ? d.row_scale : nullptr, 1,
                          piece_of(a.grad, a.N * size), piece_of(a.b, a.r * size)};
  if (a.grad_b)  // h = scale * x a^T
    g.prob[problems++] = {a.x, a.K, a.K, a.a, h.h, nullptr, nullptr, 0,
                          piece_of(a.x, a.K * size), piece_of(a.a, a.K * size)};
  cudaError_t e = run_down<T>(g, problems, s);
  // the weights' gradients first: they read x and grad again, some of which L2 still has
  if (e == cudaSuccess && (a.grad_a || a.grad_b)) e = run_grads<T>(a, g.R, h.h, d.h, s);
  if (e == cudaSuccess && a.grad_x) {
    UpArgs up = {scaled ? d.row_scale : nullptr, a.a, a.base, a.grad_x, a.offsets, a.order, a.T, a.K, a.L, a.r, g.R};
    up.turned = 1;
    e = run_up<T>(up, scaled ? d.h16 : d.h, s);
  }
  return e;
}

}  // namespace

cudaError_t launch_adapters(const AdapterArgs& a, int dtype, cudaStream_t s) {
  if (dtype == IMC_F32) return adapters<float>(a, s);
  if (dtype == IMC_F16) return adapters<__half>(a, s);
  return adapters<__nv_bfloat16>(a, s);
}

size_t adapters_bytes(int64_t T, int64_t L, int64_t r) {
  return few_rows(T, L, r) ? 0 : room_bytes(T, round16((int)r));
}
size_t adapters_backward_bytes(int64_t T, int64_t r) {
  return 2 * room_bytes(T, round16((int)r));
}

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
