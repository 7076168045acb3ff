// Quantisation to MXFP4 and back.
//
// A block of 32 consecutive values of a row shares the scale 2^e,
// e = clamp(floor(log2(max |x|)) - 2, -127, 127), so that the largest magnitude
// lands in [4, 8), and each value becomes the E2M1 number nearest to x * 2^-e
// (ties to the even code, magnitudes above 6 become 6).  floor(log2) is the
// exponent field of the fp32 maximum and 2^-e a float built from it, so every
// step but the final rounding is exact.  A block that holds an infinity or a
// NaN gets the scale byte 255 (NaN): it stands for 32 NaNs.
#include "mx_internal.cuh"
#include "ptx.cuh"

namespace imc {
namespace mx {
namespace {

// Scale byte of a block from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t max_bits) {
  const uint32_t e = max_bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - byte), the factor that brings a block into [0, 8); 0 for a NaN
// block (its codes are then 0).
__device__ __forceinline__ float scale_up(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// 2^(byte - 127) (a denormal for byte 0), NaN for 255.
__device__ __forceinline__ float scale_down(uint32_t byte) {
  if (byte == 255u) return __uint_as_float(0x7FC00000u);
  return byte == 0u ? __uint_as_float(1u << 22) : __uint_as_float(byte << 23);
}

// Eight scaled values to eight E2M1 codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float up) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0] * up), "f"(v[1] * up), "f"(v[2] * up), "f"(v[3] * up), "f"(v[4] * up),
        "f"(v[5] * up), "f"(v[6] * up), "f"(v[7] * up));
  return r;
}
__device__ __forceinline__ uint32_t max_bits8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// Which rows and columns a half-warp takes: 16 lanes cover 128 columns of a row
// (a lane 8 columns, four lanes a block of 32).  A CTA's 16 half-warps cover
// 2^cs chunks of 128 columns of 2^(4-cs) rows, and each goes on to U rows; with
// powers of two, no index is divided (64-bit divisions per item had cost more
// than the memory traffic: 59 us against 12.5 us at 8192 x 4096 bf16).
struct RowMap {
  int chunk_shift;   // cs
  int64_t chunks;    // block atoms of a row
};
template <int U>
__device__ __forceinline__ int64_t map_row(const RowMap& m, int u) {
  const int half = threadIdx.x >> 4, rows_shift = 4 - m.chunk_shift;
  return ((((int64_t)blockIdx.x * U + u) << rows_shift)) + (half >> m.chunk_shift);
}
// Matrix and row within it of flat row r (one matrix: no division).
__device__ __forceinline__ void split_row(int64_t r, int64_t rows, int64_t batch, int64_t& b,
                                          int64_t& rr) {
  b = 0;
  rr = r;
  if (batch > 1) {
    b = r / rows;
    rr = r - b * rows;
  }
}

// Rows: a half-warp writes 64 bytes of codes and one scale word per row; the U
// rows' loads are in flight together.
template <typename T, int U>
__global__ void __launch_bounds__(256) k_mx_quant_rows(const QuantArgs a, const RowMap map,
                                                       const bool vec) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const Store& st = a.st;
  const T* x = static_cast<const T*>(a.x);
  uint8_t* scales = a.q + st.scales_off;
  const int l16 = threadIdx.x & 15;
  const int64_t all_rows = a.batch * a.rows;
  const int chunk = (threadIdx.x >> 4) & ((1 << map.chunk_shift) - 1);
  for (int64_t ba = ((int64_t)blockIdx.y << map.chunk_shift) + chunk;
       ba - (chunk & 1) < map.chunks;  // the same for both halves of a warp, which shuffle together
       ba += (int64_t)gridDim.y << map.chunk_shift) {
    const int64_t col = ba * 128 + l16 * 8, blk = ba * ATOM_BLOCKS + (l16 >> 2);
    const int n = (int)(a.cols - col > 8 ? 8 : (a.cols > col ? a.cols - col : 0));
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = map_row<U>(map, u);
      int64_t b, rr;
      split_row(r, a.rows, a.batch, b, rr);
      load8<T>(x + b * a.batch_stride + rr * a.row_stride + col, r < all_rows ? n : 0, vec, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t m = max_bits8(v[u]);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t sb = scale_byte(m);
      const uint32_t code = codes8(v[u], scale_up(sb));
      // the four blocks' bytes to one word (blocks past cols hold zeros: byte 0)
      uint32_t word = sb << ((l16 >> 2) * 8);
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
      word |= __shfl_xor_sync(0xffffffffu, word, 8);
      const int64_t r = map_row<U>(map, u);
      if (r >= all_rows || ba >= map.chunks) continue;
      if (a.dest) {
        for (int d = 0; d < a.share; ++d) {
          const int64_t to = __ldg(a.dest + r * a.share + d);
          if (to < 0) continue;
          if (blk < st.blocks)
            *reinterpret_cast<uint32_t*>(a.q + to * st.pitch + blk * 16 + (l16 & 3) * 4) = code;
          if (l16 == 0) *reinterpret_cast<uint32_t*>(scales + scale_word(st, to, ba)) = word;
        }
      } else {
        int64_t b, rr;
        split_row(r, a.rows, a.batch, b, rr);
        if (blk < st.blocks)
          *reinterpret_cast<uint32_t*>(a.q + r * st.pitch + blk * 16 + (l16 & 3) * 4) = code;
        if (l16 == 0)
          *reinterpret_cast<uint32_t*>(scales + b * st.row_atoms * st.block_atoms * ATOM_BYTES +
                                       scale_word(st, rr, ba)) = word;
      }
    }
  }
}

// Transposed: x [rows, cols] to MXFP4 of x^T [cols, rows], blocks down the
// columns.  A CTA takes 128 rows x 64 columns through shared memory; four
// neighbouring lanes then take the four blocks of one column (64 contiguous
// bytes of codes and one scale word).  Each 32-row band of the staging tile is
// shifted by 8 floats, so that the four lanes' column reads fall into
// different banks.
constexpr int TC = 64, TPITCH = 65;
__device__ __forceinline__ int t_index(int r, int c) { return r * TPITCH + (r >> 5) * 8 + c; }
template <typename T>
__global__ void __launch_bounds__(256) k_mx_quant_cols(const QuantArgs a,
                                                       const bool vec) {
  __shared__ float tile[128 * TPITCH + 32];
  ptx::griddep_wait();
  ptx::griddep_launch();
  const Store st = a.st;  // of [cols, rows]
  const T* x = static_cast<const T*>(a.x);
  const int64_t tiles_r = ceil_div(a.rows, 128), tiles_c = ceil_div(a.cols, TC);
  const int64_t tiles = a.batch * tiles_r * tiles_c;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t b = t / (tiles_r * tiles_c), rem = t - b * tiles_r * tiles_c;
    const int64_t r0 = (rem / tiles_c) * 128, c0 = (rem % tiles_c) * TC;
    const T* base = x + b * a.batch_stride;
    if (vec && r0 + 128 <= a.rows && c0 + TC <= a.cols) {
      constexpr int W = 16 / (int)sizeof(T), PER_ROW = TC / W, N = 128 * PER_ROW / 256;
      uint4 u[N];  // all of a thread's 16-byte loads at once
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int at = threadIdx.x + 256 * i;
        u[i] = __ldg(reinterpret_cast<const uint4*>(base + (r0 + at / PER_ROW) * a.row_stride + c0) +
                     at % PER_ROW);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int at = threadIdx.x + 256 * i;
        T e[W];
        *reinterpret_cast<uint4*>(e) = u[i];
#pragma unroll
        for (int j = 0; j < W; ++j) tile[t_index(at / PER_ROW, at % PER_ROW * W + j)] = to_f32<T>(e[j]);
      }
    } else {
#pragma unroll 8
      for (int i = threadIdx.x; i < 128 * TC; i += 256) {
        const int r = i >> 6, c = i & 63;
        const bool in = r0 + r < a.rows && c0 + c < a.cols;
        tile[t_index(r, c)] = in ? to_f32<T>(base[(r0 + r) * a.row_stride + c0 + c]) : 0.0f;
      }
    }
    __syncthreads();
    const int c = threadIdx.x >> 2, blk = threadIdx.x & 3;
    uint32_t m = 0;
    float v[4][8];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      v[j >> 3][j & 7] = tile[t_index(blk * 32 + j, c)];
      m = max(m, __float_as_uint(v[j >> 3][j & 7]) & 0x7FFFFFFFu);
    }
    const uint32_t sb = scale_byte(m);
    const float up = scale_up(sb);
    uint32_t word = sb << (blk * 8);
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    const int64_t gblk = r0 / BLOCK + blk, row = c0 + c;
    if (row < a.cols) {
      if (gblk < st.blocks)
        *reinterpret_cast<uint4*>(a.q + (b * a.cols + row) * st.pitch + gblk * 16) =
            make_uint4(codes8(v[0], up), codes8(v[1], up), codes8(v[2], up), codes8(v[3], up));
      if (blk == 0)
        *reinterpret_cast<uint32_t*>(a.q + st.scales_off +
                                     b * st.row_atoms * st.block_atoms * ATOM_BYTES +
                                     scale_word(st, row, r0 / 128)) = word;
    }
    __syncthreads();
  }
}

// The value of one code: 0 .5 1 1.5 2 3 4 6, bit 3 the sign.
__device__ __forceinline__ float e2m1(uint32_t c) {
  const uint32_t m = c & 7u;
  // m >= 2: exponent (m >> 1) - 1, mantissa m & 1 -- an fp32 number directly
  const uint32_t bits = m >= 2u ? (((m >> 1) + 126u) << 23) | ((m & 1u) << 22)
                                : (m ? 0x3F000000u : 0u);
  return __uint_as_float(bits | ((c & 8u) << 28));
}

// The row quantiser's mapping; U rows' loads in flight together.
template <typename T, int U>
__global__ void __launch_bounds__(256) k_mx_dequant(const uint8_t* __restrict__ q, const Store st,
                                                    T* __restrict__ out, const RowMap map,
                                                    const bool vec) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int l16 = threadIdx.x & 15;
  const int64_t all_rows = st.batch * st.rows;
  for (int64_t ba = ((int64_t)blockIdx.y << map.chunk_shift) +
                    ((threadIdx.x >> 4) & ((1 << map.chunk_shift) - 1));
       ba < map.chunks; ba += (int64_t)gridDim.y << map.chunk_shift) {
    const int64_t blk = ba * ATOM_BLOCKS + (l16 >> 2), col = ba * 128 + l16 * 8;
    if (col >= st.cols) continue;
    uint32_t code[U];
    uint8_t sb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = map_row<U>(map, u);
      if (r >= all_rows) continue;
      int64_t b, rr;
      split_row(r, st.rows, st.batch, b, rr);
      code[u] = __ldg(reinterpret_cast<const uint32_t*>(q + r * st.pitch + blk * 16 + (l16 & 3) * 4));
      sb[u] = __ldg(q + st.scales_off + b * st.row_atoms * st.block_atoms * ATOM_BYTES +
                    scale_word(st, rr, ba) + (l16 >> 2));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = map_row<U>(map, u);
      if (r >= all_rows) continue;
      const float s = scale_down(sb[u]);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = e2m1(code[u] >> (4 * j)) * s;
      store8<T>(out + r * st.cols + col, (int)(st.cols - col > 8 ? 8 : st.cols - col), vec, v);
    }
  }
}

// Grid of the row kernels: chunks of 128 columns on y, rows on x, U rows per
// half-warp when that still leaves four CTAs for every SM.
struct RowGrid {
  RowMap map;
  dim3 grid;
  bool many;  // U == 4
};
RowGrid row_grid(int64_t rows, int64_t chunks) {
  RowGrid g;
  g.map.chunks = chunks;
  g.map.chunk_shift = 0;
  while (g.map.chunk_shift < 4 && (1 << g.map.chunk_shift) < chunks) ++g.map.chunk_shift;
  const int64_t y = ceil_div(chunks, 1 << g.map.chunk_shift);
  const int64_t per = 1 << (4 - g.map.chunk_shift);  // rows of a CTA at U == 1
  g.many = ceil_div(rows, per * 4) * y >= 4 * (int64_t)device_sm_count();
  g.grid = dim3((unsigned)ceil_div(rows, per * (g.many ? 4 : 1)), (unsigned)(y < 65535 ? y : 65535));
  return g;
}

template <typename T>
cudaError_t quantize(const QuantArgs& a, bool transpose, cudaStream_t s) {
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 &&
                   (a.row_stride * (int64_t)sizeof(T)) % 16 == 0 &&
                   (a.batch_stride * (int64_t)sizeof(T)) % 16 == 0;
  cudaError_t e;
  if (transpose) {
    const int64_t tiles = a.batch * ceil_div(a.rows, 128) * ceil_div(a.cols, TC);
    const int64_t cap = (int64_t)device_sm_count() * 6;
    e = launch_after_previous(k_mx_quant_cols<T>, dim3((unsigned)(tiles < cap ? tiles : cap)),
                              dim3(256), 0, s, a, vec);
  } else {
    const RowGrid g = row_grid(a.batch * a.rows, a.st.block_atoms);
    e = launch_after_previous(g.many ? k_mx_quant_rows<T, 4> : k_mx_quant_rows<T, 1>, g.grid,
                              dim3(256), 0, s, a, g.map, vec);
  }
  note_launch();
  return e;
}

template <typename T>
cudaError_t dequantize(const uint8_t* q, const Store& st, void* out, cudaStream_t s) {
  const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0 &&
                   (st.cols * (int64_t)sizeof(T)) % 16 == 0;
  const RowGrid g = row_grid(st.batch * st.rows, st.block_atoms);
  const cudaError_t e =
      launch_after_previous(g.many ? k_mx_dequant<T, 4> : k_mx_dequant<T, 1>, g.grid, dim3(256), 0,
                            s, q, st, static_cast<T*>(out), g.map, vec);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_quantize(const QuantArgs& a, int dtype, bool transpose, cudaStream_t s) {
  note_kernel_name(transpose ? "k_mx_quant_cols" : "k_mx_quant_rows");
  if (dtype == IMC_F32) return quantize<float>(a, transpose, s);
  if (dtype == IMC_F16) return quantize<__half>(a, transpose, s);
  return quantize<__nv_bfloat16>(a, transpose, s);
}

cudaError_t launch_dequantize(const uint8_t* q, const Store& st, int dtype, void* out,
                              cudaStream_t s) {
  note_kernel_name("k_mx_dequant");
  if (dtype == IMC_F32) return dequantize<float>(q, st, out, s);
  if (dtype == IMC_F16) return dequantize<__half>(q, st, out, s);
  return dequantize<__nv_bfloat16>(q, st, out, s);
}

}  // namespace mx
}  // namespace imc
