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

// Rows: 16 lanes take 128 columns of one row (a lane 8 columns, four lanes a
// block), so a half-warp writes 64 bytes of codes and one scale word.  U such
// items per half-warp are loaded before any is used.
template <typename T, int U>
__global__ void __launch_bounds__(256) k_mx_quant_rows(const QuantArgs a, const bool vec) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const Store st = a.st;
  const T* x = static_cast<const T*>(a.x);
  const int l16 = threadIdx.x & 15;
  const int64_t halves = (int64_t)gridDim.x * (blockDim.x >> 4);
  const int64_t half = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 4;
  const int64_t per_row = st.block_atoms, items = a.batch * a.rows * per_row;
  for (int64_t i0 = half - (half & 1); i0 < items; i0 += halves * U) {  // warp-uniform bound
    float v[U][8];
    int64_t row[U], ba[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + (half & 1) + u * halves;
      row[u] = i < items ? i / per_row : -1;
      ba[u] = i - row[u] * per_row;
      const int64_t col = ba[u] * 128 + l16 * 8;
      const int64_t left = row[u] >= 0 ? a.cols - col : 0;
      const int64_t b = row[u] >= 0 ? row[u] / a.rows : 0;
      const T* p = x + b * a.batch_stride + (row[u] - b * a.rows) * a.row_stride + col;
      load8<T>(p, (int)(left > 8 ? 8 : left), vec, v[u]);
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
      if (row[u] < 0) continue;
      const int64_t blk = ba[u] * ATOM_BLOCKS + (l16 >> 2);
      uint8_t* scales = a.q + st.scales_off;
      if (a.dest) {
        for (int d = 0; d < a.share; ++d) {
          const int64_t r = a.dest[row[u] * a.share + d];
          if (r < 0) continue;
          if (blk < st.blocks)
            *reinterpret_cast<uint32_t*>(a.q + r * st.pitch + blk * 16 + (l16 & 3) * 4) = code;
          if (l16 == 0)
            *reinterpret_cast<uint32_t*>(scales + scale_word(st, r, ba[u])) = word;
        }
      } else {
        const int64_t b = row[u] / a.rows, r = row[u] - b * a.rows;
        if (blk < st.blocks)
          *reinterpret_cast<uint32_t*>(a.q + row[u] * st.pitch + blk * 16 + (l16 & 3) * 4) = code;
        if (l16 == 0)
          *reinterpret_cast<uint32_t*>(scales + b * st.row_atoms * st.block_atoms * ATOM_BYTES +
                                       scale_word(st, r, ba[u])) = word;
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
__global__ void __launch_bounds__(256) k_mx_quant_cols(const QuantArgs a) {
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
#pragma unroll 8
    for (int i = threadIdx.x; i < 128 * TC; i += 256) {
      const int r = i >> 6, c = i & 63;
      const bool in = r0 + r < a.rows && c0 + c < a.cols;
      tile[t_index(r, c)] = in ? to_f32<T>(base[(r0 + r) * a.row_stride + c0 + c]) : 0.0f;
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

// 16 lanes take 128 columns of a row, as in the row quantiser.
template <typename T>
__global__ void __launch_bounds__(256) k_mx_dequant(const uint8_t* __restrict__ q, const Store st,
                                                    T* __restrict__ out, const bool vec) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int l16 = threadIdx.x & 15;
  const int64_t halves = (int64_t)gridDim.x * (blockDim.x >> 4);
  const int64_t per_row = st.block_atoms, items = st.batch * st.rows * per_row;
  for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 4; i < items; i += halves) {
    const int64_t row = i / per_row, ba = i - row * per_row;
    const int64_t blk = ba * ATOM_BLOCKS + (l16 >> 2), col = ba * 128 + l16 * 8;
    if (blk >= st.blocks || col >= st.cols) continue;
    const int64_t b = row / st.rows, r = row - b * st.rows;
    const uint32_t code =
        __ldg(reinterpret_cast<const uint32_t*>(q + row * st.pitch + blk * 16 + (l16 & 3) * 4));
    const float s = scale_down(q[st.scales_off + b * st.row_atoms * st.block_atoms * ATOM_BYTES +
                                 scale_word(st, r, ba) + (l16 >> 2)]);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e2m1(code >> (4 * j)) * s;
    const int64_t left = st.cols - col;
    store8<T>(out + row * st.cols + col, (int)(left > 8 ? 8 : left), vec, v);
  }
}

template <typename T>
cudaError_t quantize(const QuantArgs& a, bool transpose, cudaStream_t s) {
  const int64_t sms = device_sm_count();
  cudaError_t e;
  if (transpose) {
    const int64_t tiles = a.batch * ceil_div(a.rows, 128) * ceil_div(a.cols, TC);
    const int64_t cap = sms * 6;
    e = launch_after_previous(k_mx_quant_cols<T>, dim3((unsigned)(tiles < cap ? tiles : cap)),
                              dim3(256), 0, s, a);
  } else {
    const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 &&
                     (a.row_stride * (int64_t)sizeof(T)) % 16 == 0 &&
                     (a.batch_stride * (int64_t)sizeof(T)) % 16 == 0;
    const int64_t items = a.batch * a.rows * a.st.block_atoms;  // half-warps
    const int64_t blocks = ceil_div(items, 16), cap = sms * 8;
    if (blocks > cap)
      e = launch_after_previous(k_mx_quant_rows<T, 4>, dim3((unsigned)cap), dim3(256), 0, s, a, vec);
    else
      e = launch_after_previous(k_mx_quant_rows<T, 1>, dim3((unsigned)blocks), dim3(256), 0, s, a,
                                vec);
  }
  note_launch();
  return e;
}

template <typename T>
cudaError_t dequantize(const uint8_t* q, const Store& st, void* out, cudaStream_t s) {
  const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0 &&
                   (st.cols * (int64_t)sizeof(T)) % 16 == 0;
  const int64_t blocks = ceil_div(st.batch * st.rows * st.block_atoms, 16);
  const int64_t cap = (int64_t)device_sm_count() * 8;
  const cudaError_t e =
      launch_after_previous(k_mx_dequant<T>, dim3((unsigned)(blocks < cap ? blocks : cap)),
                            dim3(256), 0, s, q, st, static_cast<T*>(out), vec);
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
