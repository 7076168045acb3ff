// Internal declarations of the microscaled 4-bit (MXFP4) and expert-routing
// operators: argument structs shared by the C entry points (mx_api.cu) and the
// kernel files, the storage layout of an MXFP4 matrix, and element conversion.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "imc.h"
#include "imc_internal.cuh"

namespace imc {
namespace mx {

constexpr int BLOCK = 32;        // values that share one scale
constexpr int ATOM_ROWS = 128;   // rows of one scale atom
constexpr int ATOM_BLOCKS = 4;   // blocks of K of one scale atom (128 values)
constexpr int ATOM_BYTES = ATOM_ROWS * ATOM_BLOCKS;

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Storage of `batch` matrices [rows, cols] in MXFP4, one device buffer:
//   codes   [batch][rows][pitch] bytes, two codes a byte (even column in the
//           low half), pitch = 16 * ceil(cols / 32); the codes past cols are 0
//   scales  from a 512-byte boundary on, one byte 127 + e per block of 32, in
//           atoms of 128 rows x 4 blocks: [batch][row atom][block atom][512],
//           the byte of row r, block b of an atom at (r % 32)*16 + (r / 32)*4 + b.
// This is the order in which tcgen05.cp moves scales to tensor memory, so a
// tile's scales are one contiguous copy.  The scales of blocks past cols are
// 0; those of rows past `rows` are not written and no result depends on them
// (a row's scale enters that row's products only).
// Within a call the tokens' scales may be kept with fewer rows per atom (the rest
// of the atom unused): the MMA reads scales from a TMEM column that is a multiple
// of four, so every tile of tokens has to begin at an atom.  atom_shift is log2 of
// an atom's rows (7; less for the sorted rows of the experts' product, whose tiles
// may be lower than 128 rows), or TILES_224: tiles of 224 rows, 128 in one atom
// and 96 in the next.
constexpr int TILES_224 = 0;
struct Store {
  int64_t batch, rows, cols, blocks, pitch, row_atoms, block_atoms, codes_bytes, scales_off, bytes;
  int atom_shift;
};
__host__ __device__ inline Store store_of(int64_t batch, int64_t rows, int64_t cols,
                                          int atom_shift = 7) {
  Store s;
  s.atom_shift = atom_shift;
  s.batch = batch;
  s.rows = rows;
  s.cols = cols;
  s.blocks = ceil_div(cols, BLOCK);
  s.pitch = s.blocks * 16;
  s.row_atoms = atom_shift == TILES_224 ? 2 * ceil_div(rows, 224)
                                        : (rows + (1 << atom_shift) - 1) >> atom_shift;
  s.block_atoms = ceil_div(s.blocks, ATOM_BLOCKS);
  s.codes_bytes = batch * rows * s.pitch;
  s.scales_off = ceil_div(s.codes_bytes, 512) * 512;
  s.bytes = s.scales_off + batch * s.row_atoms * s.block_atoms * ATOM_BYTES;
  return s;
}
// Byte offset, within one matrix's scales, of the 4-byte word of row r and
// block atom ba.
__device__ __forceinline__ int64_t scale_word(const Store& st, int64_t r, int64_t ba) {
  int64_t atom = r >> st.atom_shift;
  int rr = (int)r & ((1 << st.atom_shift) - 1);
  if (st.atom_shift == TILES_224) {
    const uint32_t tile = (uint32_t)r / 224u, in = (uint32_t)r - tile * 224u;
    atom = 2 * (int64_t)tile + (in >> 7);
    rr = (int)(in & 127u);
  }
  return (atom * st.block_atoms + ba) * ATOM_BYTES + (rr & 31) * 16 + (rr >> 5) * 4;
}

struct QuantArgs {
  const void* x;          // [batch][rows][cols], rows row_stride elements apart
  int64_t batch, rows, cols, batch_stride, row_stride;
  uint8_t* q;             // Store of the result
  Store st;               // its layout (transposed: of [cols, rows])
  const int32_t* dest;    // rows of the result that row r is written to: dest[r*share ..), or null
  int share;
  uint8_t* q_rows;        // transposed: MXFP4 of x itself as well, or null
  Store st_rows;          // its layout
  // transposed, rows in expert order: row r of the `rows` padded ones is row
  // order[...] / share of x, or zeros (layout of moe_layout; null: x's own rows)
  const int32_t *offsets, *starts, *order;
  int E;
};

// One product: out[token, n] = sum_k x[token, k] * w[n, k] (+ bias[n]) (ReLU).
struct ProductArgs {
  const uint8_t* x;       // MXFP4 [x_rows, K]
  int x_shift;            // atom_shift of its scales (dense form)
  const uint8_t* w;       // MXFP4 [E][N, K]
  const float* bias;      // [E][N] or null
  void* out;              // [tokens or slots][N]
  int out_dtype, relu;
  int64_t M, N, K, x_rows;
  // experts' form (null / 0 for one dense product)
  int E;
  const int32_t *offsets, *starts, *order;
  int slots;              // T * k
  // weights' gradient: both operands lie along the sorted rows, out is [E][M][N]
  // and its part e sums over rows starts[e] .. starts[e + 1]
  bool groups;
  bool inputs_ready;      // a pre-pass of this call has waited for earlier kernels
  // few tokens: unquantised x instead of p.x (product_fused)
  const void* raw;        // row of token m, or of slot s: raw + (m or s / share) * raw_stride
  int raw_dtype, share;
  int64_t raw_stride;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Eight values of a row as floats: 16-byte loads when `vec` (the address is
// 16-byte aligned and n >= 8), else element by element; zeros past n.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool vec, float (&v)[8]) {
  if (vec && n >= 8) {
    constexpr int W = 16 / (int)sizeof(T);  // elements per 16 bytes
#pragma unroll
    for (int j = 0; j < 8 / W; ++j) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + j);
      alignas(16) T t[W];
      *reinterpret_cast<uint4*>(t) = u;
#pragma unroll
      for (int i = 0; i < W; ++i) v[j * W + i] = to_f32<T>(t[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32<T>(p[i]) : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int n, bool vec, const float (&v)[8]) {
  if (vec && n >= 8) {
    constexpr int W = 16 / (int)sizeof(T);
#pragma unroll
    for (int j = 0; j < 8 / W; ++j) {
      alignas(16) T t[W];
#pragma unroll
      for (int i = 0; i < W; ++i) t[i] = from_f32<T>(v[j * W + i]);
      reinterpret_cast<uint4*>(p)[j] = *reinterpret_cast<const uint4*>(t);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

inline int dtype_bytes(int dtype) { return dtype == IMC_F32 ? 4 : 2; }

cudaError_t launch_quantize(const QuantArgs& a, int dtype, bool transpose, cudaStream_t s);
// a and b along their columns, in one launch.
cudaError_t launch_quantize_two(const QuantArgs& a, const QuantArgs& b, int dtype, cudaStream_t s);
cudaError_t launch_dequantize(const uint8_t* q, const Store& st, int dtype, void* out,
                              cudaStream_t s);
bool product_supported();
// Whether the product quantises its tokens itself (args.raw) instead of reading
// quantised ones: few tokens, or few slots per expert.
bool product_fused(int64_t tokens);
bool experts_fused(int64_t slots, int64_t E);
// The atom_shift that the dense product of M x N x K wants of tokens that are
// quantised for it (7: the general layout).
int product_atom_shift(int64_t M, int64_t N, int64_t K);
// The atom_shift of the experts' sorted rows: log2 of the token rows of a tile
// (at most 7), or TILES_224.
int experts_atom_shift(int64_t slots, int64_t E);
// Rows that a matrix with these scale atoms has for `rows` sorted rows, whose runs
// start at multiples of 128: in tiles of 224 every 128 rows have a tile of their own.
__host__ __device__ constexpr int64_t sorted_at(int64_t rows, int atom_shift) {
  return atom_shift == TILES_224 ? rows / ATOM_ROWS * 224 : rows;
}
cudaError_t launch_product(const ProductArgs& a, cudaStream_t s);
cudaError_t product_take_watchdog(int* value);

struct RouteArgs {
  const void* logits;
  int64_t T, ld;
  int E, k, groups, top_groups, sigmoid, renorm;
  int size;               // experts of a group, and 2^20 / size rounded up
  uint32_t inv_size;
  float scale;
  const float* bias;      // [E] or null
  float* weights;         // [T,k]
  int32_t* experts;       // [T,k]
};
cudaError_t launch_route(const RouteArgs& a, int dtype, cudaStream_t s);
// grad_logits [T,E] of the weights' gradient g [T,k] (a.experts is an input).
cudaError_t launch_route_backward(const RouteArgs& a, int dtype, const float* g, void* grad_logits,
                                  cudaStream_t s);
// `counts`: scratch of layout_ctas(n) * (E + 1) words when that is more than
// one CTA.
constexpr int kLayoutMaxCtas = 128;
int layout_ctas(int64_t n);
cudaError_t launch_layout(const int32_t* experts, int n, int E, int32_t* offsets, int32_t* starts,
                          int32_t* order, int32_t* dest, int32_t* dest224, int32_t* counts,
                          cudaStream_t s);
// out_dtype: dtype, or any type for fp32 y.
cudaError_t launch_combine(const void* y, const float* w, int dtype, int64_t T, int k, int64_t N,
                           void* out, int out_dtype, cudaStream_t s);
cudaError_t launch_combine_backward(const void* grad, const void* y, const float* w, int dtype,
                                    int64_t T, int k, int64_t N, void* grad_y, float* grad_w,
                                    cudaStream_t s);

}  // namespace mx
}  // namespace imc
