// Quantisation to MXFP4 and back.
//
// A block of 32 consecutive values of a row shares the scale 2^e,
// e = clamp(floor(log2(max |x|)) - 2, -127, 127), so that the largest magnitude
// lands in [4, 8), and each value becomes the E2M1 number nearest to x * 2^-e
// (ties to the even code, magnitudes above 6 become 6).  floor(log2) is the
// exponent field of the fp32 maximum and 2^-e a float built from it, so every
// step but the final rounding is exact.  A block that holds an infinity or a
// NaN gets the scale byte 255 (NaN): it stands for 32 NaNs, whatever its codes.
#include "mx_internal.cuh"
#include "mx_quant.cuh"
#include "ptx.cuh"

namespace imc {
namespace mx {
namespace {

// Which rows and columns a lane takes: 8 lanes cover 128 columns of a row (a
// lane 16 columns, two lanes a block of 32).  A CTA's 32 such groups cover 2^cs
// chunks of 128 columns of 2^(5-cs) rows, and each goes on to U rows, rows_step
// apart; with powers of two, no index is divided (with 64-bit divisions per 8
// values, 8192 x 4096 bf16 took 59 us, with 8 values a lane 34 us, against 12.5
// us of memory traffic: both bound by instructions).
struct RowMap {
  int chunk_shift;   // cs
  int64_t chunks;    // block atoms of a row
};
constexpr int GROUPS_SHIFT = 5;  // log2 of a CTA's groups of 8 lanes

// Rows: a group of 8 lanes writes 64 bytes of codes and one scale word per row.
// 8192 x 4096: fp32 24.4 us (22.4 of memory traffic), bf16 17.1 (12.5).  Four rows a
// group changed nothing at 16 bits; CTAs that stay and load U rows ahead took 30 and
// 24 us (fewer of them fit, and they drift apart in memory).
// SORTED: row r goes to the rows dest[r * share ..) of the result (4096 x 2048 bf16 to
// eight places each 13.2 us, 15 with one lane for all scale words).
template <typename T, int U, bool SORTED>
__global__ void __launch_bounds__(256) k_mx_quant_rows(const QuantArgs a, const RowMap map,
                                                       const int vec) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const Store& st = a.st;
  uint8_t* scales = a.q + st.scales_off;
  const int l8 = threadIdx.x & 7, group = threadIdx.x >> 3, cs = map.chunk_shift;
  const int64_t all_rows = a.batch * a.rows, step = 1 << (GROUPS_SHIFT - cs);
  const int64_t row0 = (int64_t)blockIdx.x * (step * U) + (group >> cs);
  const int chunk = group & ((1 << cs) - 1);
  for (int64_t y = blockIdx.y; (y << cs) < map.chunks; y += gridDim.y) {  // the same for the CTA
    const int64_t ba = (y << cs) + chunk, col = ba * 128 + l8 * 16;
    const int n = (int)(a.cols - col > 16 ? 16 : (a.cols > col ? a.cols - col : 0));
    const T* x = static_cast<const T*>(a.x) + row0 * a.row_stride + col;
    Raw16<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = row0 + u * step;
      const T* p = x + u * (step * a.row_stride);
      if (a.batch > 1 && r < all_rows) {  // matrices need not be row_stride * rows apart
        const int64_t b = r / a.rows;
        p = static_cast<const T*>(a.x) + b * a.batch_stride + (r - b * a.rows) * a.row_stride + col;
      }
      raw[u].load(p, r < all_rows ? n : 0, vec);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint2 code;
      uint32_t word;  // blocks past cols hold zeros: byte 0
      quantize_128(raw[u], code, word);
      const int64_t r = row0 + u * step, blk = ba * ATOM_BLOCKS + (l8 >> 1);
      if (r >= all_rows || ba >= map.chunks) continue;
      uint8_t* codes = a.q + blk * 16 + (l8 & 1) * 8;
      if constexpr (SORTED) {
        // each of the eight lanes reads one place and writes the scale word there
        const uint32_t eight = 0xFFu << (threadIdx.x & 24);
        for (int d0 = 0; d0 < a.share; d0 += 8) {
          const int mine = d0 + l8 < a.share ? __ldg(a.dest + r * a.share + d0 + l8) : -1;
          if (mine >= 0) *reinterpret_cast<uint32_t*>(scales + scale_word(st, mine, ba)) = word;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            if (d0 + d >= a.share) break;
            const int to = __shfl_sync(eight, mine, d, 8);
            if (to >= 0 && blk < st.blocks)
              *reinterpret_cast<uint2*>(codes + (int64_t)to * st.pitch) = code;
          }
        }
      } else {
        if (blk < st.blocks) *reinterpret_cast<uint2*>(codes + r * st.pitch) = code;
        if (l8 == 0) {
          int64_t rr = r;
          uint8_t* sc = scales;
          if (a.batch > 1) {
            const int64_t b = r / a.rows;
            rr = r - b * a.rows;
            sc += b * st.row_atoms * st.block_atoms * ATOM_BYTES;
          }
          *reinterpret_cast<uint32_t*>(sc + scale_word(st, rr, ba)) = word;
        }
      }
    }
  }
}

// Transposed: x [rows, cols] to MXFP4 of x^T [cols, rows], blocks down the
// columns.  A lane takes one column (two neighbouring ones of 16-bit values) and
// NB blocks of 32 rows of it: a warp's loads are whole 128-byte row pieces, a
// block never leaves its lane's registers until it is codes (with x staged in
// shared memory, 8192 x 4096 bf16 took 24 us).
template <typename T>
struct ColTile {
  static constexpr int PER = 4 / (int)sizeof(T);  // columns of a lane
  static constexpr int COLS = 32 * PER, CTA_COLS = 8 * COLS;
};

// The codes of 128 rows in a warp's columns, a lane's column being first + lane * by:
// exchanged within the warp, so that four neighbouring lanes write one column's 64
// bytes; a lane alone writes half a sector at a time (8192 x 4096, us: fp32 27.3 / 28.0,
// bf16 17.6 / 19.3).
__device__ __forceinline__ void store_columns(uint4 (&buf)[128], const uint4 (&code)[4], uint8_t* to,
                                              int64_t pitch, int by, int64_t cols, int64_t blocks) {
  const int lane = threadIdx.x & 31, i = lane & 3;
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) buf[lane * 4 + (k ^ ((lane >> 1) & 3))] = code[k];
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = 8 * k + (lane >> 2);
    const uint4 v = buf[c * 4 + (i ^ ((c >> 1) & 3))];
    if (c * by < cols && i < blocks) *reinterpret_cast<uint4*>(to + c * by * pitch + i * 16) = v;
  }
}

// GATHER (NB == 4): the rows are slots in expert order, every expert's run padded
// to a multiple of 128, so that a lane's 128 rows belong to one expert.
// The CTA takes the tiles first, first + step, ...
template <typename T, int NB, bool GATHER>
__device__ __forceinline__ void quant_columns(const QuantArgs& a, const bool words, int64_t first_tile,
                                              int64_t step) {
  static_assert(!GATHER || NB == 4, "one expert's rows");
  using C = ColTile<T>;
  constexpr int PER = C::PER;
  const Store& st = a.st;  // of [cols, rows]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ uint4 buf[NB == 4 ? 8 : 1][128];
  // row tiles cover whole scale atoms: the bytes past the last row are 0
  const int64_t tiles_r = ceil_div(a.rows, 128) * (4 / NB), tiles_c = ceil_div(a.cols, C::CTA_COLS);
  const int64_t tiles = a.batch * tiles_r * tiles_c;
  for (int64_t t = first_tile; t < tiles; t += step) {
    const int64_t b = t / (tiles_r * tiles_c), rem = t - b * tiles_r * tiles_c;
    const int64_t r0 = rem / tiles_c * (32 * NB), cta_c0 = rem % tiles_c * C::CTA_COLS;
    const T* base = static_cast<const T*>(a.x) + b * a.batch_stride;
    const int64_t c = cta_c0 + warp * C::COLS + lane * PER;
    const int64_t atoms = b * st.row_atoms * st.block_atoms * ATOM_BYTES;
    uint32_t word[PER] = {};
    uint4 code[PER][NB];
    int64_t first = 0, last = 0;  // GATHER: places in `order` of row r0, and past the expert's end
    if (GATHER) {
      if (r0 >= a.starts[a.E]) continue;  // rows of no expert
      int lo = 0, hi = a.E - 1;           // the last expert whose run begins at or before r0
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.starts[mid] <= r0) lo = mid;
        else hi = mid - 1;
      }
      first = a.offsets[lo] + r0 - a.starts[lo];
      last = a.offsets[lo + 1];
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int64_t r = r0 + nb * 32;
      const T* p = base + r * a.row_stride + c;
      uint32_t u[32];
      if (GATHER) {
        const int64_t at = first + nb * 32 + lane;
        const int src = at < last ? a.order[at] / a.share : -1;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int row = __shfl_sync(0xffffffffu, src, j);
          const T* q = base + (int64_t)row * a.row_stride + c;
          if (words && row >= 0 && c + PER <= a.cols) {
            u[j] = __ldg(reinterpret_cast<const uint32_t*>(q));
          } else {
            alignas(4) T e[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i)
              e[i] = row >= 0 && c + i < a.cols ? q[i] : from_f32<T>(0.0f);
            u[j] = *reinterpret_cast<const uint32_t*>(e);
          }
        }
      } else if (words && c + PER <= a.cols && r + 32 <= a.rows) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          u[j] = __ldg(reinterpret_cast<const uint32_t*>(p + j * a.row_stride));
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          alignas(4) T e[PER];
#pragma unroll
          for (int i = 0; i < PER; ++i)
            e[i] = r + j < a.rows && c + i < a.cols ? p[j * a.row_stride + i] : from_f32<T>(0.0f);
          u[j] = *reinterpret_cast<const uint32_t*>(e);
        }
      }
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        m = PER == 1 ? max(m, u[j] & 0x7FFFFFFFu) : __vmaxu2(m, u[j] & 0x7FFF7FFFu);
      uint32_t sb[PER];
      float up[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        sb[i] = scale_byte(PER == 1 ? m : Raw16<T>::top16(i ? m >> 16 : m & 0xFFFFu));
        up[i] = scale_up(sb[i]);
      }
      if constexpr (Raw16<T>::PAIRS) {
        const uint32_t both = Raw16<T>::pair_of(up[0], up[PER - 1]);
#pragma unroll
        for (int j = 0; j < 32; ++j) u[j] = Raw16<T>::times(u[j], both);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (PER == 1) {
              v[j] = __uint_as_float(u[8 * k + j]);
            } else {
              const float2 f = Raw16<T>::two(u[8 * k + j]);
              v[j] = i ? f.y : f.x;
            }
          }
          w[k] = codes8(v, Raw16<T>::PAIRS ? 1.0f : up[i]);
        }
        code[i][nb] = make_uint4(w[0], w[1], w[2], w[3]);
        word[i] |= sb[i] << (8 * nb);
      }
    }
    const int64_t blk = r0 / BLOCK;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if constexpr (NB == 4) {
        const int64_t cw = c - lane * PER + i;
        store_columns(buf[warp], code[i], a.q + (b * a.cols + cw) * st.pitch + blk * 16, st.pitch, PER,
                      a.cols - cw, st.blocks - blk);
      }
      if (c + i >= a.cols) continue;
      if (NB != 4) {
        uint8_t* to = a.q + (b * a.cols + c + i) * st.pitch + blk * 16;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          if (blk + nb < st.blocks) *reinterpret_cast<uint4*>(to + nb * 16) = code[i][nb];
      }
      uint8_t* sc = a.q + st.scales_off + atoms + scale_word(st, c + i, blk / ATOM_BLOCKS);
      if (NB == 4) *reinterpret_cast<uint32_t*>(sc) = word[i];
      else
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) sc[blk % ATOM_BLOCKS + nb] = (uint8_t)(word[i] >> (8 * nb));
    }
  }
}

template <typename T, int NB, bool GATHER>
__global__ void __launch_bounds__(256) k_mx_quant_cols(const QuantArgs a, const bool words) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  quant_columns<T, NB, GATHER>(a, words, blockIdx.x, gridDim.x);
}
// Two matrices in one launch, the first on the first `ctas` CTAs: the gradients'
// call takes 2 us less than with a launch for each (dy 8192 x 1024, K 512, fp32:
// 33.6 / 35.7).
template <typename T, int NB>
__global__ void __launch_bounds__(256)
    k_mx_quant_two(const QuantArgs a, const bool words_a, const QuantArgs b, const bool words_b,
                   const int ctas) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  if ((int)blockIdx.x < ctas) quant_columns<T, NB, false>(a, words_a, blockIdx.x, ctas);
  else quant_columns<T, NB, false>(b, words_b, blockIdx.x - ctas, gridDim.x - ctas);
}

// x along its columns (as above) and along its rows, read once.  A CTA takes 128
// rows x 128 columns in two bands of 64 rows: eight lanes hold a row's 128 values,
// 16 each, and quantise it from their registers (one scale word, 64 contiguous
// bytes of codes); the band also goes to shared memory, where a thread then reads a
// column's block of 32.  The 16-byte chunks of a row are permuted by bits 3-4 of
// their index, so that the writes (eight lanes, every fourth chunk) fall into
// different banks like the reads.  At 8192 x 4096 fp32 34 us (25 of memory traffic;
// 32 warps an SM, each waiting for its loads); with the rows' blocks read back from
// shared memory too 39, with four bands of 32 rows and the next one's loads in flight
// at 16 warps an SM 38, the two kernels apart 52.
constexpr int BOTH = 128;  // columns of a tile
__device__ __forceinline__ int chunk_at(int ch) { return ch ^ ((ch >> 3) & 3); }
template <typename T>
__global__ void __launch_bounds__(256, 4) k_mx_quant_both(const QuantArgs a, const int vec) {
  __shared__ __align__(16) float buf[64 * BOTH];
  __shared__ uint4 out[4 * BOTH];
  __shared__ __align__(4) uint8_t bytes[4 * BOTH];
  ptx::griddep_wait();
  ptx::griddep_launch();
  const Store &st = a.st, &sr = a.st_rows;  // of [cols, rows] and of [rows, cols]
  const int64_t tiles_r = ceil_div(a.rows, 128), tiles_c = ceil_div(a.cols, BOTH);
  const int64_t t = blockIdx.x, b = t / (tiles_r * tiles_c), rem = t - b * tiles_r * tiles_c;
  const int64_t r0 = (rem / tiles_c) * 128, c0 = (rem % tiles_c) * BOTH;
  const int j = threadIdx.x & 7, r = threadIdx.x >> 3, c = threadIdx.x & 127, half = threadIdx.x >> 7;
  const int column = chunk_at(c >> 2) * 4 + (c & 3);
  const T* x = static_cast<const T*>(a.x) + b * a.batch_stride;
  const int64_t left = a.cols - c0 - 16 * j;
  const int n = left < 16 ? (left > 0 ? (int)left : 0) : 16;
  Raw16<T> raw[2];
  auto fetch = [&](int band) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = r0 + band * 64 + h * 32 + r;
      raw[h].load(x + row * a.row_stride + c0 + 16 * j, row < a.rows ? n : 0, vec);
    }
  };
  fetch(0);
  uint4 code[2];
  uint32_t byte[2];
#pragma unroll
  for (int band = 0; band < 2; ++band) {
    if (band) {
      fetch(1);
      __syncthreads();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint2 cr;
      uint32_t wr;
      quantize_128(raw[h], cr, wr);
      const int64_t row = r0 + band * 64 + h * 32 + r, blk = c0 / BLOCK + (j >> 1);
      if (row < a.rows) {
        if (blk < sr.blocks)
          *reinterpret_cast<uint2*>(a.q_rows + (b * a.rows + row) * sr.pitch + blk * 16 +
                                    (j & 1) * 8) = cr;
        if (j == 0)
          *reinterpret_cast<uint32_t*>(a.q_rows + sr.scales_off +
                                       b * sr.row_atoms * sr.block_atoms * ATOM_BYTES +
                                       scale_word(sr, row, c0 / 128)) = wr;
      }
      float v[16];
      raw[h].widen(v);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(buf + (h * 32 + r) * BOTH + chunk_at(4 * j + i) * 4) =
            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
    __syncthreads();
    float v[4][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      v[i >> 3][i & 7] = buf[(half * 32 + i) * BOTH + column];
      m = max(m, __float_as_uint(v[i >> 3][i & 7]) & 0x7FFFFFFFu);
    }
    byte[band] = scale_byte(m);
    const float up = scale_up(byte[band]);
    code[band] = make_uint4(codes8(v[0], up), codes8(v[1], up), codes8(v[2], up), codes8(v[3], up));
  }
  // Four neighbouring lanes write a column's 64 bytes (a lane alone would write half
  // a sector at a time).
#pragma unroll
  for (int band = 0; band < 2; ++band) {
    const int i = 2 * band + half;
    out[c * 4 + (i ^ ((c >> 1) & 3))] = code[band];
    bytes[c * 4 + i] = (uint8_t)byte[band];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int cc = k * 64 + (threadIdx.x >> 2), i = threadIdx.x & 3;
    const uint4 v = out[cc * 4 + (i ^ ((cc >> 1) & 3))];
    if (c0 + cc < a.cols && r0 / BLOCK + i < st.blocks)
      *reinterpret_cast<uint4*>(a.q + (b * a.cols + c0 + cc) * st.pitch + (r0 / BLOCK + i) * 16) = v;
  }
  if (half == 0 && c0 + c < a.cols)
    *reinterpret_cast<uint32_t*>(a.q + st.scales_off + b * st.row_atoms * st.block_atoms * ATOM_BYTES +
                                 scale_word(st, c0 + c, r0 / 128)) =
        reinterpret_cast<const uint32_t*>(bytes)[c];
}

// The values of eight codes, the first in the lowest four bits.
__device__ __forceinline__ void values8(uint32_t codes, float scale, float (&v)[8]) {
  uint32_t h[4];  // pairs of fp16, which holds every E2M1 value
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    v[2 * j] = f.x * scale;
    v[2 * j + 1] = f.y * scale;
  }
}

// As the row quantiser, with 16 lanes for 128 columns (8 values a lane: with 16
// the stores of a warp are too far apart, 39 against 29 us at 8192 x 4096 to
// fp32).
template <typename T, int U>
__global__ void __launch_bounds__(256) k_mx_dequant(const uint8_t* __restrict__ q, const Store st,
                                                    T* __restrict__ out, const RowMap map,
                                                    const bool vec, const bool wide) {
  ptx::griddep_wait();
  ptx::griddep_launch();
  const int l16 = threadIdx.x & 15, group = threadIdx.x >> 4, cs = map.chunk_shift;
  const int64_t all_rows = st.batch * st.rows, step = 1 << (4 - cs);
  const int64_t row0 = (int64_t)blockIdx.x * (step * U) + (group >> cs);
  const int chunk = group & ((1 << cs) - 1);
  for (int64_t y = blockIdx.y; (y << cs) < map.chunks; y += gridDim.y) {
    const int64_t ba = (y << cs) + chunk, col = ba * 128 + l16 * 8;
    const int64_t blk = ba * ATOM_BLOCKS + (l16 >> 2);
    if (col >= st.cols) continue;
    uint32_t code[U];
    uint8_t sb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = row0 + u * step;
      if (r >= all_rows) continue;
      int64_t rr = r;
      const uint8_t* sc = q + st.scales_off;
      if (st.batch > 1) {
        const int64_t b = r / st.rows;
        rr = r - b * st.rows;
        sc += b * st.row_atoms * st.block_atoms * ATOM_BYTES;
      }
      code[u] = __ldg(reinterpret_cast<const uint32_t*>(q + r * st.pitch + blk * 16 + (l16 & 3) * 4));
      sb[u] = __ldg(sc + scale_word(st, rr, ba) + (l16 >> 2));
    }
    const int n = (int)(st.cols - col > 8 ? 8 : st.cols - col);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = row0 + u * step;
      if (r >= all_rows) continue;
      float v[8];
      values8(code[u], scale_down(sb[u]), v);
      if (wide && n == 8) {  // fp32: whole 32-byte sectors
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[j]);
        ptx::st_global_v8(out + r * st.cols + col, w);
      } else {
        store8<T>(out + r * st.cols + col, n, vec, v);
      }
    }
  }
}

// Grid of the row kernels: chunks of 128 columns on y, rows on x, U rows per
// group when that still leaves four CTAs for every SM.
struct RowGrid {
  RowMap map;
  dim3 grid;
  bool many;  // U rows a group, else one
};
RowGrid row_grid(int64_t rows, int64_t chunks, int groups_shift, int u) {
  RowGrid g;
  g.map.chunks = chunks;
  g.map.chunk_shift = 0;
  while (g.map.chunk_shift < groups_shift && (1 << g.map.chunk_shift) < chunks) ++g.map.chunk_shift;
  const int64_t y = ceil_div(chunks, 1 << g.map.chunk_shift);
  const int64_t per = 1 << (groups_shift - g.map.chunk_shift);  // rows of a CTA at U == 1
  g.many = ceil_div(rows, per * u) * y >= 4 * (int64_t)device_sm_count();
  g.grid = dim3((unsigned)ceil_div(rows, per * (g.many ? u : 1)), (unsigned)(y < 65535 ? y : 65535));
  return g;
}

// The low bits of every row's address.
template <typename T>
uintptr_t row_bits(const QuantArgs& a) {
  return reinterpret_cast<uintptr_t>(a.x) | (uintptr_t)(a.row_stride * (int64_t)sizeof(T)) |
         (uintptr_t)(a.batch_stride * (int64_t)sizeof(T));
}
// CTAs of the column kernel with four blocks a lane.
template <typename T>
int64_t four_blocks(const QuantArgs& a) {
  return a.batch * ceil_div(a.cols, ColTile<T>::CTA_COLS) * ceil_div(a.rows, 128);
}

template <typename T>
cudaError_t quantize(const QuantArgs& a, bool transpose, cudaStream_t s) {
  const uintptr_t bits = row_bits<T>(a);
  const int vec = (bits & 31u) == 0 ? 2 : (bits & 15u) == 0 ? 1 : 0;
  cudaError_t e;
  if (transpose) {
    const bool words = (bits & 3u) == 0;  // 32-bit loads of whole columns or pairs of them
    const int64_t sms = device_sm_count(), four = four_blocks<T>(a), cap = sms * 8;
    if (a.q_rows) {
      const int64_t tiles = a.batch * ceil_div(a.rows, 128) * ceil_div(a.cols, BOTH);
      e = launch_after_previous(k_mx_quant_both<T>, dim3((unsigned)tiles), dim3(256), 0, s, a, vec);
    } else if (a.order) {
      e = launch_after_previous(k_mx_quant_cols<T, 4, true>,
                                dim3((unsigned)(four < cap ? four : cap)), dim3(256), 0, s, a, words);
    } else if (four >= 2 * sms) {
      e = launch_after_previous(k_mx_quant_cols<T, 4, false>, dim3((unsigned)(four < cap ? four : cap)),
                                dim3(256), 0, s, a, words);
    } else {
      e = launch_after_previous(k_mx_quant_cols<T, 1, false>,
                                dim3((unsigned)(four * 4 < cap ? four * 4 : cap)), dim3(256), 0, s,
                                a, words);
    }
  } else {
    const RowGrid g = row_grid(a.batch * a.rows, a.st.block_atoms, GROUPS_SHIFT, 2);
    const auto k = a.dest ? (g.many ? k_mx_quant_rows<T, 2, true> : k_mx_quant_rows<T, 1, true>)
                          : (g.many ? k_mx_quant_rows<T, 2, false> : k_mx_quant_rows<T, 1, false>);
    e = launch_after_previous(k, g.grid, dim3(256), 0, s, a, g.map, vec);
  }
  note_launch();
  return e;
}

template <typename T>
cudaError_t quantize_two(const QuantArgs& a, const QuantArgs& b, cudaStream_t s) {
  const int64_t sms = device_sm_count(), cap = sms * 8, fa = four_blocks<T>(a), fb = four_blocks<T>(b);
  const int per = fa + fb >= 2 * sms ? 1 : 4;  // CTAs for the work of four blocks a lane
  const int na = (int)(fa * per < cap ? fa * per : cap), nb = (int)(fb * per < cap ? fb * per : cap);
  const cudaError_t e =
      launch_after_previous(per == 1 ? k_mx_quant_two<T, 4> : k_mx_quant_two<T, 1>,
                            dim3((unsigned)(na + nb)), dim3(256), 0, s, a, (row_bits<T>(a) & 3u) == 0, b,
                            (row_bits<T>(b) & 3u) == 0, na);
  note_launch();
  return e;
}

template <typename T>
cudaError_t dequantize(const uint8_t* q, const Store& st, void* out, cudaStream_t s) {
  const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0 &&
                   (st.cols * (int64_t)sizeof(T)) % 16 == 0;
  const bool wide = sizeof(T) == 4 && vec && (reinterpret_cast<uintptr_t>(out) & 31u) == 0 &&
                    st.cols % 8 == 0;
  const RowGrid g = row_grid(st.batch * st.rows, st.block_atoms, 4, 4);
  const cudaError_t e =
      launch_after_previous(g.many ? k_mx_dequant<T, 4> : k_mx_dequant<T, 1>, g.grid, dim3(256), 0,
                            s, q, st, static_cast<T*>(out), g.map, vec, wide);
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

cudaError_t launch_quantize_two(const QuantArgs& a, const QuantArgs& b, int dtype, cudaStream_t s) {
  note_kernel_name("k_mx_quant_two");
  if (dtype == IMC_F32) return quantize_two<float>(a, b, s);
  if (dtype == IMC_F16) return quantize_two<__half>(a, b, s);
  return quantize_two<__nv_bfloat16>(a, b, s);
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
