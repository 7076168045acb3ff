// Device pieces of the MXFP4 quantisation, shared by the quantiser and by the
// product's form that quantises its few tokens itself.
#pragma once

#include <type_traits>

#include "mx_internal.cuh"
#include "ptx.cuh"

namespace imc {
namespace mx {

// Scale byte of a block from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t max_bits) {
  const uint32_t e = max_bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - byte), the factor that brings a block into [0, 8); 0 for a NaN block, whose
// codes mean nothing (0 for its numbers, some other code for its infinities and NaNs).
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
// Sixteen scaled values to sixteen codes.
__device__ __forceinline__ uint2 codes16(const float (&v)[16], float up) {
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = v[i];
    hi[i] = v[8 + i];
  }
  return make_uint2(codes8(lo, up), codes8(hi, up));
}

// A lane's 16 values of one row: loaded raw, so that the U rows' loads are in
// flight together, and widened later.
template <typename T>
struct Raw16 {
  static constexpr int N = (int)sizeof(T);  // 16-byte words
  static constexpr bool PAIRS = std::is_same<T, __nv_bfloat16>::value;
  uint4 w[N];
  // vec: 2 when p is 32-byte aligned, 1 when 16.  32-byte loads touch whole sectors: L1
  // is 33 % busy in the rows' kernel, with 16-byte loads 72 %, and the kernel that
  // quantises both ways takes 3 us less at 8192 x 4096 fp32 (rows alone 0.3).
  __device__ __forceinline__ void load(const T* p, int n, int vec) {
    if (vec == 2 && n == 16) {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        uint32_t u[8];
        ptx::ld_global_v8(u, p + i * (32 / sizeof(T)));
        w[2 * i] = make_uint4(u[0], u[1], u[2], u[3]);
        w[2 * i + 1] = make_uint4(u[4], u[5], u[6], u[7]);
      }
    } else if (vec && n == 16) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    } else {
      alignas(16) T e[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) e[i] = i < n ? p[i] : from_f32<T>(0.0f);
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint4*>(e)[i];
    }
  }
  // Bits of the largest magnitude as a float (NaN above infinity above numbers);
  // 16-bit values are compared two at a time.
  __device__ __forceinline__ uint32_t max_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        m = sizeof(T) == 4 ? max(m, u[j] & 0x7FFFFFFFu) : __vmaxu2(m, u[j] & 0x7FFF7FFFu);
    }
    return sizeof(T) == 4 ? m : top16(max(m & 0xFFFFu, m >> 16));
  }
  // A magnitude's 16 bits as the bits of a float.
  static __device__ __forceinline__ uint32_t top16(uint32_t h) {
    return is_bf16(T()) ? h << 16 : __float_as_uint(__half2float(__ushort_as_half((uint16_t)h)));
  }
  __device__ __forceinline__ void widen(float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (sizeof(T) == 4) {
          v[4 * i + j] = __uint_as_float(u[j]);
        } else {
          const float2 f = two(u[j]);
          v[8 * i + 2 * j] = f.x;
          v[8 * i + 2 * j + 1] = f.y;
        }
      }
    }
  }
  // The values times a power of two.  bf16 has fp32's exponents, so two values are
  // scaled by one multiplication before they are widened, exactly but for results
  // below 2^-126, which become the code 0 either way (8192 x 4096 by rows 17.7
  // us, widened first 18.2).
  __device__ __forceinline__ void scaled(float up, float (&v)[16]) const {
    if constexpr (PAIRS) {
      Raw16 t;
      const uint32_t both = pair_of(up, up);
#pragma unroll
      for (int i = 0; i < N; ++i)
        t.w[i] = make_uint4(times(w[i].x, both), times(w[i].y, both), times(w[i].z, both),
                            times(w[i].w, both));
      t.widen(v);
    } else {
      widen(v);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= up;
    }
  }
  // Two powers of two as a pair of bf16, and a pair times a pair.
  static __device__ __forceinline__ uint32_t pair_of(float lo, float hi) {
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
  }
  static __device__ __forceinline__ uint32_t times(uint32_t u, uint32_t by) {
    const __nv_bfloat162 r = __hmul2_rn(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                        *reinterpret_cast<const __nv_bfloat162*>(&by));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ float2 two(uint32_t u) {
    if (sizeof(T) == 2 && is_bf16(T()))
      return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
  static __device__ __forceinline__ bool is_bf16(__nv_bfloat16) { return true; }
  static __device__ __forceinline__ bool is_bf16(__half) { return false; }
  static __device__ __forceinline__ bool is_bf16(float) { return false; }
};

// The codes of a lane's 16 values and the scale word of its row's 128 columns:
// eight neighbouring lanes hold them (two lanes a block).
template <typename T>
__device__ __forceinline__ void quantize_128(const Raw16<T>& raw, uint2& code, uint32_t& word) {
  uint32_t m = raw.max_bits();
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const uint32_t sb = scale_byte(m);
  float v[16];
  raw.scaled(scale_up(sb), v);
  code = codes16(v, 1.0f);
  word = sb << (((threadIdx.x & 7) >> 1) * 8);
  word |= __shfl_xor_sync(0xffffffffu, word, 2);
  word |= __shfl_xor_sync(0xffffffffu, word, 4);
}

}  // namespace mx
}  // namespace imc
