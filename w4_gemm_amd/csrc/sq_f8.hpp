// Device helpers of the 8-bit float mode: the e4m3 rounding of a block, and the
// curves of the gated block.
#pragma once
#include "sq_i8.hpp"

namespace sq {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------- e4m3 blocks
// A block whose largest magnitude is `top` (fp32 bits without the sign) is held
// as codes e4m3(v / 2^e) with the least e >= -127 that keeps them at or below
// 448 = 1.75 * 2^8; the byte is e + 127, or 255 (NaN) where the block holds inf
// or NaN.  e depends on bits alone and v / 2^e is exact (or below the smallest
// code's half), so a code is one correctly rounded operation whatever the order
// or the split of the work.
__device__ __forceinline__ int f8_exponent(uint32_t top) {
  const int e = (int)(top >> 23);
  return e == 255 ? 255 : max(e - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), 0);
}

// 2^(127 - byte): what the block's values are multiplied by.  For byte 255 it is
// zero, which leaves inf and NaN a NaN code and finite values a zero.
__device__ __forceinline__ float f8_inverse(int byte) {
  return __uint_as_float(byte == 255 ? 0u : (uint32_t)(254 - byte) << 23);
}

// Four codes, the first in the low byte (round to nearest even; |v| <= 448).
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Largest magnitude (bits) of two bf16 words' halves, kept as two halves.
__device__ __forceinline__ uint32_t abs_max_u16(uint32_t m, uint32_t w) {
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                          __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu)));
}
__device__ __forceinline__ uint32_t u16_pair_max(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

// Eight bf16 values times f as eight codes (two words).
__device__ __forceinline__ u32x2 f8_of_bf16x8(u32x4 v, float f) {
  u32x2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    o[h] = f8_pack4(__uint_as_float(v[2 * h] << 16) * f, __uint_as_float(v[2 * h] & 0xFFFF0000u) * f,
                    __uint_as_float(v[2 * h + 1] << 16) * f,
                    __uint_as_float(v[2 * h + 1] & 0xFFFF0000u) * f);
  return o;
}

// ---------------------------------------------------------------- curves
// act(g) and act'(g) of the gated block in fp32: 0 SiLU g s(g); 1 GELU
// g Phi(g); 2 its tanh form, which is g s(2 z), z = c (g + 0.044715 g^3).
// e^x as 2^(x log2 e): the product's rounding costs x 2^-24 of the result, which
// the curves' own slopes take back.
__device__ __forceinline__ float exp_f32(float x) {
  return __builtin_amdgcn_exp2f(1.4426950408889634f * x);
}
__device__ __forceinline__ float sigmoid_f32(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp_f32(-x));
}
template <int ACT>
__device__ __forceinline__ void act_curve(float g, float& value, float& slope) {
  if constexpr (ACT == 0) {
    const float s = sigmoid_f32(g);
    value = g * s;
    slope = s * (1.0f + g * (1.0f - s));
  } else if constexpr (ACT == 1) {
    const float cdf = 0.5f * erfcf(-0.70710678118654752f * g);
    value = g * cdf;
    slope = cdf + g * 0.39894228040143268f * exp_f32(-0.5f * g * g);
  } else {
    constexpr float C2 = 1.5957691216057308f;   // 2 sqrt(2 / pi)
    const float p = sigmoid_f32(C2 * (g + 0.044715f * g * g * g));
    value = g * p;
    // p (1 - p) is zero from |g| = 13 on, where g^2 must not reach infinity
    const float c = fminf(fmaxf(g, -64.0f), 64.0f);
    slope = p + g * p * (1.0f - p) * C2 * (1.0f + 0.134145f * c * c);
  }
}
__device__ __forceinline__ float act_value(int act, float g) {
  float v, s;
  if (act == 0) act_curve<0>(g, v, s);
  else if (act == 1) act_curve<1>(g, v, s);
  else act_curve<2>(g, v, s);
  return v;
}

// N consecutive values of a row as fp32 or bf16; `left` columns remain (rows of
// an odd width are 4- or 2-byte aligned only).  PASS: runs of eight bf16 leave
// without staying in the L2, whose lines the operands need.
template <int N, bool PASS = false>
__device__ __forceinline__ void store_run(void* __restrict__ y, int64_t at, const float (&o)[N],
                                          int left, bool bf16) {
  if (bf16) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(y) + at;
    if (left >= N) {
      uint32_t w[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
      if constexpr (PASS) {
        static_assert(N == 8, "16 bytes");
        typedef uint32_t run __attribute__((ext_vector_type(4), aligned(2)));
        __builtin_nontemporal_store((run){w[0], w[1], w[2], w[3]}, reinterpret_cast<run*>(dst));
      } else {
        __builtin_memcpy(dst, w, 2 * N);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) dst[i] = f32_to_bf16(o[i]);
    }
  } else {
    float* dst = reinterpret_cast<float*>(y) + at;
    if (left >= N) {
      __builtin_memcpy(dst, o, 4 * N);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) dst[i] = o[i];
    }
  }
}

}  // namespace sq
