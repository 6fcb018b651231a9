// 8-bit float mode: the quantizers.
//
//   k_f8_weight      codes and exponents of a weight, blocks of 128 x 128
//   k_f8_rows        codes and exponents of bf16 rows, blocks of 1 x 128
//   k_f8_gated_rows  dg = dh u act'(g) and du = dh act(g) of the gated block,
//                    their codes and exponents, and both in bf16 where wanted
//
// Rounding of a block: sq_f8.hpp.
#include "sq_f8.hpp"
#include "sq_kernels.h"

namespace sq {
namespace {

// ---------------------------------------------------------------- weight
// A workgroup takes one block: 16 lanes hold a row's 128 values (eight each), 16
// rows at a time, all 64 of a thread's values in registers between the maximum
// and the rounding.  Columns from k on are zero codes.  The weight is read once,
// which is what bounds it (16384 x 6144 from fp32: 89 us, 503 MB at 5.6 TB/s; a
// copy of that size runs at 5.3).
template <bool BF16>
__device__ __forceinline__ void load8_weight(const void* __restrict__ w, int64_t at, int left,
                                             float (&v)[8]) {
  if constexpr (BF16) {
    const u32x4 p = load8_u16(reinterpret_cast<const uint16_t*>(w) + at, left);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(p[i] << 16);
      v[2 * i + 1] = __uint_as_float(p[i] & 0xFFFF0000u);
    }
  } else {
    const float* src = reinterpret_cast<const float*>(w) + at;
    if (left >= 8) {
      __builtin_memcpy(v, src, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? src[i] : 0.0f;
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(256) k_f8_weight(const void* __restrict__ w,
                                                   uint8_t* __restrict__ codes,
                                                   uint8_t* __restrict__ exps,
                                                   int32_t* __restrict__ flags, int n, int k,
                                                   int kb) {
  __shared__ uint32_t wave_top[4];
  const int tid = threadIdx.x, nbk = (int)blockIdx.x / kb, kbk = (int)blockIdx.x - nbk * kb;
  const int row0 = 128 * nbk + (tid >> 4), col = 128 * kbk + 8 * (tid & 15);
  float v[8][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 16 * i;
    if (row < n) {
      load8_weight<BF16>(w, (int64_t)row * k + col, k - col, v[i]);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) v[i][c] = 0.0f;
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) top = max(top, __float_as_uint(v[i][c]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, s));
  if ((tid & 63) == 0) wave_top[tid >> 6] = top;
  __syncthreads();
  top = max(max(wave_top[0], wave_top[1]), max(wave_top[2], wave_top[3]));
  const int e = f8_exponent(top);
  const float f = f8_inverse(e);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + 16 * i;
    if (row < n) {
      const u32x2 o = {f8_pack4(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f),
                       f8_pack4(v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f)};
      *reinterpret_cast<u32x2*>(codes + (int64_t)row * (128 * kb) + col) = o;
    }
  }
  if (tid == 0) {
    exps[blockIdx.x] = (uint8_t)e;
    if (e == 255) atomicOr(flags, 1);   // SQ_FLAG_NONFINITE
  }
}

// ---------------------------------------------------------------- rows
// Eight lanes hold a block (16 values each), a wave eight blocks of one row; the
// maximum meets in three lane swaps, so a row is read once and no block waits for
// another.  Bound by memory (4480 x 16384: 35 us, 221 MB at 6.3 TB/s); 4480 x 6144
// takes 16 us.  Rows outside the groups' ranges are skipped.
template <bool VEC>
__global__ void __launch_bounds__(256) k_f8_rows(const uint16_t* __restrict__ x,
                                                 const int32_t* __restrict__ offsets, int groups,
                                                 uint8_t* __restrict__ codes,
                                                 uint8_t* __restrict__ exps, int m, int k, int kb,
                                                 int lax, int pitch) {
  const int lane = threadIdx.x & 63;
  const int per = (kb + 7) >> 3;
  const int unit = __builtin_amdgcn_readfirstlane((int)blockIdx.x * 4 + (int)(threadIdx.x >> 6));
  const int row = unit / per;
  if (row >= m) return;
  if (offsets && (row < offsets[0] || row >= offsets[groups])) return;
  const int blk = (unit - row * per) * 8 + (lane >> 3);
  const int col = 128 * blk + 16 * (lane & 7);
  const uint16_t* src = x + (int64_t)row * k + col;
  u32x4 v[2] = {};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int left = k - col - 8 * h;
    if constexpr (VEC) {
      if (left > 0) v[h] = *reinterpret_cast<const u32x4*>(src + 8 * h);
    } else if (left > 0) {
      v[h] = load8_u16(src + 8 * h, left);
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = abs_max_u16(top, v[i >> 2][i & 3]);
  top = u16_pair_max(top);
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, s));
  const int e = f8_exponent(top << 16);
  const float f = f8_inverse(e);
  if (blk >= kb) return;
  const u32x2 lo = f8_of_bf16x8(v[0], f), hi = f8_of_bf16x8(v[1], f);
  *reinterpret_cast<u32x4*>(codes + ((int64_t)row * pitch + blk) * 128 + 16 * (lane & 7)) =
      (u32x4){lo[0], lo[1], hi[0], hi[1]};
  if ((lane & 7) == 0) exps[(int64_t)row * lax + blk] = (uint8_t)e;
}

// ---------------------------------------------------------------- gated rows
// Sixteen lanes hold a block (eight values each), a wave four blocks of one row.
// dg and du are computed in fp32 and rounded twice, each time from there: to
// e4m3 for the products and to bf16 for the caller.  Block b of a row's codes is
// dg's, block nb + b du's.  Bound by memory: 12 bytes a value (4480 x 16384: 150 us,
// 883 MB at 5.9 TB/s).
template <int ACT, bool VEC>
__global__ void __launch_bounds__(256) k_f8_gated_rows(
    const uint16_t* __restrict__ dh, const uint16_t* __restrict__ g,
    const uint16_t* __restrict__ u, const int32_t* __restrict__ offsets, int groups,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ exps, uint16_t* __restrict__ dg_out,
    uint16_t* __restrict__ du_out, int m, int n, int nb, int lax, int pitch) {
  const int lane = threadIdx.x & 63, sub = lane & 15;
  const int per = (nb + 3) >> 2;
  const int unit = __builtin_amdgcn_readfirstlane((int)blockIdx.x * 4 + (int)(threadIdx.x >> 6));
  const int row = unit / per;
  if (row >= m) return;
  if (offsets && (row < offsets[0] || row >= offsets[groups])) return;
  const int blk = (unit - row * per) * 4 + (lane >> 4);
  const int col = 128 * blk + 8 * sub, left = n - col;
  const int64_t at = (int64_t)row * n + col;
  u32x4 vd = {}, vg = {}, vu = {};
  if (left > 0) {
    if constexpr (VEC) {
      vd = *reinterpret_cast<const u32x4*>(dh + at);
      vg = *reinterpret_cast<const u32x4*>(g + at);
      vu = *reinterpret_cast<const u32x4*>(u + at);
    } else {
      vd = load8_u16(dh + at, left);
      vg = load8_u16(g + at, left);
      vu = load8_u16(u + at, left);
    }
  }
  float dg[8], du[8];
  uint32_t tg = 0, tu = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const auto half = [&](const u32x4& v) {
      return __uint_as_float(i & 1 ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
    };
    float value, slope;
    act_curve<ACT>(half(vg), value, slope);
    // dh u is exact; where it passes fp32's range the slope may bring dg back, so
    // there both factors (each above 1 then) are halved 64 times and dg doubled
    const float d = half(vd), both = d * half(vu);
    dg[i] = both * slope;
    if (__builtin_isinf(both)) dg[i] = (d * 0x1p-64f) * (half(vu) * 0x1p-64f) * slope * 0x1p64f * 0x1p64f;
    du[i] = d * value;
    tg = max(tg, __float_as_uint(dg[i]) & 0x7FFFFFFFu);
    tu = max(tu, __float_as_uint(du[i]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int s = 1; s < 16; s <<= 1) {
    tg = max(tg, (uint32_t)__shfl_xor((int)tg, s));
    tu = max(tu, (uint32_t)__shfl_xor((int)tu, s));
  }
  if (blk >= nb) return;
  const int eg = f8_exponent(tg), eu = f8_exponent(tu);
  const float fg = f8_inverse(eg), fu = f8_inverse(eu);
  uint8_t* dst = codes + ((int64_t)row * pitch + blk) * 128 + 8 * sub;
  *reinterpret_cast<u32x2*>(dst) =
      (u32x2){f8_pack4(dg[0] * fg, dg[1] * fg, dg[2] * fg, dg[3] * fg),
              f8_pack4(dg[4] * fg, dg[5] * fg, dg[6] * fg, dg[7] * fg)};
  *reinterpret_cast<u32x2*>(dst + 128 * nb) =
      (u32x2){f8_pack4(du[0] * fu, du[1] * fu, du[2] * fu, du[3] * fu),
              f8_pack4(du[4] * fu, du[5] * fu, du[6] * fu, du[7] * fu)};
  if (sub == 0) {
    exps[(int64_t)row * lax + blk] = (uint8_t)eg;
    exps[(int64_t)row * lax + nb + blk] = (uint8_t)eu;
  }
  if (dg_out && left > 0) store_run<8>(dg_out, at, dg, left, true);
  if (du_out && left > 0) store_run<8>(du_out, at, du, left, true);
}

}  // namespace

hipError_t launch_f8_weight(const void* w, int w_bf16, uint8_t* codes, uint8_t* exps,
                            int32_t* flags, int64_t n, int64_t k, hipStream_t stream) {
  const int kb = (int)((k + 127) / 128);
  const dim3 grid((unsigned)((n + 127) / 128 * kb));
  if (w_bf16)
    hipLaunchKernelGGL(k_f8_weight<true>, grid, dim3(256), 0, stream, w, codes, exps, flags,
                       (int)n, (int)k, kb);
  else
    hipLaunchKernelGGL(k_f8_weight<false>, grid, dim3(256), 0, stream, w, codes, exps, flags,
                       (int)n, (int)k, kb);
  return hipGetLastError();
}

int64_t f8_rows_blocks(int64_t m, int64_t cols, bool gated) {
  const int64_t cb = (cols + 127) / 128;
  return (m * (gated ? (cb + 3) / 4 : (cb + 7) / 8) + 3) / 4;
}

hipError_t launch_f8_rows(const uint16_t* x, const int32_t* offsets, int groups, uint8_t* codes,
                          uint8_t* exps, int64_t m, int64_t k, int lax, int pitch,
                          hipStream_t stream) {
  const dim3 grid((unsigned)f8_rows_blocks(m, k, false));
  const int kb = (int)((k + 127) / 128);
  if (k % 8 == 0)
    hipLaunchKernelGGL(k_f8_rows<true>, grid, dim3(256), 0, stream, x, offsets, groups, codes, exps,
                       (int)m, (int)k, kb, lax, pitch);
  else
    hipLaunchKernelGGL(k_f8_rows<false>, grid, dim3(256), 0, stream, x, offsets, groups, codes,
                       exps, (int)m, (int)k, kb, lax, pitch);
  return hipGetLastError();
}

hipError_t launch_f8_gated_rows(const uint16_t* dh, const uint16_t* g, const uint16_t* u, int act,
                                const int32_t* offsets, int groups, uint8_t* codes, uint8_t* exps,
                                uint16_t* dg, uint16_t* du, int64_t m, int64_t n, int lax,
                                int pitch, hipStream_t stream) {
  const dim3 grid((unsigned)f8_rows_blocks(m, n, true));
  const int nb = (int)((n + 127) / 128);
#define SQ_F8_GATED(ACT, VEC)                                                                     \
  hipLaunchKernelGGL((k_f8_gated_rows<ACT, VEC>), grid, dim3(256), 0, stream, dh, g, u, offsets, \
                     groups, codes, exps, dg, du, (int)m, (int)n, nb, lax, pitch)
  if (n % 8 == 0) {
    if (act == 0) SQ_F8_GATED(0, true);
    else if (act == 1) SQ_F8_GATED(1, true);
    else SQ_F8_GATED(2, true);
  } else {
    if (act == 0) SQ_F8_GATED(0, false);
    else if (act == 1) SQ_F8_GATED(1, false);
    else SQ_F8_GATED(2, false);
  }
#undef SQ_F8_GATED
  return hipGetLastError();
}

}  // namespace sq
