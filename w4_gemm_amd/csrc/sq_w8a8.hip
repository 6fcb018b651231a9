// 8-bit forward of the int8 mode (W8A8), for one layer and for experts:
//
//   y = s w (q c^T) + (x down) up^T
//
// with q, s the 8-bit integers and the scale of each token of x H (H the
// normalized Hadamard-256), c, w the payload's codes and row scales.
//
// Rotation and rounding of a token.  A block of 256 values with absmax below
// 2^e is held as integers X = trunc(x 2^(23 - e)) (bf16 values down to
// 2^-15 of the block's largest exponent are exact), so the Sylvester sums
// R = X S stay below 2^31 and are exact in int32 in any order; then
//   r = fp32(R) 2^(e - 27)                      (= x H, one rounding)
//   a = max(max_k |r|, 2^-100), s = fp32(a / 127), i = fp32(127 / a)
//   q = round_half_even(fp32(r i))              (|q| <= 127)
// Every step is one correctly rounded operation: the integers do not depend
// on the order of summation, the split of the work or the batch around a
// token.  A token that holds inf or NaN gets s = NaN and q = 0.
//
// Kernels:
//   k_w8a8_prep  q, s of every row, and the K slices of t = x down (bf16 MFMA)
//   k_w8a8_gemm  q c^T on v_mfma_i32_16x16x64_i8 (exact: K <= 65536 keeps the
//                sums below 2^31), scales and rank-r branch in the epilogue
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "sq_i8.hpp"
#include "sq_kernels.h"

namespace sq {
namespace {

// ---------------------------------------------------------------- pre-phase
// Unnormalized 256-point transform of integers held as in fwht_cross64_swap
// (64 consecutive columns per lane, four lanes l, l ^ 16, l ^ 32 per block);
// afterwards register 32a + 16b + r of lane group g holds column
// swap_col(g, 32a + 16b + r).
__device__ __forceinline__ void iwht256(int (&v)[64]) {
#pragma unroll
  for (int h = 1; h < 64; h <<= 1)
#pragma unroll
    for (int i = 0; i < 64; ++i)
      if ((i & h) == 0) {
        const int a = v[i], b = v[i + h];
        v[i] = a + b;
        v[i + h] = a - b;
      }
#pragma unroll
  for (int p = 0; p < 32; ++p) {
    const auto r = __builtin_amdgcn_permlane16_swap((uint32_t)v[p], (uint32_t)v[p + 32], false, false);
    const int x = (int)r[0], y = (int)r[1];
    v[p] = x + y;
    v[p + 32] = x - y;
  }
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    if (i & 16) continue;
    const auto r = __builtin_amdgcn_permlane32_swap((uint32_t)v[i], (uint32_t)v[i + 16], false, false);
    const int x = (int)r[0], y = (int)r[1];
    v[i] = x + y;
    v[i + 16] = x - y;
  }
}

constexpr int PREP_MAX_ROWS = 64;   // rows per workgroup at most
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// The first workgroups compute t (they run longest); the others hold
// rows_per_wg rows each, four lanes per (row, block) pair, 16 pairs per wave.
template <int RW>
__global__ void __launch_bounds__(1024) k_w8a8_prep(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ down,
    const int32_t* __restrict__ offsets, int groups, int8_t* __restrict__ xq,
    float* __restrict__ xs, float* __restrict__ t_part, int m, int k, int rank, int rows_per_wg,
    int project_wgs, int slices) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  const int tid = threadIdx.x, lane = tid & 63;
  if ((int)blockIdx.x < project_wgs) {
    if (rank == 16)
      project<16, RW, true>(x, down, offsets, groups, t_part, dyn, m, k, blockIdx.x, slices);
    else if (rank == 32)
      project<32, RW, true>(x, down, offsets, groups, t_part, dyn, m, k, blockIdx.x, slices);
    else
      project<64, RW, true>(x, down, offsets, groups, t_part, dyn, m, k, blockIdx.x, slices);
    return;
  }
  const int wg = (int)blockIdx.x - project_wgs;
  __shared__ uint32_t row_max[PREP_MAX_ROWS];
  if (tid < PREP_MAX_ROWS) row_max[tid] = 0;
  __syncthreads();
  const int nb = k >> 8;
  const int pair = (tid >> 6) * 16 + (lane & 15), g = lane >> 4;
  const int lrow = pair / nb, blk = pair - lrow * nb;
  const int row = wg * rows_per_wg + lrow;
  const bool live = lrow < rows_per_wg && row < m;
  float v[64];
  int e = 0;
  if (live) {
    const u32x4* src = reinterpret_cast<const u32x4*>(x + (int64_t)row * k + blk * 256 + 64 * g);
    u32x4 q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = src[j];
    u16x2 mx2 = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = q[j][i] & 0x7FFF7FFFu;
        mx2 = __builtin_elementwise_max(mx2, __builtin_bit_cast(u16x2, w));
      }
    uint32_t mx = max((uint32_t)mx2[0], (uint32_t)mx2[1]);
    mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16));
    mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32));
    const int be = max((int)(mx >> 7), 1);   // biased exponent of the block: |x| < 2^(be - 126)
    e = be - 153;                            // unit of R / 16
    int iv[64];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = q[j][i];
        iv[8 * j + 2 * i] = (int)__builtin_amdgcn_ldexpf(__uint_as_float(w << 16), 149 - be);
        iv[8 * j + 2 * i + 1] =
            (int)__builtin_amdgcn_ldexpf(__uint_as_float(w & 0xFFFF0000u), 149 - be);
      }
    iwht256(iv);
    float am = 0.0f;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      v[i] = (float)iv[i];
      am = fmaxf(am, fabsf(v[i]));
    }
    uint32_t bits = __float_as_uint(__builtin_amdgcn_ldexpf(am, e));
    if (mx >= 0x7F80u) bits = I8_NAN_BITS;
    bits = max(bits, (uint32_t)__shfl_xor((int)bits, 16));
    bits = max(bits, (uint32_t)__shfl_xor((int)bits, 32));
    if (g == 0) atomicMax(&row_max[lrow], bits);
  }
  __syncthreads();
  if (!live) return;
  const uint32_t rbits = row_max[lrow];
  const bool finite = rbits < 0x7F800000u;
  const float a = fmaxf(__uint_as_float(rbits), I8_MIN_ABSMAX);
  // inv 2^e times R rounds as inv times r does: r is a power of two times R
  const float f = finite ? __builtin_amdgcn_ldexpf(127.0f / a, e) : 0.0f;
  if (blk == 0 && g == 0) xs[row] = finite ? a / 127.0f : __uint_as_float(I8_NAN_BITS);
  // registers 32a + 16b + r: four runs of 16 consecutive columns
  int8_t* dst = xq + (int64_t)row * k + blk * 256;
#pragma unroll
  for (int run = 0; run < 4; ++run) {
    u32x4 o;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b[i] = __float_as_uint(v[16 * run + 4 * w + i] * f + I8_ROUND);
      const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u);
      const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u);
      o[w] = lo | (hi << 16);
    }
    *reinterpret_cast<u32x4*>(dst + swap_col(g, 16 * run)) = o;
  }
}

// ---------------------------------------------------------------- contraction
// BM x 256 output tile per workgroup (BM = 32 FM), 2 x 4 waves of 16 FM x 64
// (FM x 4 MFMA tiles).  One stage = 128 bytes of K of each operand row, two
// stages in LDS.  Both operands stream global -> LDS with direct 16-byte
// buffer loads that cover whole 128-byte lines (64-byte halves of lines cost
// 5 % of the 4480 x 16384 x 6144 contraction).  Chunk c of LDS row r sits at
// slot c ^ g_swz(r).
// LDS row 64 w + 16 j + f of the weight holds output column 64 w + 4 f + j, so
// that a lane ends up with four consecutive columns and stores them as they
// are.  The 256-row tile (FM = 8, unsplit) takes all 256 registers and spills
// seven of them (32 bytes of scratch per lane); no other form spills.
constexpr int G_BN = 256, G_THREADS = 512;

// Swizzle of 128-byte rows.  A loop of nothing but the fragment reads runs
// 1.9 times as long under c ^ (r & 7) ^ ((r >> 3) & 1), 3.7 times without any.
__device__ __forceinline__ int g_swz(int r) { return r & 7; }

// Four consecutive values of a row, fp32 or bf16; `left` columns remain (rows
// of an odd N are 4- or 2-byte aligned only).
__device__ __forceinline__ void store4(void* __restrict__ y, int64_t at, f32x4 o, int left,
                                       int y_bf16) {
  if (y_bf16) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(y) + at;
    const u32x2 b = {pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
    if (left >= 4) {
      __builtin_memcpy(dst, &b, 8);
    } else {
      for (int c = 0; c < left; ++c) dst[c] = (uint16_t)(b[c >> 1] >> (16 * (c & 1)));
    }
  } else {
    float* dst = reinterpret_cast<float*>(y) + at;
    if (left >= 4) {
      __builtin_memcpy(dst, &o, 16);
    } else {
      for (int c = 0; c < left; ++c) dst[c] = o[c];
    }
  }
}

template <int FM, bool SPLIT>
__global__ void __launch_bounds__(G_THREADS, 1) k_w8a8_gemm(
    const int8_t* __restrict__ xq, const float* __restrict__ xs,
    const float* __restrict__ t_part, const int8_t* __restrict__ codes,
    const uint16_t* __restrict__ scales, const uint16_t* __restrict__ up,
    const int32_t* __restrict__ offsets, int groups, void* __restrict__ y, int m, int n, int k,
    int rank, int slices, int y_bf16, int most_tiles, int splits, int32_t* __restrict__ partial) {
  constexpr int FN = 4, BM = 32 * FM;
  constexpr int BN = G_BN, WN = 4, WAVES = 8, THREADS = G_THREADS;
  // one load instruction of every wave covers 64 rows of 128 bytes
  constexpr int NA = (BM + 63) / 64, NB = BN / 64;
  constexpr int A_STAGE = NA * 64 * 128, B_STAGE = BN * 128;
  __shared__ __attribute__((aligned(16))) uint8_t a0[A_STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t a1[A_STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t b0[B_STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t b1[B_STAGE];
  __shared__ __attribute__((aligned(16))) float row_s[SPLIT ? 4 : BM];
  __shared__ __attribute__((aligned(16))) float col_w[SPLIT ? 4 : BN];
  // t of the tile's rows as bf16 parts (hi, lo and, for fp32 results, a third:
  // 2^-24 of t then), chunk (part, eight ranks, row) of 16 bytes.  Rank 16 has
  // room of its own and is fetched before the loop; the larger ranks (up to
  // 3 * 8 * BM chunks) take the weight's stage buffers after it.
  __shared__ __attribute__((aligned(16))) uint8_t t_early[SPLIT ? 16 : 3 * 2 * BM * 16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int fr = lane & 15, g = lane >> 4;
  const int nt = (n + BN - 1) / BN;
  const int mt = row_tile_count(offsets, groups, m, BM, most_tiles, lane);
  // workgroup b: K split b / tiles of tile b % tiles
  const int tiles = mt * nt;
  const int split = __builtin_amdgcn_readfirstlane(tiles ? (int)blockIdx.x / tiles : splits);
  if (split >= splits) return;
  int64_t tm, tn;
  xcd_tile((int)blockIdx.x - split * tiles, tiles, nt, tm, tn);
  RowTile rt;
  if (!find_row_tile(offsets, groups, m, BM, __builtin_amdgcn_readfirstlane((int)tm), lane, rt))
    return;
  // scalar registers for everything the descriptors are built from
  const int grp = __builtin_amdgcn_readfirstlane(rt.group);
  const int rows = __builtin_amdgcn_readfirstlane(rt.rows);
  const int64_t m0 = __builtin_amdgcn_readfirstlane(rt.row0);
  const int n0 = __builtin_amdgcn_readfirstlane((int)tn) * BN;
  const int cols = min(BN, n - n0);
  const int64_t brow0 = (int64_t)grp * n + n0;   // first weight row of the tile
  // stages of 128 values: an even number (the splits cut K in multiples of 256)
  const int st0 = 2 * __builtin_amdgcn_readfirstlane((int)((int64_t)split * (k >> 8) / splits));
  const int ST =
      2 * __builtin_amdgcn_readfirstlane((int)((int64_t)(split + 1) * (k >> 8) / splits)) - st0;

  // loaders: instruction i of wave w fills LDS rows 64 i + 8 w .. +8, through a
  // descriptor of its own (64 rows each) so that one offset serves all; rows
  // past the tile lie beyond their descriptor and fetch nothing
  const int lr = 8 * wave + (lane >> 3);
  const uint32_t lslot = 16u * (uint32_t)((lane & 7) ^ g_swz(lr));
  const uint32_t off_a = (uint32_t)lr * (uint32_t)k + lslot;
  const uint32_t off_b = (uint32_t)(4 * (lr & 15) + (lr >> 4)) * (uint32_t)k + lslot;
  const int8_t *a_base = xq + m0 * k, *b_base = codes + brow0 * k;
  const int kb = st0 * 128;
  auto issue = [&](int st, uint8_t* ab, uint8_t* bb) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(a_base + (int64_t)(64 * i) * k), (short)0, max(rows - 64 * i, 0) * k, 0x00020000);
      const __amdgpu_buffer_rsrc_t b_rsrc = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(b_base + (int64_t)(64 * i) * k), (short)0, max(cols - 64 * i, 0) * k, 0x00020000);
      if (i < NA)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            a_rsrc, (i8_lds_t)(ab + (WAVES * i + wave) * 1024), 16, off_a, kb + st * 128, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          b_rsrc, (i8_lds_t)(bb + (WAVES * i + wave) * 1024), 16, off_b, kb + st * 128, 0, 0);
    }
  };
  issue(0, a0, b0);
  issue(min(1, ST - 1), a1, b1);
  const int rank8 = rank >> 3, parts = y_bf16 ? 2 : 3;
  const int c0 = 64 * wn + 4 * fr, left = cols - c0;   // the lane's four columns
  auto t_chunk = [&](int part, int r8, int row) -> uint8_t* {
    const int at = ((part * rank8 + r8) * BM + row) * 16;
    if (rank8 <= 2) return t_early + at;
    return at < B_STAGE ? b0 + at : at < 2 * B_STAGE ? b1 + (at - B_STAGE) : a0 + (at - 2 * B_STAGE);
  };
  auto fetch_t = [&]() {
    for (int q = tid; q < BM * rank8; q += THREADS) {
      const int row = q % BM, r8 = q / BM;
      u32x4 part[3];
      project_sum8(t_part, m, rank, slices, (int)m0 + min(row, rows - 1), 8 * r8, part);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        if (p < parts) *reinterpret_cast<u32x4*>(t_chunk(p, r8, row)) = part[p];
    }
  };
  // rows of up, eight ranks per lane group.  The 32-wide MFMA takes rank 16
  // twice: lane groups 0, 1 carry one part of t, groups 2, 3 the next.
  const bool twice = rank8 == 2;
  bf16x8 bu[FN];
  auto fetch_up = [&](int rr) {
    const int r8 = twice ? g & 1 : rr + g;
#pragma unroll
    for (int j = 0; j < FN; ++j)
      bu[j] = r8 < rank8 ? *reinterpret_cast<const bf16x8*>(
                               up + (brow0 + min(c0 + j, cols - 1)) * rank + 8 * r8)
                         : (bf16x8){};
  };
  if constexpr (!SPLIT) {
    // what the epilogue needs comes in with the first stages
    for (int i = tid; i < BM + BN; i += THREADS) {
      if (i < BM)
        row_s[i] = xs[m0 + min(i, rows - 1)];
      else
        col_w[i - BM] = fp16_bits_to_f32(scales[brow0 + min(i - BM, cols - 1)]);
    }
    if (rank8 <= 2) fetch_t();
    fetch_up(0);
  }

  // fragment addresses: K half h is chunks 4 h .. 4 h + 3; 16-row tile i of
  // wave row wm is tile 2 i + wm of the workgroup
  const uint32_t a_row = (uint32_t)(16 * wm + fr) * 128, b_row = (uint32_t)(64 * wn + fr) * 128;
  uint32_t slot[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) slot[h] = 16u * (uint32_t)((4 * h + g) ^ g_swz(fr));
  i32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (i32x4){0, 0, 0, 0};
  auto sync = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(SQ_WAIT_VM0);
    __builtin_amdgcn_s_waitcnt(SQ_WAIT_LGKM0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  sync();
  // the loop over the first F of the wave's FM row tiles
  auto contract = [&](auto count) {
    constexpr int F = decltype(count)::value;
    struct Frag {
      i32x4 a[F], b[FN];
    };
    auto read = [&](Frag& f, const uint8_t* ab, const uint8_t* bb, int h) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
        f.b[j] = *reinterpret_cast<const i32x4*>(bb + b_row + slot[h] + j * 2048);
#pragma unroll
      for (int i = 0; i < F; ++i)
        f.a[i] = *reinterpret_cast<const i32x4*>(ab + a_row + slot[h] + i * 4096);
    };
    auto compute = [&](const Frag& f) {
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
    };
    auto interleave = [&]() {
#pragma unroll
      for (int i = 0; i < F + FN; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                // one LDS read
        __builtin_amdgcn_sched_group_barrier(0x008, F >= 4 ? 2 : 1, 0);   // MFMAs
      }
      __builtin_amdgcn_sched_group_barrier(0x008, F >= 4 ? F * FN - 2 * (F + FN) : 1, 0);
    };
    // global loads spread over the MFMAs: in a burst behind the barrier they
    // hold up every wave's issue (16 us of 4480 x 16384 x 6144)
    auto interleave_loads = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);   // one global load
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, F >= 2 ? F * FN / 8 : 1, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, F >= 2 ? F * FN / 8 : 1, 0);
      }
    };
    // One stage.  The K half in registers is contracted while the next one is
    // read.  At the barrier every wave has read all of the stage, so its buffers
    // take stage st + 2, and stage st + 1 has landed.  Loads past the last stage
    // fetch the last one again, into buffers that are not read any more.
    Frag f0, f1;
    auto stage = [&](int st, uint8_t* ab, uint8_t* bb, const uint8_t* an, const uint8_t* bn) {
      read(f1, ab, bb, 1);
      compute(f0);
      interleave();
      sync();
      issue(min(st + 2, ST - 1), ab, bb);
      read(f0, an, bn, 0);
      compute(f1);
      interleave_loads();
      __builtin_amdgcn_sched_barrier(0);
    };
    read(f0, a0, b0, 0);
    for (int st = 0; st < ST; st += 2) {
      stage(st, a0, b0, a1, b1);
      stage(st + 1, a1, b1, a0, b0);
    }
  };
  // a group's last tile is often half empty: it contracts half the row tiles
  constexpr int HALF = (FM + 1) / 2;
  if (FM >= 4 && rows <= 32 * HALF)
    contract(std::integral_constant<int, HALF>{});
  else
    contract(std::integral_constant<int, FM>{});
  __builtin_amdgcn_s_waitcnt(SQ_WAIT_VM0);   // the re-fetches have landed
  __builtin_amdgcn_sched_barrier(0);

  // acc[i][j][v] is row 32 i + 16 wm + 4 g + v, column 64 wn + 4 fr + j
  const int rbase = 16 * wm;
  if constexpr (SPLIT) {
    // the splits' integer sums meet in k_w8a8_join
    int32_t* dst = partial + ((int64_t)split * m + m0) * n + n0 + c0;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = rbase + 32 * i + 4 * g + v;
        if (r >= rows) continue;
        const i32x4 o = {acc[i][0][v], acc[i][1][v], acc[i][2][v], acc[i][3][v]};
        if (left >= 4) {
          __builtin_memcpy(dst + (int64_t)r * n, &o, 16);
        } else {
          for (int c = 0; c < left; ++c) dst[(int64_t)r * n + c] = o[c];
        }
      }
    return;
  }
  if (rank8 > 2) {
    __syncthreads();   // every wave is done with the stage buffers
    fetch_t();
    __syncthreads();
  }
  // scales, the column's first: |acc w| < 2^47 cannot overflow whatever the
  // row's magnitude is
  f32x4 out[FM][FN];
  const f32x4 wsc = *reinterpret_cast<const f32x4*>(&col_w[c0]);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const f32x4 sr = *reinterpret_cast<const f32x4*>(&row_s[rbase + 32 * i + 4 * g]);
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) out[i][j][v] = (float)acc[i][j][v] * wsc[j] * sr[v];
  }
  // rank-r branch t up^T
  for (int rr = 0; rr < rank8; rr += 4) {
    if (rr > 0) fetch_up(rr);
    for (int p = 0; p < parts; p += twice ? 2 : 1) {
      const int part = twice ? p + (g >> 1) : p, r8 = twice ? g & 1 : rr + g;
      const bool live = part < parts && r8 < rank8;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const bf16x8 at =
            live ? *reinterpret_cast<const bf16x8*>(t_chunk(part, r8, rbase + 32 * i + fr))
                 : (bf16x8){};
#pragma unroll
        for (int j = 0; j < FN; ++j)
          out[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(at, bu[j], out[i][j], 0, 0, 0);
      }
    }
  }
  // stores of four columns: 16 lanes write one row's 128 (bf16) or 256 bytes
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = rbase + 32 * i + 4 * g + v;
      if (r >= rows) continue;
      const f32x4 o = {out[i][0][v], out[i][1][v], out[i][2][v], out[i][3][v]};
      store4(y, (m0 + r) * n + n0 + c0, o, left, y_bf16);
    }
}

// Sum of the splits' integers (exact, in any order), scales and rank-r branch.
// One workgroup takes 16 rows of one group x 64 columns, a thread four columns
// of one row: at a few rows the partial sums are read by many workgroups with
// up to eight loads of a thread in flight (a form of 16 rows x 256 columns with
// the branch on MFMA took 7.8 us at 48 x 6144 and 8 splits).
__global__ void __launch_bounds__(256) k_w8a8_join(
    const int32_t* __restrict__ partial, const float* __restrict__ xs,
    const float* __restrict__ t_part, const uint16_t* __restrict__ scales,
    const uint16_t* __restrict__ up, const int32_t* __restrict__ offsets, int groups,
    void* __restrict__ y, int m, int n, int rank, int slices, int y_bf16, int splits) {
  __shared__ __attribute__((aligned(16))) float t_lds[16 * 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int nt = (n + 63) >> 6;
  const int tile = (int)blockIdx.x / nt;
  RowTile rt;
  if (!find_row_tile(offsets, groups, m, 16, tile, lane, rt)) return;
  const int lrow = tid >> 4, c0 = ((int)blockIdx.x - tile * nt) * 64 + 4 * (tid & 15);
  const int left = n - c0, row = rt.row0 + min(lrow, rt.rows - 1);
  i32x4 s = {0, 0, 0, 0};
  for (int sp = 0; sp < splits; sp += 8) {
    i32x4 p[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int32_t* src = partial + ((int64_t)min(sp + u, splits - 1) * m + row) * n + c0;
      p[u] = (i32x4){0, 0, 0, 0};
      if (left >= 4) {
        __builtin_memcpy(&p[u], src, 16);
      } else {
        for (int c = 0; c < left; ++c) p[u][c] = src[c];
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (sp + u < splits) s += p[u];
  }
  for (int q = tid; q < rt.rows * rank; q += 256) {
    float t = 0.0f;
    for (int sl = 0; sl < slices; sl += 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = t_part[((int64_t)min(sl + u, slices - 1) * m + rt.row0) * rank + q];
#pragma unroll
      for (int u = 0; u < 8; ++u) t += sl + u < slices ? v[u] : 0.0f;
    }
    t_lds[q] = t;
  }
  const int64_t wrow = (int64_t)rt.group * n;
  const float sr = xs[row];
  f32x4 out;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    out[j] = (float)s[j] * fp16_bits_to_f32(scales[wrow + min(c0 + j, n - 1)]) * sr;
  __syncthreads();
  if (lrow >= rt.rows || left <= 0) return;
  for (int r0 = 0; r0 < rank; r0 += 8) {
    const f32x4 ta = *reinterpret_cast<const f32x4*>(&t_lds[lrow * rank + r0]);
    const f32x4 tb = *reinterpret_cast<const f32x4*>(&t_lds[lrow * rank + r0 + 4]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4 u = *reinterpret_cast<const u32x4*>(up + (wrow + min(c0 + j, n - 1)) * rank + r0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float t0 = i < 2 ? ta[2 * i] : tb[2 * i - 4], t1 = i < 2 ? ta[2 * i + 1] : tb[2 * i - 3];
        out[j] = __builtin_fmaf(t0, __uint_as_float(u[i] << 16), out[j]);
        out[j] = __builtin_fmaf(t1, __uint_as_float(u[i] & 0xFFFF0000u), out[j]);
      }
    }
  }
  store4(y, (int64_t)row * n + c0, out, left, y_bf16);
}

// ---------------------------------------------------------------- small tiles
// 16 MT x 16 NT output tile per workgroup; its waves split K (256-value blocks
// in turn) and read both operands straight from memory in MFMA order: lane
// (f, g) holds 16 bytes of row f, K 64 s + 16 g.  With few rows the codes are
// read once and bound the time; nothing is shared between waves until the
// int32 partial sums, which meet in LDS (exact, so the split does not show).
// U of a block's four 64-value steps are in flight while the U before them are
// contracted.
template <int MT, int NT, int U>
__global__ void __launch_bounds__(512) k_w8a8_stream(
    const int8_t* __restrict__ xq, const float* __restrict__ xs,
    const float* __restrict__ t_part, const int8_t* __restrict__ codes,
    const uint16_t* __restrict__ scales, const uint16_t* __restrict__ up,
    const int32_t* __restrict__ offsets, int groups, void* __restrict__ y, int m, int n, int k,
    int rank, int slices, int y_bf16, int most_tiles) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  constexpr int BM = 16 * MT, BN = 16 * NT;
  const int tid = threadIdx.x, lane = tid & 63, fr = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = __builtin_amdgcn_readfirstlane((int)(blockDim.x >> 6));
  const int nt = (n + BN - 1) / BN;
  const int mt = row_tile_count(offsets, groups, m, BM, most_tiles, lane);
  if ((int64_t)blockIdx.x >= (int64_t)mt * nt) return;
  int64_t tm, tn;
  xcd_tile(blockIdx.x, (int64_t)mt * nt, nt, tm, tn);
  RowTile rt;
  if (!find_row_tile(offsets, groups, m, BM, __builtin_amdgcn_readfirstlane((int)tm), lane, rt))
    return;
  const int grp = __builtin_amdgcn_readfirstlane(rt.group);
  const int rows = __builtin_amdgcn_readfirstlane(rt.rows);
  const int64_t m0 = __builtin_amdgcn_readfirstlane(rt.row0);
  const int n0 = __builtin_amdgcn_readfirstlane((int)tn) * BN;
  const int cols = min(BN, n - n0);
  const int64_t brow0 = (int64_t)grp * n + n0;
  const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(xq + m0 * k), (short)0, rows * k, 0x00020000);
  const __amdgpu_buffer_rsrc_t b_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(codes + brow0 * k), (short)0, cols * k, 0x00020000);
  uint32_t off_a[MT], off_b[NT];   // rows past the tile repeat its last row
#pragma unroll
  for (int i = 0; i < MT; ++i)
    off_a[i] = (uint32_t)min(16 * i + fr, rows - 1) * (uint32_t)k + 16u * g;
#pragma unroll
  for (int j = 0; j < NT; ++j)
    off_b[j] = (uint32_t)min(16 * j + fr, cols - 1) * (uint32_t)k + 16u * g;

  struct Steps {
    i32x4 a[U][MT], b[U][NT];
  };
  const int nb = k >> 8;
  constexpr int PER = 4 / U;                       // groups of U steps per block
  const int todo = (nb - wave + waves - 1) / waves * PER;   // of this wave
  auto load = [&](Steps& f, int q) {
    // group q of this wave: block wave + waves (q / PER), steps U (q % PER) ..
    const int at = (wave + waves * (q / PER)) * 256 + 64 * U * (q % PER);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
        f.b[u][j] = __builtin_bit_cast(
            i32x4, __builtin_amdgcn_raw_buffer_load_b128(b_rsrc, off_b[j], at + 64 * u, 0));
#pragma unroll
      for (int i = 0; i < MT; ++i)
        f.a[u][i] = __builtin_bit_cast(
            i32x4, __builtin_amdgcn_raw_buffer_load_b128(a_rsrc, off_a[i], at + 64 * u, 0));
    }
  };
  i32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = (i32x4){0, 0, 0, 0};
  auto compute = [&](const Steps& f) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.a[u][i], f.b[u][j], acc[i][j], 0, 0, 0);
  };
  Steps f0, f1;
  if (todo > 0) load(f0, 0);
  int q = 0;
  for (; q + 2 <= todo; q += 2) {
    load(f1, q + 1);
    compute(f0);
    if (q + 2 < todo) load(f0, q + 2);
    compute(f1);
  }
  if (q < todo) compute(f0);

  // t parts of the rows: part, eight ranks, row -> 16 bytes; then the sums
  const int rank8 = rank >> 3, parts = y_bf16 ? 2 : 3;
  uint8_t* t_lds = dyn;
  uint8_t* red = dyn + (size_t)3 * rank8 * BM * 16;
  for (int c = tid; c < BM * rank8; c += blockDim.x) {
    const int row = c % BM, r8 = c / BM;
    u32x4 part[3];
    project_sum8(t_part, m, rank, slices, (int)m0 + min(row, rows - 1), 8 * r8, part);
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<u32x4*>(t_lds + ((p * rank8 + r8) * BM + row) * 16) = part[p];
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<i32x4*>(red + ((wave * MT + i) * NT + j) * 1024 + lane * 16) = acc[i][j];
  __syncthreads();
  // 16 x 16 tiles in turn: row 16 i + 4 g + v, column 16 j + fr
  for (int tile = wave; tile < MT * NT; tile += waves) {
    const int i = tile / NT, j = tile % NT;
    i32x4 s = {0, 0, 0, 0};
    for (int w = 0; w < waves; ++w)
      s += *reinterpret_cast<const i32x4*>(red + (w * MT * NT + tile) * 1024 + lane * 16);
    const int col = 16 * j + fr;
    const int64_t wrow = brow0 + min(col, cols - 1);
    const float wsc = fp16_bits_to_f32(scales[wrow]);
    f32x4 out;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      out[v] = (float)s[v] * wsc * xs[m0 + min(16 * i + 4 * g + v, rows - 1)];
    for (int rr = 0; rr < rank8; rr += 4) {
      const bool rk = rr + g < rank8;
      const bf16x8 bu =
          rk ? *reinterpret_cast<const bf16x8*>(up + wrow * rank + 8 * (rr + g)) : (bf16x8){};
      for (int p = 0; p < parts; ++p) {
        const bf16x8 at = rk ? *reinterpret_cast<const bf16x8*>(
                                   t_lds + ((p * rank8 + rr + g) * BM + 16 * i + fr) * 16)
                             : (bf16x8){};
        out = __builtin_amdgcn_mfma_f32_16x16x32_bf16(at, bu, out, 0, 0, 0);
      }
    }
    if (col >= cols) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = 16 * i + 4 * g + v;
      if (r >= rows) continue;
      const int64_t at = (m0 + r) * n + n0 + col;
      if (y_bf16)
        reinterpret_cast<uint16_t*>(y)[at] = f32_to_bf16(out[v]);
      else
        reinterpret_cast<float*>(y)[at] = out[v];
    }
  }
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// Tile of the contraction.  Each form's time (us) is modelled and the least
// chosen; the constants are fitted to 4400 timed (M, N, K, groups) between
// 1 x 64 x 256 and 16384 x 4096 x 4096 / 4480 x 16384 x 16384, over which the
// choice takes 1.015 times the best form on average.  What decides:
//   small tiles (waves split K, operands straight from memory): the time grows
//     with the K steps of a wave and with the tiles per CU; 16 x 32 reads the
//     codes once for up to 16 rows (1 x 16384 x 6144: 25 us against 34 us for
//     a 64 x 256 tile with 4 splits) and 64 x 64 shares them among more rows
//     (777 x 1003 x 2304: 21 against 26 us);
//   large tiles (operands shared in LDS): whole rounds of 256 tiles, one stage
//     of 128 K after another; few tiles split K so that every CU has one (48 x
//     6144 x 16384: 38 us with 8 splits, 175 us with one), at the price of the
//     partial sums' trip through memory;
//   none is faster than its codes arrive.
// 128 x 128 tiles of four waves, two workgroups per CU, were the best form by
// up to 10 % at a few shapes (1024 x 4096 x 8192) and by 0.3 % on average: not
// kept.
struct SmallTile {
  int mt, nt;
  double fixed, step, share, enough, tile;
};
constexpr SmallTile kSmall[] = {{1, 1, 8.2, 1.05, 2.15, 0.0, 0.1},
                                {1, 2, 9.0, 1.5, 3.05, 0.0, 0.3},
                                {2, 4, 9.8, 3.5, 5.7, 0.2, 0.6},
                                {4, 4, 11.9, 4.9, 8.9, 0.55, 1.2}};
struct LargeTile {
  int rows;
  double fixed, tile, stage;     // us, us per round, us per stage and round
  double join, bytes, parts;     // join: us, MB of partial sums per us, rounds of parts count more
};
constexpr LargeTile kLarge[] = {{64, 7.9, 4.2, 0.75, 6.8, 3.4, 1.37},
                                {128, 7.3, 5.6, 1.0, 7.7, 1.9, 1.0},
                                {224, 0.0, 14.2, 1.06, 0, 0, 0},
                                {256, 0.0, 14.3, 1.17, 0, 0, 0}};

void choose_tile(W8A8Plan& p) {
  const int64_t nb = p.k / 256;
  const double codes = (double)std::min<int64_t>(p.groups, p.m) * (double)p.n * (double)p.k / 5.6e6;
  // up to 12 rows per group the 16-row tiles, which read the codes once, are
  // the best form (by 0.5 % on average over 1900 timed shapes the others were
  // better, and up to 1.5 times slower where the model preferred them)
  const bool few = p.m <= 12 * std::min<int64_t>(p.groups, p.m);
  double best = 1e30;
  p.splits = 1;
  for (const SmallTile& t : kSmall) {
    if (few && t.mt > 1) break;
    // tiles per CU; with many of them two blocks of K per wave hide the loads
    // better than more waves (128 rows, 64 experts of 2816 x 2048: 61 us with
    // four waves, 82 us with eight)
    const double tiles = i8_expected_tiles(p.m, p.groups, 16 * t.mt) *
                         (double)((p.n + 16 * t.nt - 1) / (16 * t.nt)) / 256.0;
    const int64_t waves =
        tiles > 4 ? std::clamp<int64_t>(nb / 2, 1, 8) : std::min<int64_t>(nb, 8);
    const double us = t.fixed + std::max(codes, t.step * (double)((nb + waves - 1) / waves) +
                                                    t.share * std::max(0.0, tiles - t.enough) *
                                                        (double)nb / 8.0 +
                                                    t.tile * tiles);
    if (us < best) {
      best = us;
      p.tile_m = 16 * t.mt;
      p.tile_n = 16 * t.nt;
      p.waves = (int)waves;
    }
  }
  for (const LargeTile& t : kLarge) {
    if (few) break;
    const double tiles =
        i8_expected_tiles(p.m, p.groups, t.rows) * (double)((p.n + G_BN - 1) / G_BN) / 256.0;
    for (int s : {1, 2, 3, 4, 6, 8, 12}) {
      if (s > nb || (s > 1 && t.bytes == 0)) break;
      double rounds = p.groups > 1 ? std::max(1.0, tiles * s + 0.3) : std::ceil(tiles * s);
      if (s > 1) rounds *= t.parts;
      double us = t.fixed + std::max(codes, rounds * (t.tile + t.stage * (double)p.k / 128.0 / s));
      if (s > 1) us += t.join + (double)p.m * (double)p.n * s * 4e-6 / t.bytes;
      if (us < best) {
        best = us;
        p.tile_m = t.rows;
        p.tile_n = G_BN;
        p.splits = s;
      }
    }
  }
}

}  // namespace

// Row tiles of tile_m rows that `groups` groups of m rows together can have.
int64_t i8_tile_bound(int64_t m, int groups, int tile_m) {
  const int64_t used = std::min<int64_t>(groups, m);
  return groups <= 1 ? (m + tile_m - 1) / tile_m : (m + used * (tile_m - 1)) / tile_m;
}

// Row tiles to expect: of exponentially distributed group sizes (experts are
// loaded unevenly), the mean of ceil(size / tile_m) times the groups.
double i8_expected_tiles(int64_t m, int groups, int tile_m) {
  if (groups <= 1) return (double)((m + tile_m - 1) / tile_m);
  const double used = (double)std::max<int64_t>(1, std::min<int64_t>(groups, m));
  return used / (1.0 - std::exp(-(double)tile_m * used / (double)std::max<int64_t>(m, 1)));
}

// Row tile and K slices of the rank-r projection: 32-row tiles from 64 rows per
// group on (they read the factor half as often), and enough slices for 4096
// waves, at least one 256-column block per wave and at most four (the
// contraction reads t once per slice: two slices instead of eight take 9 us off
// 4480 x 16384 x 6144), except for the few tiles of small calls.
void i8_project_plan(int64_t m, int groups, int64_t cols, int waves, int rank, int* t_rows,
                     int* slices) {
  const int64_t used = std::max<int64_t>(1, std::min<int64_t>(groups, m));
  *t_rows = m / used >= 64 ? 32 : 16;
  const int64_t tiles = i8_tile_bound(m, groups, *t_rows), blocks = (cols + 255) / 256;
  const int64_t most = std::min<int64_t>((blocks + waves - 1) / waves, tiles < 16 ? 64 : 4);
  *slices = rank ? (int)std::max<int64_t>(1, std::min(most, 4096 / (tiles * waves) + 1)) : 0;
}

W8A8Plan plan_w8a8(int64_t m, int64_t n, int64_t k, int groups, int rank) {
  W8A8Plan p{};
  p.m = m; p.n = n; p.k = k; p.groups = groups; p.rank = rank;
  // Rows and waves of a pre-phase workgroup: four lanes per 256-value block,
  // 16 blocks per wave.  Among 1 to 4 waves the count that leaves the fewest
  // lanes idle (K = 6144: 2 rows on 3 waves, none idle); rows of more than 64
  // blocks take a workgroup each.
  const int64_t nb = k / 256;
  int rows = 1, waves = (int)((nb + 15) / 16);
  double best = 0.0;
  for (int w = 1; w <= 4; ++w) {
    const int64_t r = std::min<int64_t>({16 * w / nb, PREP_MAX_ROWS, m});
    if (r < 1) continue;
    const double use = (double)(r * nb) / (16.0 * w);
    if (use > best - 1e-9) {   // of equals the larger: t has few workgroups otherwise
      best = use;
      rows = (int)r;
      waves = w;
    }
  }
  p.prep_rows = rows;
  p.prep_waves = waves;
  choose_tile(p);
  i8_project_plan(m, groups, k, waves, rank, &p.t_rows, &p.slices);
  size_t off = 0;
  p.off_xq = off; off = align256(off + (size_t)m * k);
  p.off_xs = off; off = align256(off + (size_t)m * 4);
  p.off_t = off;  off = align256(off + (size_t)p.slices * m * rank * 4);
  p.off_part = off; off = align256(off + (p.splits > 1 ? (size_t)p.splits * m * n * 4 : 0));
  p.total = off;
  return p;
}

hipError_t launch_w8a8(const W8A8Plan& p, const uint16_t* x, const int32_t* offsets,
                       const int8_t* codes, const uint16_t* scales, const uint16_t* up,
                       const uint16_t* down, void* y, int y_bf16, void* workspace,
                       hipStream_t stream) {
  char* base = static_cast<char*>(workspace);
  int8_t* xq = reinterpret_cast<int8_t*>(base + p.off_xq);
  float* xs = reinterpret_cast<float*>(base + p.off_xs);
  float* t = reinterpret_cast<float*>(base + p.off_t);
  const int m = (int)p.m, n = (int)p.n, k = (int)p.k;
  const int64_t qwgs = (p.m + p.prep_rows - 1) / p.prep_rows;
  const int64_t twgs = i8_tile_bound(p.m, p.groups, p.t_rows) * p.slices;
  const size_t lds = (size_t)p.prep_waves * 64 * p.rank;
#define SQ_W8A8_PREP(RW)                                                                        \
  hipLaunchKernelGGL((k_w8a8_prep<RW>), dim3((unsigned)(qwgs + twgs)), dim3(64 * p.prep_waves), \
                     lds, stream, x, down, offsets, p.groups, xq, xs, t, m, k, p.rank,          \
                     p.prep_rows, (int)twgs, p.slices)
  if (p.t_rows == 16) SQ_W8A8_PREP(1);
  else SQ_W8A8_PREP(2);
#undef SQ_W8A8_PREP
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int most_tiles = (int)i8_tile_bound(p.m, p.groups, p.tile_m);
  const int64_t tiles = most_tiles * ((p.n + p.tile_n - 1) / p.tile_n);
  if (p.tile_n <= 64) {
    const size_t slds = (size_t)3 * (p.rank / 8) * p.tile_m * 16 +
                        (size_t)p.waves * (p.tile_m / 16) * (p.tile_n / 16) * 1024;
#define SQ_W8A8_STREAM(MT, NT, U)                                                                 \
  hipLaunchKernelGGL((k_w8a8_stream<MT, NT, U>), dim3((unsigned)tiles), dim3(64 * p.waves), slds, \
                     stream, xq, xs, t, codes, scales, up, offsets, p.groups, y, m, n, k, p.rank, \
                     p.slices, y_bf16, most_tiles)
    if (p.tile_n == 16) SQ_W8A8_STREAM(1, 1, 4);
    else if (p.tile_m == 16) SQ_W8A8_STREAM(1, 2, 4);
    else if (p.tile_m == 32) SQ_W8A8_STREAM(2, 4, 2);
    else SQ_W8A8_STREAM(4, 4, 2);
#undef SQ_W8A8_STREAM
    return hipGetLastError();
  }
  int32_t* part = reinterpret_cast<int32_t*>(base + p.off_part);
#define SQ_W8A8_GEMM(FM, SPLIT)                                                                    \
  hipLaunchKernelGGL((k_w8a8_gemm<FM, SPLIT>), dim3((unsigned)(tiles * p.splits)),                 \
                     dim3(G_THREADS), 0, stream, xq, xs, t, codes, scales, up, offsets, p.groups,  \
                     y, m, n, k, p.rank, p.slices, y_bf16, most_tiles, p.splits, part)
  if (p.splits > 1) {
    if (p.tile_m == 128) SQ_W8A8_GEMM(4, true);
    else SQ_W8A8_GEMM(2, true);
  } else if (p.tile_m == 256) SQ_W8A8_GEMM(8, false);
  else if (p.tile_m == 224) SQ_W8A8_GEMM(7, false);
  else if (p.tile_m == 128) SQ_W8A8_GEMM(4, false);
  else SQ_W8A8_GEMM(2, false);
#undef SQ_W8A8_GEMM
  if (p.splits > 1) {
    if ((err = hipGetLastError()) != hipSuccess) return err;
    hipLaunchKernelGGL(k_w8a8_join,
                       dim3((unsigned)(i8_tile_bound(p.m, p.groups, 16) * ((p.n + 63) / 64))),
                       dim3(256), 0, stream, part, xs, t, scales, up, offsets, p.groups, y, m, n,
                       p.rank, p.slices, y_bf16, p.splits);
  }
  return hipGetLastError();
}

}  // namespace sq
