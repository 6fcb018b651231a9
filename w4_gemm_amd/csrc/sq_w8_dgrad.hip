// Input gradient of the int8 mode, for one layer and for experts:
//
//   dx = dy W_hat = ((dy w) c) H + (dy up) down^T
//
// with c, w the payload's codes and row scales (H H = I moves the rotation to
// the output).  Gradients keep more bits than the forward's tokens: each row
// of v = fp32(dy w) is held as 16-bit integers
//   a = max(max_n |v|, 2^-100), t = fp32(a / 32512), i = fp32(32512 / a)
//   d = round_half_even(fp32(v i)) = 256 hi + lo,   |hi| <= 127, -128 <= lo < 128
// (a step of 2^-15 of the row's largest value: finer than fp16's 2^-11 of each
// value down to 2^-4 of the largest, coarser below; relative error of dx over
// 4096 x 1024, fp16 rows in brackets: Gaussian rows 3.5e-5 [2.1e-4], Student t
// with 2 degrees of freedom 2.3e-4 [1.9e-4], one column x 1000 5.6e-4 [2.1e-5],
// softmax minus one-hot 5.4e-4 [1.7e-5]; a bf16 W_hat or dx has 1.7e-3), and
// the product runs as two 8-bit ones on
// v_mfma_i32_16x16x64_i8 that share each fragment of c: it costs what one
// fp16 product costs and converts no codes.  The sums are exact in int32 for
// N <= 131072: hi's stay below 127 * 128 * 131072 < 2^31, lo's reach
// 128 * 128 * 131072 = 2^31 at that N alone, where the product mends the one
// sum that wraps.  A row that holds inf or NaN (or meets a scale that is)
// gives a row of NaN.
//
// Kernels:
//   k_w8_dgrad_prep  hi, lo, t of every row, and the N slices of dy up
//   k_w8_dgrad_gemm  (256 hi + lo) c, the 256-point transform of each block
//                    of 256 columns, the scale and the rank-r branch
//   k_w8_dgrad_join  the same end for the sums of several N splits
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "sq_i8.hpp"
#include "sq_kernels.h"

namespace sq {
namespace {

// ---------------------------------------------------------------- pre-phase
constexpr int DP_THREADS = 256;

// The first workgroups compute the rank-r projection (they run longest); the
// others hold 4 / WPR rows each, WPR waves per row.  d is [m][npad / 64][hi 64 |
// lo 64], zero past n: one 128-byte line holds both halves of 64 values.
// A thread keeps the first HELD groups of eight values of its row in registers
// between the two passes (longer rows are read again, and so are rows whose
// length is no multiple of eight, which keep none).
// VEC: n is a multiple of eight (rows are 16-byte aligned then).  RANK (16 also
// where there are no factors): the projection's registers set how many waves a
// SIMD holds, the rows' too: 8192 x 2816 takes 28 us at rank 16, 38 us in a
// kernel that has rank 64 in it as well.
template <int RANK, int RW, bool VEC, int WPR, int HELD>
__global__ void __launch_bounds__(DP_THREADS) k_w8_dgrad_prep(
    const uint16_t* __restrict__ dy, const uint16_t* __restrict__ scales,
    const uint16_t* __restrict__ up, const int32_t* __restrict__ offsets, int groups,
    int8_t* __restrict__ d, float* __restrict__ ts, float* __restrict__ t_part, int m, int n,
    int npad, int project_wgs, int slices) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  const int tid = threadIdx.x, lane = tid & 63;
  if ((int)blockIdx.x < project_wgs) {
    project<RANK, RW, VEC>(dy, up, offsets, groups, t_part, dyn, m, n, blockIdx.x, slices);
    return;
  }
  __shared__ uint32_t row_max[4];
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = ((int)blockIdx.x - project_wgs) * (4 / WPR) + (WPR == 1 ? wave : 0);
  const int first = WPR == 1 ? lane * 8 : tid * 8;
  constexpr int STEP = WPR * 64 * 8;
  const int grp = row < m ? group_of_row(offsets, groups, row, lane) : -1;
  // rows behind the last group are not read by the product either; the whole
  // workgroup (WPR 4) or wave (WPR 1) leaves together
  if (grp < 0) return;
  const uint16_t* src = dy + (int64_t)row * n;
  const uint16_t* sc = scales + (int64_t)grp * n;
  auto load8 = [&](const uint16_t* p, int c) {   // zeros past n
    if constexpr (VEC) {
      u32x4 v = {0u, 0u, 0u, 0u};
      if (c < n) v = *reinterpret_cast<const u32x4*>(p + c);
      return v;
    } else {
      return load8_u16(p + c, n - c);
    }
  };
  auto times_scale = [&](u32x4 v, int c, float (&o)[8]) {
    const u32x4 s = load8(sc, c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(v[i] << 16) * fp16_bits_to_f32(s[i] & 0xFFFFu);
      o[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u) * fp16_bits_to_f32(s[i] >> 16);
    }
  };
  // largest magnitude as bits: infinities and NaN order above every finite value
  uint32_t mx = 0;
  u32x4 held[HELD > 0 ? HELD : 1];
#pragma unroll
  for (int h = 0; h < HELD; ++h) held[h] = load8(src, first + h * STEP);
#pragma unroll
  for (int h = 0; h < HELD; ++h) {
    float v[8];
    times_scale(held[h], first + h * STEP, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  }
  for (int c = first + HELD * STEP; c < n; c += STEP) {
    float v[8];
    times_scale(load8(src, c), c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, s));
  if (WPR > 1) {
    if (lane == 0) row_max[wave] = mx;
    __syncthreads();
    mx = max(max(row_max[0], row_max[1]), max(row_max[2], row_max[3]));
  }
  const bool finite = mx < 0x7F800000u;
  const float a = fmaxf(__uint_as_float(mx), I8_MIN_ABSMAX);
  const float inv = 32512.0f / a;
  if (first == 0) ts[row] = finite ? a / 32512.0f : __uint_as_float(I8_NAN_BITS);
  int8_t* dst = d + (int64_t)row * 2 * npad;
  auto put = [&](u32x4 raw, int c) {
    float v[8];
    times_scale(raw, c, v);
    u32x2 oh, ol;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b[i] = finite ? __float_as_uint(v[4 * w + i] * inv + I8_ROUND) : 0u;
      // low 16 bits of the integer: lo in byte 0; hi in byte 1 once half a
      // step of hi is added
      ol[w] = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u) |
              __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
      oh[w] = __builtin_amdgcn_perm(b[1] + 128u, b[0] + 128u, 0x0C0C0501u) |
              __builtin_amdgcn_perm(b[3] + 128u, b[2] + 128u, 0x05010C0Cu);
    }
    int8_t* o = dst + 2 * (c & ~63) + (c & 63);
    *reinterpret_cast<u32x2*>(o) = oh;
    *reinterpret_cast<u32x2*>(o + 64) = ol;
  };
#pragma unroll
  for (int h = 0; h < HELD; ++h)
    if (first + h * STEP < npad) put(held[h], first + h * STEP);
  for (int c = first + HELD * STEP; c < npad; c += STEP) put(load8(src, c), c);
}

// ---------------------------------------------------------------- contraction
// BM x 256 output tile (BM = 32 FM; 256 columns are one Hadamard block) per
// workgroup, eight waves of 16 FM x 64.  One stage = 64 rows of c: their 256
// code bytes (16 KB) and the 128 bytes of hi and lo of each row of d, four
// stages in LDS.  Both stream global -> LDS with direct 16-byte buffer loads.
//   rows of d: chunk c of row r at slot c ^ (r & 7);
//   code rows: chunk c of row r at slot c ^ b_swz(r).  A fragment of c needs 16
//   consecutive n of one column per lane: two transposed reads, each of eight
//   rows x 16 columns per 16 lanes (lane 2j + h points at row j, columns
//   8h..8h+7; lane i receives column i).  b_swz spreads the 32 rows that one
//   instruction touches over all sixteen 16-byte slots of a row (without it a
//   loop of these reads takes 12 times as long).
constexpr int D_BN = 256, D_THREADS = 512;
constexpr int D_B = 16 * 1024, D_STAGE = 32 * 1024;   // code rows behind the rows of d
__shared__ __attribute__((aligned(16))) uint8_t d_buf0[D_STAGE];
__shared__ __attribute__((aligned(16))) uint8_t d_buf1[D_STAGE];
__shared__ __attribute__((aligned(16))) uint8_t d_buf2[D_STAGE];
__shared__ __attribute__((aligned(16))) uint8_t d_buf3[D_STAGE];

__device__ __forceinline__ int b_swz(int r) { return (r & 7) | (((r >> 4) & 1) << 3); }
// 16-byte unit u (of 64) of a row of 256 fp32 sums in the epilogue
__device__ __forceinline__ int c_unit(int row, int u) { return u ^ (row & 15); }
// 32 rows of 256 fp32 sums per LDS object
__device__ __forceinline__ uint8_t* c_rows(int block32) {
  return block32 == 0 ? d_buf0 : block32 == 1 ? d_buf1 : block32 == 2 ? d_buf2 : d_buf3;
}

template <int FM>
__global__ void __launch_bounds__(D_THREADS, 1) k_w8_dgrad_gemm(
    const int8_t* __restrict__ d, const float* __restrict__ ts, const float* __restrict__ t_part,
    const int8_t* __restrict__ codes, const uint16_t* __restrict__ down,
    const int32_t* __restrict__ offsets, int groups, void* __restrict__ dx, int m, int n, int npad,
    int k, int rank, int slices, int dx_bf16, int most_tiles, int max_split,
    int64_t* __restrict__ partial) {
  constexpr int FN = 4, BM = 32 * FM;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int fr = lane & 15, g = lane >> 4;
  const int nt = k / D_BN;
  const int mt = row_tile_count(offsets, groups, m, BM, most_tiles, lane);
  // workgroup b: tile b, or part (b - full) / rem of tile full + (b - full) % rem
  const int tiles = mt * nt;
  const Tail tail = tile_tail(tiles, max_split);
  int lin = blockIdx.x, split = 0, splits = 1;
  if (lin >= tail.full) {
    if (tail.full == tiles) return;
    splits = __builtin_amdgcn_readfirstlane(tail.splits);
    split = __builtin_amdgcn_readfirstlane((lin - tail.full) / (tiles - tail.full));
    if (split >= splits) return;
    lin -= split * (tiles - tail.full);
  }
  int64_t tm, tn;
  xcd_tile(lin, tiles, nt, tm, tn);
  RowTile rt;
  if (!find_row_tile(offsets, groups, m, BM, __builtin_amdgcn_readfirstlane((int)tm), lane, rt))
    return;
  const int grp = __builtin_amdgcn_readfirstlane(rt.group);
  const int rows = __builtin_amdgcn_readfirstlane(rt.rows);
  const int64_t m0 = __builtin_amdgcn_readfirstlane(rt.row0);
  const int k0 = __builtin_amdgcn_readfirstlane((int)tn) * D_BN;
  // stages of 64 rows of c: a multiple of four (the splits cut npad in 256s)
  const int nb = npad >> 8;
  const int st0 = 4 * __builtin_amdgcn_readfirstlane((int)((int64_t)split * nb / splits));
  const int ST = 4 * __builtin_amdgcn_readfirstlane((int)((int64_t)(split + 1) * nb / splits)) - st0;

  // loaders: instruction i of wave w fills rows 8 (8 i + w) .. +8 of d (128
  // bytes each) and code rows 4 (8 i + w) .. +4, through descriptors of 64 and
  // 32 rows; rows of d past the tile and code rows past n lie beyond them and
  // fetch nothing (there d is zero or unused)
  const int la = 8 * wave + (lane >> 3), lb = 4 * wave + (lane >> 4);
  const uint32_t off_a = (uint32_t)la * (uint32_t)(2 * npad) + 16u * (uint32_t)((lane & 7) ^ (la & 7));
  const uint32_t off_b = (uint32_t)lb * (uint32_t)k + 16u * (uint32_t)((lane & 15) ^ b_swz(lb));
  const int8_t* a_base = d + m0 * 2 * npad;
  const int8_t* b_base = codes + (int64_t)grp * n * k + k0;
  auto issue = [&](int st, uint8_t* buf) {
    const int n0 = (st0 + st) * 64;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (64 * i < BM) {
        const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
            (void*)(a_base + (int64_t)(64 * i) * 2 * npad), (short)0,
            max(rows - 64 * i, 0) * 2 * npad, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(a_rsrc, (i8_lds_t)(buf + (8 * i + wave) * 1024), 16,
                                                 off_a, 2 * n0, 0, 0);
      }
      const int left = min(max(n - n0 - 32 * i, 0), 32);
      const __amdgpu_buffer_rsrc_t b_rsrc = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(b_base + (int64_t)(n0 + 32 * i) * k), (short)0,
          left > 0 ? (left - 1) * k + D_BN : 0, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          b_rsrc, (i8_lds_t)(buf + D_B + (8 * i + wave) * 1024), 16, off_b, 0, 0, 0);
    }
  };
  constexpr int LOADS = BM > 64 ? 4 : 3;   // per stage and wave
  issue(0, d_buf0);
  issue(1, d_buf1);
  issue(2, d_buf2);
  issue(3, d_buf3);

  // fragments (16-row tile i of wave row wm is tile 2 i + wm of the workgroup):
  // hi chunks g, lo chunks 4 + g of row fr; transposed read u of
  // column tile j: row 16 g + 8 u + fr / 2, columns 64 wn + 16 j + 8 (fr & 1)
  const uint32_t a_row = (uint32_t)(16 * wm + fr) * 128;
  const int tr_row = 16 * g + (fr >> 1);
  const uint32_t b_row = D_B + (uint32_t)tr_row * 256 + 8u * (uint32_t)(fr & 1);
  const int tr_swz = b_swz(tr_row);
  // The epilogue's row scale and first ranks of t, where the registers allow:
  // wave w ends up with rows 16 w + fr.  The 32-wide MFMA takes rank 16 twice:
  // lane groups 0, 1 carry one part of t, groups 2, 3 the next.
  constexpr bool EARLY = FM == 2;
  const bool twice = rank == 16;
  const uint16_t* down0 = down + ((int64_t)grp * k + k0) * rank;
  float early_s = 0.0f;
  u32x4 early_t[3] = {};
  if (EARLY && 16 * wave < rows) {
    const int er = (int)m0 + min(16 * wave + fr, rows - 1);
    early_s = ts[er];
    const int r0 = twice ? 8 * (g & 1) : 8 * g;
    if (rank > 0) project_sum8(t_part, m, rank, slices, er, r0, early_t);
  }

  i32x4 ah[FM][FN], al[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) ah[i][j] = al[i][j] = (i32x4){0, 0, 0, 0};
  auto sync = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(sq_wait_vm(2 * LOADS));
    __builtin_amdgcn_s_waitcnt(SQ_WAIT_LGKM0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  __builtin_amdgcn_s_waitcnt(sq_wait_vm(3 * LOADS));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  // the loop over the first F of the wave's FM row tiles
  auto contract = [&](auto count) {
    constexpr int F = decltype(count)::value;
    struct Frag {
      i32x4 h[F], l[F], b[FN];
    };
    auto read = [&](Frag& f, const uint8_t* buf) {
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        i32x2 p[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          p[u] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (__attribute__((address_space(3))) i32x2*)(buf + b_row + u * 2048 +
                                                         16 * ((4 * wn + j) ^ tr_swz)));
        f.b[j] = (i32x4){p[0][0], p[0][1], p[1][0], p[1][1]};
      }
#pragma unroll
      for (int i = 0; i < F; ++i) {
        f.h[i] = *reinterpret_cast<const i32x4*>(buf + a_row + i * 4096 + 16 * (g ^ (fr & 7)));
        f.l[i] = *reinterpret_cast<const i32x4*>(buf + a_row + i * 4096 + 16 * ((4 + g) ^ (fr & 7)));
      }
    };
    auto compute = [&](const Frag& f) {
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          ah[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.h[i], f.b[j], ah[i][j], 0, 0, 0);
          al[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.l[i], f.b[j], al[i][j], 0, 0, 0);
        }
    };
    // 2 F + 8 LDS reads and four global loads among 8 F MFMAs
    auto interleave = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, F, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, F, 0);
      }
    };
    // One stage: stage s sits in registers; at the barrier every wave has read
    // it, so its buffer takes stage s + 4, and stage s + 1 has landed (the two
    // after it are still on their way); the fragments of stage s + 1 are read
    // under the MFMAs of stage s.  Loads past the last stage fetch the last one
    // again, into buffers that are not read any more.
    auto step = [&](int s, const Frag& cur, Frag& nxt, uint8_t* buf, const uint8_t* next) {
      sync();
      issue(min(s + 4, ST - 1), buf);
      read(nxt, next);
      compute(cur);
      interleave();
    };
    Frag f0, f1;
    read(f0, d_buf0);
    for (int s = 0; s < ST; s += 4) {
      step(s, f0, f1, d_buf0, d_buf1);
      step(s + 1, f1, f0, d_buf1, d_buf2);
      step(s + 2, f0, f1, d_buf2, d_buf3);
      step(s + 3, f1, f0, d_buf3, d_buf0);
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
  // A low sum of 2^31 (every lo and every code -128: a row below the absmax
  // floor) has wrapped to INT32_MIN, which no other sum gives, as none is below
  // -127 * 128 * 131072.  256 of it move over to the high sum.
  if (n == I8_DGRAD_MAX_N) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (al[i][j][v] == INT32_MIN) {
            al[i][j][v] = INT32_MAX - 255;
            ah[i][j][v] += 1;
          }
  }

  // lane (fr, g) holds rows 4g + v and column fr of each 16 x 16 tile
  if (splits > 1) {
    // partial [part][tail tile][BM][256]
    int64_t* dst = partial + ((int64_t)split * (tiles - tail.full) + lin - tail.full) * (BM * 256);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 32 * i + 16 * wm + 4 * g + v;
        if (r >= rows) continue;
#pragma unroll
        for (int j = 0; j < FN; ++j)
          dst[r * 256 + 64 * wn + 16 * j + fr] = (int64_t)ah[i][j][v] * 256 + al[i][j][v];
      }
    return;
  }
  // Rank-r branch: output row 4g' + i of tile qp = 4 q + p of its MFMAs is column
  // 64 q + 16 g' + 4 p + i.  down's rows of the first 32 ranks come in under the
  // exchange and the transform where the registers allow (1001 x 2051 x 4096,
  // rank 64: 36 -> 32 us; with 128 rows they spill).
  const int dcol = 16 * (fr >> 2) + (fr & 3);
  const int trow = (int)m0 + min(16 * wave + fr, rows - 1);
  auto rank0 = [&](int rr) { return twice ? 8 * (g & 1) : rr + 8 * g; };
  auto down8 = [&](int qp, int rr) {
    const uint16_t* base = down0 + (64 * (qp >> 2) + 4 * (qp & 3)) * rank;
    return *reinterpret_cast<const u32x4*>(base + (uint32_t)(dcol * rank + rank0(rr)));
  };
  u32x4 dv[EARLY ? 16 : 1], part[3] = {early_t[0], early_t[1], early_t[2]};
  if (EARLY && rank > 0 && 16 * wave < rows) {
#pragma unroll
    for (int qp = 0; qp < 16; ++qp) dv[qp] = down8(qp, 0);
  }
  __syncthreads();   // every wave is done with the stage buffers
  // Sums in fp32.  Column bits: fr 0-3, j 4-5, wn 6-7.  The butterflies over j
  // run here, the others after the exchange.
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    uint8_t* st = c_rows(i);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = (float)ah[i][j][v] * 256.0f + (float)al[i][j][v];
      const float s0 = c[0] + c[1], s1 = c[0] - c[1], s2 = c[2] + c[3], s3 = c[2] - c[3];
      const float o[4] = {s0 + s2, s1 + s3, s0 - s2, s1 - s3};
      const int row = 16 * wm + 4 * g + v;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float*>(st + row * 1024 + 16 * c_unit(row, 16 * wn + 4 * j + (fr >> 2)) +
                                  4 * (fr & 3)) = o[j];
    }
  }
  __syncthreads();
  // wave w takes rows 16w .. 16w+15: lane (fr, g) owns row 16w + fr and the
  // columns with j = g: w[16 q + p] is column 64 q + 16 g + p
  if (16 * wave >= min(rows, BM)) return;
  float w[64];
  {
    const uint8_t* st = c_rows(wave >> 1);
    const int row = 16 * (wave & 1) + fr;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const f32x4 f = *reinterpret_cast<const f32x4*>(st + row * 1024 +
                                                        16 * c_unit(row, 16 * q + 4 * g + p));
#pragma unroll
        for (int i = 0; i < 4; ++i) w[16 * q + 4 * p + i] = f[i];
      }
  }
#pragma unroll
  for (int h = 1; h < 64; h <<= 1)
#pragma unroll
    for (int i = 0; i < 64; ++i)
      if ((i & h) == 0) {
        const float a = w[i], b = w[i + h];
        w[i] = a + b;
        w[i + h] = a - b;
      }
  const int row = 16 * wave + fr;
  const float f = (EARLY ? early_s : ts[trow]) * 0.0625f;
#pragma unroll
  for (int i = 0; i < 64; ++i) w[i] *= f;
  // rank-r branch with the columns as MFMA rows, MFMA column fr the lane's row
  for (int rr = 0; rr < rank; rr += 32) {
    if (!EARLY || rr > 0) project_sum8(t_part, m, rank, slices, trow, rank0(rr), part);
    if (EARLY && rr > 0) {
#pragma unroll
      for (int qp = 0; qp < 16; ++qp) dv[qp] = down8(qp, rr);
    }
    if (twice && g >= 2) {
      part[0] = part[1];
      part[1] = (u32x4){0u, 0u, 0u, 0u};
    } else if (twice) {
      part[1] = part[2];
    }
#pragma unroll
    for (int qp = 0; qp < 16; ++qp) {
      const bf16x8 dn = __builtin_bit_cast(bf16x8, EARLY ? dv[qp] : down8(qp, rr));
      f32x4 acc = {w[4 * qp], w[4 * qp + 1], w[4 * qp + 2], w[4 * qp + 3]};
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dn, __builtin_bit_cast(bf16x8, part[0]), acc, 0, 0, 0);
      if (!twice || !dx_bf16)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dn, __builtin_bit_cast(bf16x8, part[1]), acc, 0, 0, 0);
      if (!twice && !dx_bf16)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dn, __builtin_bit_cast(bf16x8, part[2]), acc, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[4 * qp + i] = acc[i];
    }
  }
  if (dx_bf16) {
    if (row >= rows) return;
    uint16_t* dst = reinterpret_cast<uint16_t*>(dx) + (m0 + row) * k + k0 + 16 * g;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = pack_bf16x2(w[16 * q + 8 * h + 2 * i], w[16 * q + 8 * h + 2 * i + 1]);
        *reinterpret_cast<u32x4*>(dst + 64 * q + 8 * h) = o;
      }
    return;
  }
  // fp32 goes back through the wave's own 16 rows of LDS, so that a store covers
  // a whole row (1001 x 2051 x 4096: 28 -> 24.6 us; bf16 gains nothing by it)
  int wr = fr;
  asm volatile("" : "+v"(wr));   // addresses worked out again, not held since the exchange
  uint8_t* st = c_rows(wave >> 1) + 16 * (wave & 1) * 1024;
#pragma unroll
  for (int qp = 0; qp < 16; ++qp)
    *reinterpret_cast<f32x4*>(st + wr * 1024 + 16 * c_unit(wr, 16 * (qp >> 2) + 4 * g + (qp & 3))) =
        (f32x4){w[4 * qp], w[4 * qp + 1], w[4 * qp + 2], w[4 * qp + 3]};
  __builtin_amdgcn_s_waitcnt(SQ_WAIT_LGKM0);
  __builtin_amdgcn_wave_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  float* dst = reinterpret_cast<float*>(dx) + (m0 + 16 * wave) * k + k0 + 4 * lane;
#pragma unroll
  for (int r = 0; r < 16; ++r)
    if (r < rows - 16 * wave)
      *reinterpret_cast<f32x4*>(dst + (int64_t)r * k) =
          *reinterpret_cast<const f32x4*>(st + r * 1024 + 16 * c_unit(r, lane));
}

// Sum of the parts' integers of the tail tiles (exact: below 2^45), transform,
// scale and rank-r branch.  One wave per row and block of 256 columns, four
// columns per lane; blockIdx.x / (BM / 4) is the tail tile.
__global__ void __launch_bounds__(256) k_w8_dgrad_join(
    const int64_t* __restrict__ partial, const float* __restrict__ ts,
    const float* __restrict__ t_part, const uint16_t* __restrict__ down,
    const int32_t* __restrict__ offsets, int groups, void* __restrict__ dx, int m, int k, int rank,
    int slices, int dx_bf16, int max_split, int tile_m, int most_tiles) {
  __shared__ float t_lds[4][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nt = k >> 8, tiles = row_tile_count(offsets, groups, m, tile_m, most_tiles, lane) * nt;
  const Tail tail = tile_tail(tiles, max_split);
  const int splits = tail.splits, rem = tiles - tail.full;
  const int tail_tile = (int)blockIdx.x / (tile_m / 4);
  if (tail_tile >= rem) return;
  int64_t tm, tn;
  xcd_tile(tail.full + tail_tile, tiles, nt, tm, tn);
  RowTile rt;
  if (!find_row_tile(offsets, groups, m, tile_m, __builtin_amdgcn_readfirstlane((int)tm), lane, rt))
    return;
  const int grp = rt.group, lrow = ((int)blockIdx.x % (tile_m / 4)) * 4 + wave;
  if (lrow >= rt.rows) return;
  const int row = rt.row0 + lrow, c0 = (int)tn * 256 + 4 * lane;
  typedef int64_t i64x2 __attribute__((ext_vector_type(2)));
  int64_t s[4] = {};
  for (int sp = 0; sp < splits; sp += 4) {
    i64x2 p[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const i64x2* src = reinterpret_cast<const i64x2*>(
          partial + (((int64_t)min(sp + u, splits - 1) * rem + tail_tile) * tile_m + lrow) * 256 +
          4 * lane);
      p[u][0] = src[0];
      p[u][1] = src[1];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (sp + u < splits)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += p[u][i >> 1][i & 1];
  }
  for (int r = lane; r < rank; r += 64) {
    float t = 0.0f;
    for (int sl = 0; sl < slices; sl += 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = t_part[((int64_t)min(sl + u, slices - 1) * m + row) * rank + r];
#pragma unroll
      for (int u = 0; u < 8; ++u) t += sl + u < slices ? v[u] : 0.0f;
    }
    t_lds[wave][r] = t;   // read by this wave only
  }
  float c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = (float)s[i];
  const float s0 = c[0] + c[1], s1 = c[0] - c[1], s2 = c[2] + c[3], s3 = c[2] - c[3];
  c[0] = s0 + s2; c[1] = s1 + s3; c[2] = s0 - s2; c[3] = s1 - s3;
#pragma unroll
  for (int h = 1; h < 64; h <<= 1) {
    const float sg = (lane & h) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __builtin_fmaf(sg, c[i], __shfl_xor(c[i], h));
  }
  const float f = ts[row] * 0.0625f;
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] *= f;
  __builtin_amdgcn_s_waitcnt(SQ_WAIT_LGKM0);
  __builtin_amdgcn_wave_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  for (int r0 = 0; r0 < rank; r0 += 8) {
    const f32x4 ta = *reinterpret_cast<const f32x4*>(&t_lds[wave][r0]);
    const f32x4 tb = *reinterpret_cast<const f32x4*>(&t_lds[wave][r0 + 4]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4 u =
          *reinterpret_cast<const u32x4*>(down + ((int64_t)grp * k + c0 + j) * rank + r0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float t0 = i < 2 ? ta[2 * i] : tb[2 * i - 4], t1 = i < 2 ? ta[2 * i + 1] : tb[2 * i - 3];
        c[j] = __builtin_fmaf(t0, __uint_as_float(u[i] << 16), c[j]);
        c[j] = __builtin_fmaf(t1, __uint_as_float(u[i] & 0xFFFF0000u), c[j]);
      }
    }
  }
  const int64_t at = (int64_t)row * k + c0;
  if (dx_bf16)
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(dx) + at) =
        (u32x2){pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3])};
  else
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(dx) + at) = (f32x4){c[0], c[1], c[2], c[3]};
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// Rows of the tile and parts of a tail tile, by modelled time (us): rounds of a
// fixed part and one part per stage, and for split tails the partial sums' trip
// through memory.  The constants are fitted to 9200 timed shapes, over which the
// choice takes 1.009 times the best form.  Both sides measured: 512 x 4096 x 4096
// 40 us with 64 rows, 51 with 128; 4480 x 16384 x 6144 866 and 751 (795 without
// parts); 1 x 16384 x 6144 34 us in 8 parts, 107 whole; 2000 x 1000 x 8192 64 and 60.
struct DgradTile {
  int rows;
  double tile, stage;   // us per round, us per stage of 64 and round
};
constexpr DgradTile kTiles[] = {{64, 8.5, 0.46}, {128, 17.0, 0.67}};

void choose_tile(W8DgradPlan& p) {
  const double stages = (double)p.npad / 64.0;
  const int64_t nb = p.npad / 256;
  double best = 1e30;
  for (const DgradTile& t : kTiles) {
    const double rows_each = (double)p.m / std::max<int64_t>(1, std::min<int64_t>(p.groups, p.m));
    const double tiles = i8_expected_tiles(p.m, p.groups, t.rows) * (double)(p.k / D_BN);
    const double whole = std::floor(tiles / I8_CUS), rem = tiles - whole * I8_CUS;
    for (int s : {1, 2, 4, 8, 16}) {
      if (s > nb) break;
      const double parts = rem > 0 ? std::max(1.0, std::min<double>(s, std::floor(I8_CUS / rem))) : 1;
      double us = whole * (t.tile + stages * t.stage);
      if (rem > 0) us += t.tile + stages / parts * t.stage;
      // a launch and 16 bytes per partial sum
      if (s > 1) us += 3.8;
      if (parts > 1) us += 4.3 + rem * parts * std::min<double>(t.rows, rows_each) * 256 * 16 / 3.9e6;
      if (us < best) {
        best = us;
        p.tile_m = t.rows;
        p.max_split = s;
      }
    }
  }
}

}  // namespace

W8DgradPlan plan_w8_dgrad(int64_t m, int64_t n, int64_t k, int groups, int rank) {
  W8DgradPlan p{};
  p.m = m; p.n = n; p.k = k; p.groups = groups; p.rank = rank;
  p.npad = (n + 255) / 256 * 256;
  choose_tile(p);
  i8_project_plan(m, groups, n, DP_THREADS / 64, rank, &p.t_rows, &p.slices);
  size_t off = 0;
  p.off_d = off;  off = align256(off + (size_t)m * p.npad * 2);
  p.off_ts = off; off = align256(off + (size_t)m * 4);
  p.off_t = off;  off = align256(off + (size_t)p.slices * m * rank * 4);
  // partial sums of the tail: at most one tile per CU, and no more than all rows
  const size_t tiles = (size_t)i8_tile_bound(m, groups, p.tile_m) * (k / 256) * p.max_split;
  p.off_part = off;
  off = align256(off + (p.max_split > 1 ? std::min<size_t>(tiles, I8_CUS) * p.tile_m * 256 * 8 : 0));
  p.total = off;
  return p;
}

hipError_t launch_w8_dgrad(const W8DgradPlan& p, const uint16_t* dy, const int32_t* offsets,
                           const int8_t* codes, const uint16_t* scales, const uint16_t* up,
                           const uint16_t* down, void* dx, int dx_bf16, void* workspace,
                           hipStream_t stream) {
  char* base = static_cast<char*>(workspace);
  int8_t* d = reinterpret_cast<int8_t*>(base + p.off_d);
  float* ts = reinterpret_cast<float*>(base + p.off_ts);
  float* t = reinterpret_cast<float*>(base + p.off_t);
  const int m = (int)p.m, n = (int)p.n, k = (int)p.k, npad = (int)p.npad;
  // rows of up to 2048 values take one wave, longer ones four
  const int wpr = n <= 2048 ? 1 : 4;
  const int64_t qwgs = wpr == 1 ? (p.m + 3) / 4 : p.m;
  const int64_t twgs = i8_tile_bound(p.m, p.groups, p.t_rows) * p.slices;
  const size_t lds = (size_t)(DP_THREADS / 64) * 64 * p.rank;
#define SQ_W8DP(RANK, RW, VEC, WPR, HELD)                                                        \
  hipLaunchKernelGGL((k_w8_dgrad_prep<RANK, RW, VEC, WPR, HELD>), dim3((unsigned)(qwgs + twgs)), \
                     dim3(DP_THREADS), lds, stream, dy, scales, up, offsets, p.groups, d, ts, t, \
                     m, n, npad, (int)twgs, p.slices)
#define SQ_W8DP_ROWS(RANK, RW)                                  \
  do {                                                          \
    if (n % 8 != 0 && wpr == 1) SQ_W8DP(RANK, RW, false, 1, 0); \
    else if (n % 8 != 0) SQ_W8DP(RANK, RW, false, 4, 0);        \
    else if (n <= 512) SQ_W8DP(RANK, RW, true, 1, 1);           \
    else if (n <= 2048) SQ_W8DP(RANK, RW, true, 1, 4);          \
    else if (n <= 4096) SQ_W8DP(RANK, RW, true, 4, 2);          \
    else if (n <= 8192) SQ_W8DP(RANK, RW, true, 4, 4);          \
    else SQ_W8DP(RANK, RW, true, 4, 8);                         \
  } while (0)
#define SQ_W8DP_RANK(RANK)                   \
  do {                                       \
    if (p.t_rows == 16) SQ_W8DP_ROWS(RANK, 1); \
    else SQ_W8DP_ROWS(RANK, 2);              \
  } while (0)
  if (p.rank <= 16) SQ_W8DP_RANK(16);
  else if (p.rank == 32) SQ_W8DP_RANK(32);
  else SQ_W8DP_RANK(64);
#undef SQ_W8DP_RANK
#undef SQ_W8DP_ROWS
#undef SQ_W8DP
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  // the tail's parts are at most one per CU more than the tiles
  const int most_tiles = (int)i8_tile_bound(p.m, p.groups, p.tile_m);
  const int64_t bound = most_tiles * (p.k / D_BN);
  const int64_t tail_bound = std::min<int64_t>(bound, I8_CUS / 2);
  const int64_t tiles = p.max_split > 1 ? bound + std::min<int64_t>(bound * (p.max_split - 1), I8_CUS) : bound;
  int64_t* part = reinterpret_cast<int64_t*>(base + p.off_part);
#define SQ_W8DG(FM)                                                                               \
  hipLaunchKernelGGL((k_w8_dgrad_gemm<FM>), dim3((unsigned)tiles), dim3(D_THREADS), 0, stream, d, \
                     ts, t, codes, down, offsets, p.groups, dx, m, n, npad, k, p.rank, p.slices,  \
                     dx_bf16, most_tiles, p.max_split, part)
  if (p.tile_m == 128) SQ_W8DG(4);
  else SQ_W8DG(2);
#undef SQ_W8DG
  if ((err = hipGetLastError()) != hipSuccess) return err;
  // offsets may leave any number of tiles, so only the plan tells whether a tail can be cut
  if (p.max_split > 1) {
    hipLaunchKernelGGL(k_w8_dgrad_join, dim3((unsigned)(tail_bound * (p.tile_m / 4))), dim3(256), 0,
                       stream, part, ts, t, down, offsets, p.groups, dx, m, k, p.rank, p.slices,
                       dx_bf16, p.max_split, p.tile_m, most_tiles);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace sq
