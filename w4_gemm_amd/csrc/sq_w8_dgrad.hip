// Input gradient of the int8 mode, for one layer and for experts:
//
//   dx = dy W_hat = ((dy w) c) H + (dy up) down^T
//
// with c, w the payload's codes and row scales (H H = I moves the rotation to
// the output).  Gradients keep more bits than the forward's tokens: each row
// of v = fp32(dy w) is held as 16-bit integers
//   a = max(max_n |v|, 2^-100), t = fp32(a / 32512), i = fp32(32512 / a)
//   d = round_half_even(fp32(v i)) = 256 hi + lo,   |hi| <= 127, -128 <= lo < 128
// (a step of 2^-15 of the row's largest value, against fp16's 2^-11 of each
// value), and the product runs as two 8-bit ones on
// v_mfma_i32_16x16x64_i8 that share each fragment of c: it costs what one
// fp16 product costs and converts no codes.  The sums are exact in int32 for
// N <= 131072.  A row that holds inf or NaN (or meets a scale that is) gives
// a row of NaN.
//
// Kernels:
//   k_w8_dgrad_prep  hi, lo, t of every row, and the N slices of dy up
//   k_w8_dgrad_gemm  (256 hi + lo) c, the 256-point transform of each block
//                    of 256 columns, the scale and the rank-r branch
#include <algorithm>

#include "sq_i8.hpp"
#include "sq_kernels.h"

namespace sq {
namespace {

// ---------------------------------------------------------------- pre-phase
constexpr int DP_THREADS = 256;

// Workgroups 0 .. quant_wgs-1: WPR waves per row (1, or 4 for long rows); the
// rest compute the rank-r projection.  hi, lo are [m][npad], zero past n.
template <int RANK, int WPR>
__global__ void __launch_bounds__(DP_THREADS) k_w8_dgrad_prep(
    const uint16_t* __restrict__ dy, const uint16_t* __restrict__ scales,
    const uint16_t* __restrict__ up, const int32_t* __restrict__ offsets, int groups,
    int8_t* __restrict__ dhi, int8_t* __restrict__ dlo, float* __restrict__ ts,
    float* __restrict__ t_part, int m, int n, int npad, int quant_wgs, int slices) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  const int tid = threadIdx.x, lane = tid & 63;
  if (RANK > 0 && (int)blockIdx.x >= quant_wgs) {
    const int b = (int)blockIdx.x - quant_wgs;
    RowTile rt;
    if (!find_row_tile(offsets, groups, m, 16, b / slices, lane, rt)) return;
    project_tile<RANK ? RANK : 16>(dy, up + (int64_t)rt.group * n * RANK, t_part, dyn, m, n, rt,
                                   b % slices, slices);
    return;
  }
  __shared__ uint32_t row_max[4];
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = (int)blockIdx.x * (4 / WPR) + (WPR == 1 ? wave : 0);
  const int first = WPR == 1 ? lane * 8 : tid * 8;
  constexpr int STEP = WPR * 64 * 8;
  const int grp = row < m ? group_of_row(offsets, groups, row, lane) : -1;
  // rows behind the last group are not read by the product either; the whole
  // workgroup (WPR 4) or wave (WPR 1) leaves together
  if (grp < 0) return;
  const uint16_t* src = dy + (int64_t)row * n;
  const uint16_t* sc = scales + (int64_t)grp * n;
  auto load = [&](int c, float (&v)[8]) {
    const u32x4 d = load8_u16(src + c, n - c), s = load8_u16(sc + c, n - c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(d[i] << 16) * fp16_bits_to_f32(s[i] & 0xFFFFu);
      v[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u) * fp16_bits_to_f32(s[i] >> 16);
    }
  };
  // largest magnitude as bits: infinities and NaN order above every finite value
  uint32_t mx = 0;
  for (int c = first; c < n; c += STEP) {
    float v[8];
    load(c, v);
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
  for (int c = first; c < npad; c += STEP) {
    float v[8];
    load(c, v);   // zeros past n
    u32x2 oh, ol;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t h = 0, l = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // low 16 bits of the integer: lo in byte 0; hi in byte 1 once half a
        // step of hi is added
        const uint32_t b = finite ? __float_as_uint(v[4 * w + i] * inv + I8_ROUND) : 0u;
        l |= (b & 0xFFu) << (8 * i);
        h |= (((b + 128u) >> 8) & 0xFFu) << (8 * i);
      }
      oh[w] = h;
      ol[w] = l;
    }
    *reinterpret_cast<u32x2*>(dhi + (int64_t)row * npad + c) = oh;
    *reinterpret_cast<u32x2*>(dlo + (int64_t)row * npad + c) = ol;
  }
}

// ---------------------------------------------------------------- contraction
// 128 rows x 256 columns (one Hadamard block) per workgroup, eight waves of
// 64 x 64.  One stage = 64 rows of c: its 256-byte code rows (16 KB) and 64
// bytes of hi and of lo for each row (16 KB), streamed global -> LDS with
// direct 16-byte buffer loads into four stage buffers, two stages ahead.
//   hi/lo rows: chunk c of row r at slot c ^ ((r >> 1) & 3);
//   code rows: chunk c of row r at slot c ^ b_swz(r).  A B fragment needs 16
//   consecutive n of one column per lane: two transposed reads, each of eight
//   rows x 16 columns per 16 lanes (lane 2j + h points at row j, columns
//   8h..8h+7; lane i receives column i).  b_swz spreads the 32 rows that one
//   instruction touches over all sixteen 16-byte slots of a row.
constexpr int D_BM = 128, D_BN = 256, D_THREADS = 512;
constexpr int D_STAGE = 32 * 1024;
__shared__ __attribute__((aligned(16))) uint8_t d_buf0[D_STAGE];
__shared__ __attribute__((aligned(16))) uint8_t d_buf1[D_STAGE];
__shared__ __attribute__((aligned(16))) uint8_t d_buf2[D_STAGE];
__shared__ __attribute__((aligned(16))) uint8_t d_buf3[D_STAGE];

__device__ __forceinline__ int b_swz(int r) { return (r & 7) | (((r >> 4) & 1) << 3); }
// 16-byte unit u (of 64) of a row of 256 fp32 sums in the epilogue
__device__ __forceinline__ int c_unit(int row, int u) { return u ^ (row & 15); }

__global__ void __launch_bounds__(D_THREADS, 1) k_w8_dgrad_gemm(
    const int8_t* __restrict__ dhi, const int8_t* __restrict__ dlo, const float* __restrict__ ts,
    const float* __restrict__ t_part, const int8_t* __restrict__ codes,
    const uint16_t* __restrict__ down, const int32_t* __restrict__ offsets, int groups,
    void* __restrict__ dx, int m, int n, int npad, int k, int rank, int slices, int dx_bf16) {
  constexpr int FM = 4, FN = 4;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int fr = lane & 15, g = lane >> 4;
  const int nt = k / D_BN;
  const int mt = row_tile_count(offsets, groups, m, D_BM, lane);
  if ((int64_t)blockIdx.x >= (int64_t)mt * nt) return;
  int64_t tm, tn;
  xcd_tile(blockIdx.x, (int64_t)mt * nt, nt, tm, tn);
  RowTile rt;
  if (!find_row_tile(offsets, groups, m, D_BM, __builtin_amdgcn_readfirstlane((int)tm), lane, rt))
    return;
  const int grp = __builtin_amdgcn_readfirstlane(rt.group);
  const int rows = __builtin_amdgcn_readfirstlane(rt.rows);
  const int64_t m0 = __builtin_amdgcn_readfirstlane(rt.row0);
  const int k0 = __builtin_amdgcn_readfirstlane((int)tn) * D_BN;
  const int KT = npad >> 6;

  const __amdgpu_buffer_rsrc_t h_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(dhi + m0 * npad), (short)0, rows * npad, 0x00020000);
  const __amdgpu_buffer_rsrc_t l_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(dlo + m0 * npad), (short)0, rows * npad, 0x00020000);
  const int8_t* cbase = codes + (int64_t)grp * n * k + k0;
  // loaders: wave w fills rows 16w .. +16 of hi and of lo (64-byte rows) and
  // code rows 8w .. 8w+7 (two instructions of four 256-byte rows)
  uint32_t off_a, off_b[2];
  {
    const int r = 16 * wave + (lane >> 2);
    off_a = (uint32_t)min(r, rows - 1) * (uint32_t)npad + 16u * (uint32_t)((lane & 3) ^ ((r >> 1) & 3));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int br = 8 * wave + 4 * i + (lane >> 4);
      off_b[i] = (uint32_t)br * (uint32_t)k + 16u * (uint32_t)((lane & 15) ^ b_swz(br));
    }
  }
  auto issue = [&](int kt, uint8_t* buf) {
    // code rows at or past n lie beyond the descriptor and read as zeros
    const int64_t nrow = (int64_t)kt * 64;
    const int left = min(64, n - (int)nrow);
    const __amdgpu_buffer_rsrc_t b_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(cbase + nrow * k), (short)0, (left - 1) * k + D_BN, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(h_rsrc, (i8_lds_t)(buf + wave * 1024), 16, off_a,
                                             kt * 64, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(l_rsrc, (i8_lds_t)(buf + 8192 + wave * 1024), 16,
                                             off_a, kt * 64, 0, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          b_rsrc, (i8_lds_t)(buf + 16384 + (8 * wave + 4 * i) * 256), 16, off_b[i], 0, 0, 0);
  };
  const uint32_t a_lane = (uint32_t)(64 * wm + fr) * 64 + 16 * (uint32_t)(g ^ ((fr >> 1) & 3));
  // transposed read u of column tile j: row 16 g + 8 u + fr / 2 (whose swizzle
  // is that of its low three bits and g), columns 64 wn + 16 j + 8 (fr & 1)
  const int tr_row = 16 * g + (fr >> 1);
  const uint32_t b_lane = 16384u + (uint32_t)tr_row * 256 + 8u * (uint32_t)(fr & 1);
  const int tr_swz = b_swz(tr_row);
  i32x4 ah[FM][FN], al[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) ah[i][j] = al[i][j] = (i32x4){0, 0, 0, 0};
  auto compute = [&](const uint8_t* buf) {
    i32x4 bf[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      i32x2 h[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
        h[u] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2*)(buf + b_lane + u * 2048 +
                                                       16 * ((4 * wn + j) ^ tr_swz)));
      bf[j] = (i32x4){h[0][0], h[0][1], h[1][0], h[1][1]};
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const i32x4 hf = *reinterpret_cast<const i32x4*>(buf + a_lane + i * 1024);
      const i32x4 lf = *reinterpret_cast<const i32x4*>(buf + 8192 + a_lane + i * 1024);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        ah[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(hf, bf[j], ah[i][j], 0, 0, 0);
        al[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(lf, bf[j], al[i][j], 0, 0, 0);
      }
    }
  };
  auto sync = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(sq_wait_vm(4));
    __builtin_amdgcn_s_waitcnt(SQ_WAIT_LGKM0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  // Stage s lives in buffer s % 4; a step waits for its stage, meets the other
  // waves, issues stage s + 2 (into the buffer of stage s - 2) and computes.
  // Loads past the last stage fetch the last one again.
  issue(0, d_buf0);
  issue(min(1, KT - 1), d_buf1);
  int kt = 0;
  for (; kt + 4 <= KT; kt += 4) {
    sync();
    issue(min(kt + 2, KT - 1), d_buf2);
    compute(d_buf0);
    sync();
    issue(min(kt + 3, KT - 1), d_buf3);
    compute(d_buf1);
    sync();
    issue(min(kt + 4, KT - 1), d_buf0);
    compute(d_buf2);
    sync();
    issue(min(kt + 5, KT - 1), d_buf1);
    compute(d_buf3);
  }
  if (kt < KT) {
    sync();
    issue(min(kt + 2, KT - 1), d_buf2);
    compute(d_buf0);
    if (kt + 1 < KT) {
      sync();
      issue(min(kt + 3, KT - 1), d_buf3);
      compute(d_buf1);
      if (kt + 2 < KT) {
        sync();
        compute(d_buf2);
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(SQ_WAIT_VM0);   // the re-fetches have landed
  __syncthreads();                           // every wave is done with the buffers

  __builtin_amdgcn_sched_barrier(0);
  // Sums of 32 rows per buffer in fp32.  Lane (fr, g) of the product holds
  // rows 4g + v and column fr of a tile; column bits: fr 0-3, j 4-5, wn 6-7.
  // The butterflies over j run here, the others after the exchange.
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    uint8_t* st = wm == 0 ? (i < 2 ? d_buf0 : d_buf1) : (i < 2 ? d_buf2 : d_buf3);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = (float)ah[i][j][v] * 256.0f + (float)al[i][j][v];
      const float s0 = c[0] + c[1], s1 = c[0] - c[1], s2 = c[2] + c[3], s3 = c[2] - c[3];
      const float o[4] = {s0 + s2, s1 + s3, s0 - s2, s1 - s3};
      const int lr = 16 * (i & 1) + 4 * g + v;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float*>(st + lr * 1024 + 16 * c_unit(lr, 16 * wn + 4 * j + (fr >> 2)) +
                                  4 * (fr & 3)) = o[j];
    }
  }
  __syncthreads();
  // wave w takes rows 16w .. 16w+15: lane (fr, g) owns row 16w + fr and the
  // columns with j = g: w[16 q + p] is column 64 q + 16 g + p
  if (16 * wave >= rows) return;
  float w[64];
  {
    const uint8_t* st = (wave >> 1) == 0 ? d_buf0
                        : (wave >> 1) == 1 ? d_buf1
                        : (wave >> 1) == 2 ? d_buf2 : d_buf3;
    const int lr = 16 * (wave & 1) + fr;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const f32x4 f = *reinterpret_cast<const f32x4*>(st + lr * 1024 +
                                                        16 * c_unit(lr, 16 * q + 4 * g + p));
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
  const int row = 16 * wave + fr, rrow = (int)m0 + min(row, rows - 1);
  const float f = ts[rrow] * 0.0625f;
#pragma unroll
  for (int i = 0; i < 64; ++i) w[i] *= f;
  // rank-r branch with the columns as MFMA rows: output row 4g' + i of tile
  // (q, p) is column 64 q + 16 g' + 4 p + i, MFMA column fr the lane's row
  for (int rr = 0; rr < rank; rr += 32) {
    const bool rk = rr + 8 * g < rank;
    u32x4 part[3] = {};
    if (rk) project_sum8(t_part, m, rank, slices, rrow, rr + 8 * g, part);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int64_t col = (int64_t)grp * k + k0 + 64 * q + 16 * (fr >> 2) + 4 * p + (fr & 3);
        const bf16x8 dv = rk ? *reinterpret_cast<const bf16x8*>(down + col * rank + rr + 8 * g)
                             : (bf16x8){};
        const int b = 16 * q + 4 * p;
        f32x4 acc = {w[b], w[b + 1], w[b + 2], w[b + 3]};
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dv, __builtin_bit_cast(bf16x8, part[0]), acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dv, __builtin_bit_cast(bf16x8, part[1]), acc, 0, 0, 0);
        if (!dx_bf16)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dv, __builtin_bit_cast(bf16x8, part[2]), acc, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[b + i] = acc[i];
      }
  }
  if (row >= rows) return;
  const int64_t out0 = (m0 + row) * k + k0 + 16 * g;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (dx_bf16) {
      u32x4* dst = reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(dx) + out0 + 64 * q);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = pack_bf16x2(w[16 * q + 8 * h + 2 * i], w[16 * q + 8 * h + 2 * i + 1]);
        dst[h] = o;
      }
    } else {
      f32x4* dst = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(dx) + out0 + 64 * q);
#pragma unroll
      for (int p = 0; p < 4; ++p)
        dst[p] = (f32x4){w[16 * q + 4 * p], w[16 * q + 4 * p + 1], w[16 * q + 4 * p + 2],
                         w[16 * q + 4 * p + 3]};
    }
  }
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

W8DgradPlan plan_w8_dgrad(int64_t m, int64_t n, int64_t k, int groups, int rank) {
  W8DgradPlan p{};
  p.m = m; p.n = n; p.k = k; p.groups = groups; p.rank = rank;
  p.npad = (n + 63) / 64 * 64;
  p.slices = rank ? i8_project_slices(i8_tile_bound(m, groups, 16), n, DP_THREADS / 64) : 0;
  size_t off = 0;
  p.off_hi = off; off = align256(off + (size_t)m * p.npad);
  p.off_lo = off; off = align256(off + (size_t)m * p.npad);
  p.off_ts = off; off = align256(off + (size_t)m * 4);
  p.off_t = off;  off = align256(off + (size_t)p.slices * m * rank * 4);
  p.total = off;
  return p;
}

hipError_t launch_w8_dgrad(const W8DgradPlan& p, const uint16_t* dy, const int32_t* offsets,
                           const int8_t* codes, const uint16_t* scales, const uint16_t* up,
                           const uint16_t* down, void* dx, int dx_bf16, void* workspace,
                           hipStream_t stream) {
  char* base = static_cast<char*>(workspace);
  int8_t* dhi = reinterpret_cast<int8_t*>(base + p.off_hi);
  int8_t* dlo = reinterpret_cast<int8_t*>(base + p.off_lo);
  float* ts = reinterpret_cast<float*>(base + p.off_ts);
  float* t = reinterpret_cast<float*>(base + p.off_t);
  const int m = (int)p.m, n = (int)p.n, k = (int)p.k, npad = (int)p.npad;
  // rows of up to 2048 values take one wave (32 values per lane), longer ones four
  const int wpr = n <= 2048 ? 1 : 4;
  const int64_t qwgs = wpr == 1 ? (p.m + 3) / 4 : p.m;
  const int64_t twgs = i8_tile_bound(p.m, p.groups, 16) * p.slices;
  const size_t lds = (size_t)(DP_THREADS / 64) * 64 * p.rank;
#define SQ_W8DP(R, WPR)                                                                          \
  hipLaunchKernelGGL((k_w8_dgrad_prep<R, WPR>), dim3((unsigned)(qwgs + twgs)), dim3(DP_THREADS), \
                     lds, stream, dy, scales, up, offsets, p.groups, dhi, dlo, ts, t, m, n, npad, \
                     (int)qwgs, p.slices)
#define SQ_W8DP_RANK(WPR)              \
  do {                                 \
    if (p.rank == 0) SQ_W8DP(0, WPR);  \
    else if (p.rank == 16) SQ_W8DP(16, WPR); \
    else if (p.rank == 32) SQ_W8DP(32, WPR); \
    else SQ_W8DP(64, WPR);             \
  } while (0)
  if (wpr == 1) SQ_W8DP_RANK(1);
  else SQ_W8DP_RANK(4);
#undef SQ_W8DP_RANK
#undef SQ_W8DP
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int64_t tiles = i8_tile_bound(p.m, p.groups, D_BM) * (p.k / D_BN);
  hipLaunchKernelGGL(k_w8_dgrad_gemm, dim3((unsigned)tiles), dim3(D_THREADS), 0, stream, dhi, dlo,
                     ts, t, codes, down, offsets, p.groups, dx, m, n, npad, k, p.rank, p.slices,
                     dx_bf16);
  return hipGetLastError();
}

}  // namespace sq
