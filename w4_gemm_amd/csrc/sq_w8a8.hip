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

// Workgroups 0 .. quant_wgs-1 hold rows_per_wg rows each, four lanes per
// (row, block) pair, 16 pairs per wave; the rest compute t.
template <int RANK>
__global__ void __launch_bounds__(1024) k_w8a8_prep(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ down,
    const int32_t* __restrict__ offsets, int groups, int8_t* __restrict__ xq,
    float* __restrict__ xs, float* __restrict__ t_part, int m, int k, int rows_per_wg,
    int quant_wgs, int slices) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  const int tid = threadIdx.x, lane = tid & 63;
  if (RANK > 0 && (int)blockIdx.x >= quant_wgs) {
    const int b = (int)blockIdx.x - quant_wgs;
    RowTile rt;
    if (!find_row_tile(offsets, groups, m, 16, b / slices, lane, rt)) return;
    project_tile<RANK ? RANK : 16>(x, down + (int64_t)rt.group * k * RANK, t_part, dyn, m, k, rt,
                                   b % slices, slices);
    return;
  }
  __shared__ uint32_t row_max[PREP_MAX_ROWS];
  if (tid < PREP_MAX_ROWS) row_max[tid] = 0;
  __syncthreads();
  const int nb = k >> 8;
  const int pair = (tid >> 6) * 16 + (lane & 15), g = lane >> 4;
  const int lrow = pair / nb, blk = pair - lrow * nb;
  const int row = (int)blockIdx.x * rows_per_wg + lrow;
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
// 256 x 256 output tile per workgroup, eight waves of 128 x 64 (8 x 4 MFMA
// tiles).  One stage = 64 bytes of K of each operand row; both operands
// stream global -> LDS with direct 16-byte buffer loads into three stage
// buffers, two stages ahead of the MFMAs.  Chunk c of row r sits at slot
// c ^ ((r >> 1) & 3), which keeps the 16-byte fragment reads free of bank
// conflicts.
constexpr int G_BM = 256, G_BN = 256, G_THREADS = 512;
constexpr int G_STAGE = 256 * 64;
__shared__ __attribute__((aligned(16))) uint8_t g_a0[G_STAGE];
__shared__ __attribute__((aligned(16))) uint8_t g_a1[G_STAGE];
__shared__ __attribute__((aligned(16))) uint8_t g_a2[G_STAGE];
__shared__ __attribute__((aligned(16))) uint8_t g_b0[G_STAGE];
__shared__ __attribute__((aligned(16))) uint8_t g_b1[G_STAGE];
__shared__ __attribute__((aligned(16))) uint8_t g_b2[G_STAGE];

__global__ void __launch_bounds__(G_THREADS, 1) k_w8a8_gemm(
    const int8_t* __restrict__ xq, const float* __restrict__ xs,
    const float* __restrict__ t_part, const int8_t* __restrict__ codes,
    const uint16_t* __restrict__ scales, const uint16_t* __restrict__ up,
    const int32_t* __restrict__ offsets, int groups, void* __restrict__ y, int m, int n, int k,
    int rank, int slices, int y_bf16) {
  constexpr int FM = 8, FN = 4;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int fr = lane & 15, g = lane >> 4;
  const int nt = (n + G_BN - 1) / G_BN;
  const int mt = row_tile_count(offsets, groups, m, G_BM, lane);
  if ((int64_t)blockIdx.x >= (int64_t)mt * nt) return;
  int64_t tm, tn;
  xcd_tile(blockIdx.x, (int64_t)mt * nt, nt, tm, tn);
  RowTile rt;
  if (!find_row_tile(offsets, groups, m, G_BM, __builtin_amdgcn_readfirstlane((int)tm), lane, rt))
    return;
  // scalar registers for everything the descriptors are built from
  const int grp = __builtin_amdgcn_readfirstlane(rt.group);
  const int rows = __builtin_amdgcn_readfirstlane(rt.rows);
  const int64_t m0 = __builtin_amdgcn_readfirstlane(rt.row0);
  const int n0 = __builtin_amdgcn_readfirstlane((int)tn) * G_BN;
  const int cols = min(G_BN, n - n0);
  const int64_t brow0 = (int64_t)grp * n + n0;   // first weight row of the tile
  const int KT = k >> 6;

  const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(xq + m0 * k), (short)0, rows * k, 0x00020000);
  const __amdgpu_buffer_rsrc_t b_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(codes + brow0 * k), (short)0, cols * k, 0x00020000);
  uint32_t off_a[2], off_b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 32 * wave + 16 * i + (lane >> 2);
    const uint32_t slot = (uint32_t)((lane & 3) ^ ((r >> 1) & 3));
    off_a[i] = (uint32_t)min(r, rows - 1) * (uint32_t)k + 16u * slot;
    off_b[i] = (uint32_t)min(r, cols - 1) * (uint32_t)k + 16u * slot;
  }
  auto issue = [&](int kt, uint8_t* ab, uint8_t* bb) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(a_rsrc, (i8_lds_t)(ab + (32 * wave + 16 * i) * 64),
                                               16, off_a[i], kt * 64, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(b_rsrc, (i8_lds_t)(bb + (32 * wave + 16 * i) * 64),
                                               16, off_b[i], kt * 64, 0, 0);
    }
  };
  const uint32_t swz = (uint32_t)(g ^ ((fr >> 1) & 3));
  const uint32_t a_lane = (uint32_t)(128 * wm + fr) * 64 + 16 * swz;
  const uint32_t b_lane = (uint32_t)(64 * wn + fr) * 64 + 16 * swz;
  i32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (i32x4){0, 0, 0, 0};
  auto compute = [&](const uint8_t* ab, const uint8_t* bb) {
    i32x4 bf[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) bf[j] = *reinterpret_cast<const i32x4*>(bb + b_lane + j * 1024);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const i32x4 af = *reinterpret_cast<const i32x4*>(ab + a_lane + i * 1024);
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af, bf[j], acc[i][j], 0, 0, 0);
    }
  };
  auto sync = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(sq_wait_vm(4));
    __builtin_amdgcn_s_waitcnt(SQ_WAIT_LGKM0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  // Stage s lives in buffer s % 3.  Each step waits for its own loads of the
  // stage (four of the next stage may still be in flight), meets the other
  // waves, refills the buffer of stage s - 1 with stage s + 2 and computes.
  // Loads past the last stage fetch the last one again, into a buffer that is
  // not read any more.
  issue(0, g_a0, g_b0);
  issue(min(1, KT - 1), g_a1, g_b1);
  int kt = 0;
  for (; kt + 3 <= KT; kt += 3) {
    sync();
    issue(min(kt + 2, KT - 1), g_a2, g_b2);
    compute(g_a0, g_b0);
    sync();
    issue(min(kt + 3, KT - 1), g_a0, g_b0);
    compute(g_a1, g_b1);
    sync();
    issue(min(kt + 4, KT - 1), g_a1, g_b1);
    compute(g_a2, g_b2);
  }
  if (kt < KT) {
    sync();
    issue(min(kt + 2, KT - 1), g_a2, g_b2);
    compute(g_a0, g_b0);
    if (kt + 1 < KT) {
      sync();
      compute(g_a1, g_b1);
    }
  }
  __builtin_amdgcn_s_waitcnt(SQ_WAIT_VM0);   // the re-fetches have landed

  // scales, the column's first: |acc w| < 2^47 cannot overflow whatever the
  // row's magnitude is; acc[i][j][v] is row 128 wm + 16 i + 4 g + v, column 64 wn + 16 j + fr
  const int rbase = 128 * wm, cbase = 64 * wn;
  f32x4 out[FM][FN];
  float wsc[FN];
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 0; j < FN; ++j)
    wsc[j] = fp16_bits_to_f32(scales[brow0 + min(cbase + 16 * j + fr, cols - 1)]);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float sr = xs[m0 + min(rbase + 16 * i + 4 * g + v, rows - 1)];
#pragma unroll
      for (int j = 0; j < FN; ++j) out[i][j][v] = (float)acc[i][j][v] * wsc[j] * sr;
    }
  // rank-r branch: (t_hi + t_lo) up^T (rank 16: the upper half of the 32-wide
  // step reads zeros)
  for (int rr = 0; rr < rank; rr += 32) {
    const bool rk = rr + 8 * g < rank;
    bf16x8 bu[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j)
      bu[j] = rk ? *reinterpret_cast<const bf16x8*>(
                       up + (brow0 + min(cbase + 16 * j + fr, cols - 1)) * rank + rr + 8 * g)
                 : (bf16x8){};
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      bf16x8 hi = {}, lo = {};
      if (rk)
        project_sum8(t_part, m, rank, slices, (int)m0 + min(rbase + 16 * i + fr, rows - 1),
                     rr + 8 * g, hi, lo);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        out[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, bu[j], out[i][j], 0, 0, 0);
        out[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, bu[j], out[i][j], 0, 0, 0);
      }
    }
  }
  if (!y_bf16) {
    float* yf = reinterpret_cast<float*>(y);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = rbase + 16 * i + 4 * g + v;
        if (r >= rows) continue;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int c = cbase + 16 * j + fr;
          if (c < cols) yf[(m0 + r) * n + n0 + c] = out[i][j][v];
        }
      }
    return;
  }
  // bf16: each wave turns 64 x 64 values at a time into 128-byte row segments
  // in 8 KB of the stage buffers (16-byte chunk c of row r at slot
  // c ^ a_swz(r)), so that every store instruction writes whole segments
  __syncthreads();   // every wave is done with the stage buffers
  const int wb = wave >> 1;
  uint8_t* st = (wb == 0 ? g_a0 : wb == 1 ? g_a1 : wb == 2 ? g_b0 : g_b1) + (wave & 1) * 8192;
  const bool wide = (n & 7) == 0;
#pragma unroll
  for (int h = 0; h < FM / 4; ++h) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int lr = 16 * i + 4 * g + v;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int c = 16 * j + fr;
          *reinterpret_cast<uint16_t*>(st + lr * 128 + 16 * ((c >> 3) ^ a_swz(lr)) + 2 * (c & 7)) =
              f32_to_bf16(out[4 * h + i][j][v]);
        }
      }
    __builtin_amdgcn_s_waitcnt(SQ_WAIT_LGKM0);
    __builtin_amdgcn_wave_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int lr = 8 * it + (lane >> 3), chunk = lane & 7;
      const int r = rbase + 64 * h + lr, c = cbase + 8 * chunk;
      const u32x4 o = *reinterpret_cast<const u32x4*>(st + lr * 128 + 16 * (chunk ^ a_swz(lr)));
      if (r >= rows || c >= cols) continue;
      uint16_t* dst = reinterpret_cast<uint16_t*>(y) + (m0 + r) * n + n0 + c;
      if (wide) {
        *reinterpret_cast<u32x4*>(dst) = o;
      } else {
        const uint16_t* hv = reinterpret_cast<const uint16_t*>(&o);
        for (int i = 0; i < 8 && c + i < cols; ++i) dst[i] = hv[i];
      }
    }
    __builtin_amdgcn_s_waitcnt(SQ_WAIT_LGKM0);   // the reads are done before the next pass writes
    __builtin_amdgcn_wave_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
  }
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

// Row tiles of tile_m rows that `groups` groups of m rows together can have.
int64_t i8_tile_bound(int64_t m, int groups, int tile_m) {
  const int64_t used = std::min<int64_t>(groups, m);
  return groups <= 1 ? (m + tile_m - 1) / tile_m : (m + used * (tile_m - 1)) / tile_m;
}

// K slices of the rank-r projection: enough 16-row tiles x slices to put two
// workgroups on each of the 256 CUs, at least one 256-column block per wave.
int i8_project_slices(int64_t tiles16, int64_t cols, int waves) {
  const int64_t blocks = (cols + 255) / 256;
  const int64_t most = (blocks + waves - 1) / waves;
  return (int)std::max<int64_t>(1, std::min(most, (512 + tiles16 - 1) / tiles16));
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
    if (use > best + 1e-9) {
      best = use;
      rows = (int)r;
      waves = w;
    }
  }
  p.prep_rows = rows;
  p.prep_waves = waves;
  p.slices = rank ? i8_project_slices(i8_tile_bound(m, groups, 16), k, waves) : 0;
  size_t off = 0;
  p.off_xq = off; off = align256(off + (size_t)m * k);
  p.off_xs = off; off = align256(off + (size_t)m * 4);
  p.off_t = off;  off = align256(off + (size_t)p.slices * m * rank * 4);
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
  const int64_t twgs = i8_tile_bound(p.m, p.groups, 16) * p.slices;
  const size_t lds = (size_t)p.prep_waves * 64 * p.rank;
#define SQ_W8A8_PREP(R)                                                                        \
  hipLaunchKernelGGL((k_w8a8_prep<R>), dim3((unsigned)(qwgs + twgs)),                          \
                     dim3(64 * p.prep_waves), lds, stream, x, down, offsets, p.groups, xq, xs, \
                     t, m, k, p.prep_rows, (int)qwgs, p.slices)
  if (p.rank == 0) SQ_W8A8_PREP(0);
  else if (p.rank == 16) SQ_W8A8_PREP(16);
  else if (p.rank == 32) SQ_W8A8_PREP(32);
  else SQ_W8A8_PREP(64);
#undef SQ_W8A8_PREP
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int64_t tiles = i8_tile_bound(p.m, p.groups, G_BM) * ((p.n + G_BN - 1) / G_BN);
  hipLaunchKernelGGL(k_w8a8_gemm, dim3((unsigned)tiles), dim3(G_THREADS), 0, stream, xq, xs, t,
                     codes, scales, up, offsets, p.groups, y, m, n, k, p.rank, p.slices, y_bf16);
  return hipGetLastError();
}

}  // namespace sq
