// Products of the 8-bit float mode, for one layer and for experts.  Rows a are
// rounded to e4m3 with a power of two per 128 values along the contraction
// (sq_f8_rows.hip), the weight's codes have one per 128 x 128:
//
//   forward   y = Q(x) W^T
//   gated     h = act(g) u, g = Q(x) Wg^T, u = Q(x) Wu^T
//   gradient  dx = Q(dy) W, and dx = Q(dg) Wg + Q(du) Wu
//
// v_mfma_scale_f32_16x16x128_f8f6f4 contracts one block of each operand's row
// with both powers of two for free: they are why the mode's scales are powers of
// two.  The instruction sums its products in groups of eight consecutive values
// and drops what lies below 2^-13 of a group's largest product (measured: bits
// 2^-14 down vanish, towards zero; between groups and against the accumulator
// it keeps 24 bits).  The largest goes by the codes' exponent fields, where a
// subnormal code stands at 2^-6 (448 opposite 2^-9 takes products of 2^-12 with
// it) and zeros do not count.  For Gaussian rows that is 2^-17 of sum |a b|,
// 1.5e-5 of the result's norm, up to 5e-5 where codes spread over all exponents:
// a hundredth of a bf16 result's own rounding, and 250 times an fp32 result's.
// So results of 16 bits take it, and fp32 results take fp16 MFMA on the codes as
// fp16 (every e4m3 value is one; products exact, sums in fp32), with the powers
// of two applied to each block's sum: 2.5e-7 at K = 16384.  That instruction has
// half the rate, and its conversions take turns with it (matrix unit busy 0.39 of
// the cycles): 4480 x 6144 x 16384 takes 930 us, 342 with bf16 results.
#include <algorithm>
#include <type_traits>

#include "sq_f8.hpp"
#include "sq_kernels.h"

namespace sq {
namespace {

enum { F8_FWD = 0, F8_GATED = 1, F8_GRAD = 2 };

struct F8Args {
  const uint8_t *a, *ax;          // rows: codes [m][128 stages], exponents [m][lax]
  const uint8_t *b0, *b1;         // weight codes [groups][n][128 kb] (b1: up)
  const uint8_t *x0, *x1;         // their exponents [groups][nb][kb]
  const int32_t* offsets;
  void* y;
  uint16_t *g, *u;                // gated: both projections in bf16, or null
  float* partial;
  int groups, m, n, k, kb, nb;
  int lax, pitch, stages;         // bytes of a row's exponents; blocks of 128 of a row's codes; of the contraction
  int y_bf16, act, most_tiles, splits;
};

struct F16Frag {
  half8 h[4];
};
// 32 codes of a lane as fp16, in order.
__device__ __forceinline__ F16Frag f8_to_f16(const i32x8& c) {
  F16Frag o;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const half2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)c[2 * w], 1.0f, false);
    const half2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)c[2 * w], 1.0f, true);
    const half2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)c[2 * w + 1], 1.0f, false);
    const half2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)c[2 * w + 1], 1.0f, true);
    o.h[w] = (half8){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
  }
  return o;
}
__device__ __forceinline__ f32x4 f16_block(const F16Frag& w, const F16Frag& a) {
  f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 4; ++s) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.h[s], a.h[s], p, 0, 0, 0);
  return p;
}
// acc + p 2^(byte sum - 254)
__device__ __forceinline__ void add_scaled(f32x4& acc, const f32x4& p, int bytes) {
#pragma unroll
  for (int v = 0; v < 4; ++v) acc[v] += __builtin_amdgcn_ldexpf(p[v], bytes - 254);
}

// ---------------------------------------------------------------- tiles
// Products alone: 4480 x 6144 x 16384 in 342 us = 2.64 P operations/s, matrix unit
// busy 0.65 of the cycles at the 2 GHz it holds; the gated block 4480 x 16384 x
// 6144, which stores 440 MB, 705 us = 2.56 P, its backward 715-760 us, where 2.5 GB
// come from beyond the L2.  About 9 us of each round of 256 tiles are its first
// loads and its stores.
// Large tiles (224 and 256 rows) run on four waves, one per SIMD, with 128 columns
// each: per MFMA they read two thirds of what eight waves of 64 columns read from
// LDS, whose reads and the loads' writes otherwise take as long as the matrix unit
// (4480 x 6144 x 16384: 396 -> 378 us).  Rows of codes are an odd number of
// 128-byte blocks apart in the workspace (gated, above: 941 -> 906 us).
// BM = 32 FM rows per workgroup x 256 columns of the weight tile (gated: 128
// columns of gate and the same 128 of up), two wave rows of 16 FM x WN wave
// columns of 16 FN.  The weight is the MFMA's first operand, so that a lane ends
// up with consecutive columns of one row.  One stage = one block of 128 along
// the contraction, two stages in LDS, global -> LDS with direct 16-byte buffer
// loads.
//   rows and forward weight rows (128 bytes): chunk c of row r at slot c ^ (r & 7);
//   gradient, weight rows of 256 bytes: slot c ^ grad_swz(r), read transposed
//   (see sq_w8_dgrad.hip).
// Forward: row 16 j + 4 q + v of a wave column's LDS rows holds its column 32 (j /
// 2) + 8 q + 4 (j & 1) + v, so that lane (fr, g) has runs of eight columns of row
// fr and four lanes store 64 bytes in a row; gated: the first half of the rows
// are gate's, the second the same of up.
constexpr int F8_BN = 256;
constexpr int F8_BSTAGE = F8_BN * 128;
constexpr int F8_MAX_THREADS = 512;
constexpr int F8_MAX_STAGES = 1024;   // of one workgroup: the planner splits longer contractions

__device__ __forceinline__ int grad_swz(int r) { return (r & 7) | (((r >> 4) & 1) << 3); }

// acc += w a on AGPRs that stay in place.  (Through the builtin the compiler
// permutes 224 or more accumulators: 1.7 moves per MFMA.)  The compiler knows of
// no hazard around it: the s_nop covers an operand that a vector instruction has
// just written (it costs nothing measurable: an MFMA takes 32 cycles); results
// are read behind the contraction only, after 32 wait states (pinned_wait), and
// where pinned_row lets them be: the compiler, which sees no reason to wait,
// otherwise reads some of them, or stores them to scratch memory, before the wait.
template <int B>
__device__ __forceinline__ void pinned_mfma(f32x4& acc, const i32x8& w, const i32x8& a, int we,
                                            int re) {
  asm("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,%5,0] "
      "op_sel_hi:[0,%6,0]"
      : "+a"(acc)
      : "v"(w), "v"(a), "v"(we), "v"(re), "n"(B & 1), "n"(B >> 1));
}

template <int N>
__device__ __forceinline__ void pinned_row(f32x4 (&acc)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+a"(acc[i]));
}
__device__ __forceinline__ void pinned_wait() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

template <int FM, int WN, int MODE, int ACT, bool F16, bool SPLIT>
__global__ void __launch_bounds__(128 * WN, 1) k_f8_gemm(const F8Args p) {
  constexpr int WAVES = 2 * WN, THREADS = 64 * WAVES, FN = 16 / WN, BM = 32 * FM;
  // one load instruction of every wave covers LOAD rows of 128 bytes
  constexpr int LOAD = 8 * WAVES, NA = (BM + LOAD - 1) / LOAD, NB = F8_BN / LOAD;
  // row tiles 0 to 3 and the others apart: the compiler waits for every load into
  // an LDS array before it reads from that array
  constexpr int LOW = BM < 128 ? BM : 128, HIGH = BM > 128 ? NA * LOAD - 128 : 16;
  constexpr bool PINNED = WN == 2;
  constexpr int WIDTH = MODE == F8_GATED ? 128 : 256;   // columns of the result per tile
  __shared__ __attribute__((aligned(16))) uint8_t a0[LOW * 128];
  __shared__ __attribute__((aligned(16))) uint8_t a1[LOW * 128];
  __shared__ __attribute__((aligned(16))) uint8_t a0_high[HIGH * 128];
  __shared__ __attribute__((aligned(16))) uint8_t a1_high[HIGH * 128];
  __shared__ __attribute__((aligned(16))) uint8_t b0[F8_BSTAGE];
  __shared__ __attribute__((aligned(16))) uint8_t b1[F8_BSTAGE];
  // exponents: the rows' of four stages, twice, in the order [stage][wave
  // row][fr][row tile]; all of the tile's two weight blocks'
  __shared__ __attribute__((aligned(16))) uint8_t ea[2][4][256];
  __shared__ __attribute__((aligned(16))) uint8_t eb[F8_MAX_STAGES][2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int fr = lane & 15, g = lane >> 4;
  const int out_cols = MODE == F8_GRAD ? p.k : p.n;
  const int nt = (out_cols + WIDTH - 1) / WIDTH;
  const int mt = row_tile_count(p.offsets, p.groups, p.m, BM, p.most_tiles, lane);
  const int tiles = mt * nt;
  const int split = __builtin_amdgcn_readfirstlane(tiles ? (int)blockIdx.x / tiles : p.splits);
  if (split >= p.splits) return;
  int64_t tm, tn;
  xcd_tile((int)blockIdx.x - split * tiles, tiles, nt, tm, tn);
  RowTile rt;
  if (!find_row_tile(p.offsets, p.groups, p.m, BM, __builtin_amdgcn_readfirstlane((int)tm), lane, rt))
    return;
  const int grp = __builtin_amdgcn_readfirstlane(rt.group);
  const int rows = __builtin_amdgcn_readfirstlane(rt.rows);
  const int64_t m0 = __builtin_amdgcn_readfirstlane(rt.row0);
  const int c0 = __builtin_amdgcn_readfirstlane((int)tn) * WIDTH;   // first result column
  const int cols = min(WIDTH, out_cols - c0);
  const int lda = 128 * p.pitch, ldb = 128 * p.kb;
  // stages st0 .. st0 + ST - 1; splits cut in fours, as the exponents' words do
  const int quads = (p.stages + 3) >> 2;
  const int q0 = __builtin_amdgcn_readfirstlane((int)((int64_t)split * quads / p.splits));
  const int q1 = __builtin_amdgcn_readfirstlane((int)((int64_t)(split + 1) * quads / p.splits));
  const int st0 = 4 * q0, ST = min(4 * q1, p.stages) - st0;

  // ---- loaders
  const int lr = 8 * wave + (lane >> 3);
  const uint32_t chunk = 16u * (uint32_t)((lane & 7) ^ (lr & 7));
  const uint32_t off_a = (uint32_t)lr * (uint32_t)lda + chunk;
  const uint8_t* a_base = p.a + m0 * lda;
  // Forward weights: LDS row LOAD i + lr holds column b_col(i) + that of row lr.
  const int tile0 = lr >> 4;   // of the lane's row in the wave column's FN tiles, for i = 0
  const int bl = 8 * ((lr >> 2) & 3) + 4 * (tile0 & 1) + (lr & 3) +
                 (MODE == F8_FWD ? 32 * (tile0 >> 1) : 0);
  const uint32_t off_b = (uint32_t)bl * (uint32_t)ldb + chunk;
  // LOAD rows are a wave column's 64 (WN = 4), or two of its eight tiles
  auto b_col = [&](int i) {
    if constexpr (WN == 4) return MODE == F8_GATED ? 32 * i : 64 * i;
    else return MODE == F8_GATED ? 64 * (i >> 2) + 32 * (i & 1) : 128 * (i >> 2) + 32 * (i & 3);
  };
  // Gradient: the weight rows of stage st from their first column of the tile;
  // rows past the weight's last lie beyond the descriptor and arrive as zeros.
  const int gr = 4 * wave + (lane >> 4);
  uint32_t off_g[2];   // of load instructions with even and odd numbers
#pragma unroll
  for (int i = 0; i < 2; ++i)
    off_g[i] = (uint32_t)gr * (uint32_t)ldb +
               16u * (uint32_t)((lane & 15) ^ grad_swz(gr + 4 * WAVES * i));
  struct Rows {
    const uint8_t* base;
    int bytes;
  };
  auto grad_rows = [&](int st) {
    const int s = st0 + st, seg = s >= p.nb, n0 = 128 * (s - (seg ? p.nb : 0));
    return Rows{(seg ? p.b1 : p.b0) + ((int64_t)grp * p.n + n0) * ldb + c0,
                (min(p.n - n0, 128) - 1) * ldb + min(256, ldb - c0)};
  };
  const __amdgpu_buffer_rsrc_t a_rsrc =
      __builtin_amdgcn_make_buffer_rsrc((void*)a_base, (short)0, rows * lda, 0x00020000);
  const __amdgpu_buffer_rsrc_t b_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((MODE == F8_GATED && WN == 4 && wave >= 4 ? p.b1 : p.b0) +
              ((int64_t)grp * p.n + c0) * ldb),
      (short)0, cols * ldb, 0x00020000);
  const __amdgpu_buffer_rsrc_t u_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((MODE == F8_GATED ? p.b1 : p.b0) + ((int64_t)grp * p.n + c0) * ldb), (short)0,
      cols * ldb, 0x00020000);
  // s: the stage's buffers
  auto issue_a = [&](int st, int s, int i) {
    constexpr int PER = 128 / LOAD;   // load instructions of row tiles 0 to 3
    uint8_t* to = i < PER ? (s & 1 ? a1 : a0) + (WAVES * i + wave) * 1024
                          : (s & 1 ? a1_high : a0_high) + (WAVES * (i - PER) + wave) * 1024;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(a_rsrc, (i8_lds_t)to, 16,
                                             off_a + (uint32_t)(LOAD * i * lda), (st0 + st) * 128, 0, 0);
  };
  auto issue_b = [&](int st, const Rows& from, int s, int i) {
    const i8_lds_t to = (i8_lds_t)((s & 1 ? b1 : b0) + (WAVES * i + wave) * 1024);
    if constexpr (MODE == F8_GRAD) {
      const __amdgpu_buffer_rsrc_t rsrc =
          __builtin_amdgcn_make_buffer_rsrc((void*)from.base, (short)0, from.bytes, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, to, 16,
                                               off_g[i & 1] + (uint32_t)(4 * WAVES * i * ldb), 0, 0, 0);
    } else {
      const uint32_t off = off_b + (uint32_t)(b_col(i) * ldb);
      if (MODE == F8_GATED && WN == 2 && (i & 2))   // up's tiles; with WN = 4 waves 4 to 7 have them
        __builtin_amdgcn_raw_ptr_buffer_load_lds(u_rsrc, to, 16, off, (st0 + st) * 128, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(b_rsrc, to, 16, off, (st0 + st) * 128, 0, 0);
    }
  };
  auto issue = [&](int st, int s) {
    const Rows from = MODE == F8_GRAD ? grad_rows(st) : Rows{};
#pragma unroll
    for (int i = 0; i < NB; ++i) issue_b(st, from, s, i);
#pragma unroll
    for (int i = 0; i < NA; ++i) issue_a(st, s, i);
  };
  // row exponents: every thread has the word of one row (some rows twice)
  constexpr int EROWS = BM <= 64 ? 64 : BM <= 128 ? 128 : 256;
  const int erow = tid & (EROWS - 1), e_at = ((erow >> 4) & 1) * 128 + (erow & 15) * 8 + (erow >> 5);
  const uint8_t* e_src = p.ax + (m0 + min(erow, rows - 1)) * p.lax;
  uint32_t ew;
  auto load_exps = [&](int q) { ew = *reinterpret_cast<const uint32_t*>(e_src + 4 * min(q, quads - 1)); };
  auto put_exps = [&](int buf) {
#pragma unroll
    for (int s = 0; s < 4; ++s) ea[buf][s][e_at] = (uint8_t)(ew >> (8 * s));
  };
  auto weight_exps = [&]() {
    for (int t = tid; t < 2 * ST; t += THREADS) {
      const int which = t & 1, s = st0 + (t >> 1);
      uint8_t v;
      if constexpr (MODE == F8_FWD)
        v = p.x0[((int64_t)grp * p.nb + min((c0 >> 7) + which, p.nb - 1)) * p.kb + s];
      else if constexpr (MODE == F8_GATED)
        v = (which ? p.x1 : p.x0)[((int64_t)grp * p.nb + (c0 >> 7)) * p.kb + s];
      else
        v = (s >= p.nb ? p.x1 : p.x0)[((int64_t)grp * p.nb + (s >= p.nb ? s - p.nb : s)) * p.kb +
                                      min((c0 >> 7) + which, p.kb - 1)];
      eb[t >> 1][which] = v;
    }
  };

  issue(0, 0);
  issue(min(1, ST - 1), 1);
  load_exps(q0);
  weight_exps();
  put_exps(0);

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
  auto sync = [&](auto on_way) {   // this many loads of a wave may be on their way
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(sq_wait_vm(decltype(on_way)::value));
    __builtin_amdgcn_s_waitcnt(SQ_WAIT_LGKM0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  sync(std::integral_constant<int, 0>{});

  // ---- fragments: lane (fr, g) holds bytes 16 g .. and 64 + 16 g .. of its row
  const uint32_t a_row = (uint32_t)(16 * wm + fr) * 128, b_row = (uint32_t)(16 * FN * wn + fr) * 128;
  const uint32_t slot0 = 16u * (uint32_t)(g ^ (fr & 7)), slot1 = 16u * (uint32_t)((4 + g) ^ (fr & 7));
  const int tr_row = 16 * g + (fr >> 1), tr_swz = grad_swz(tr_row);
  const uint32_t t_row = (uint32_t)tr_row * 256 + 8u * (uint32_t)(fr & 1);
  auto read_a = [&](int s, int i) {
    const uint8_t* ab = (i < 4 ? (s & 1 ? a1 : a0) : (s & 1 ? a1_high : a0_high)) + a_row + (i & 3) * 4096;
    const i32x4 lo = *reinterpret_cast<const i32x4*>(ab + slot0);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(ab + slot1);
    return (i32x8){lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  auto read_b = [&](int s, int j) {
    const uint8_t* bb = s & 1 ? b1 : b0;
    if constexpr (MODE == F8_GRAD) {
      i32x2 t[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)   // rows 16 g + 8 (u & 1) + 64 (u / 2)
        t[u] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2*)(bb + t_row + (u & 1) * 2048 + (u >> 1) * 16384 +
                                                       16 * ((FN * wn + j) ^ tr_swz)));
      return (i32x8){t[0][0], t[0][1], t[1][0], t[1][1], t[2][0], t[2][1], t[3][0], t[3][1]};
    } else {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(bb + b_row + slot0 + j * 2048);
      const i32x4 hi = *reinterpret_cast<const i32x4*>(bb + b_row + slot1 + j * 2048);
      return (i32x8){lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
  };
  // exponents of the lane's row tiles (byte i) and of its columns' weight block
  // (forward, gradient: the wave's columns lie in one; gated: gate, up)
  struct Exps {
    u32x2 rows;
    int w[2];
  };
  auto read_exps = [&](Exps& e, int st) {
    e.rows = *reinterpret_cast<const u32x2*>(&ea[(st >> 2) & 1][st & 3][128 * wm + 8 * fr]);
    if constexpr (MODE == F8_GATED) {
      e.w[0] = eb[st][0];
      e.w[1] = eb[st][1];
    } else {
      e.w[0] = e.w[1] = eb[st][FN * wn / 8];
    }
  };

  auto contract = [&](auto count) {
    constexpr int F = decltype(count)::value;
    // The stage's last H row tiles are contracted together behind its barrier, the
    // L before them in pairs.
    constexpr int H = F16 ? 2 : F > 4 ? F - 4 : F, L = F - H, NP = L / 2, FIRST = L ? 2 : H;
    constexpr bool EARLY = PINNED && NP == 2;
    const std::integral_constant<int, EARLY ? NA + NB : 0> on_way;
    auto product = [&](int i, int j, const i32x8& w, const i32x8& a, const Exps& e) {
      const int we = e.w[j / (FN / 2)], re = (int)e.rows[i >> 2];
      if constexpr (F16) {
        add_scaled(acc[i][j], f16_block(f8_to_f16(w), f8_to_f16(a)), we + ((re >> (8 * (i & 3))) & 255));
      } else if constexpr (PINNED) {
        switch (i & 3) {
          case 0: pinned_mfma<0>(acc[i][j], w, a, we, re); break;
          case 1: pinned_mfma<1>(acc[i][j], w, a, we, re); break;
          case 2: pinned_mfma<2>(acc[i][j], w, a, we, re); break;
          default: pinned_mfma<3>(acc[i][j], w, a, we, re); break;
        }
      } else {
#define SQ_F8_MFMA(B) __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, acc[i][j], 0, 0, 0, we, B, re)
        switch (i & 3) {
          case 0: acc[i][j] = SQ_F8_MFMA(0); break;
          case 1: acc[i][j] = SQ_F8_MFMA(1); break;
          case 2: acc[i][j] = SQ_F8_MFMA(2); break;
          default: acc[i][j] = SQ_F8_MFMA(3); break;
        }
#undef SQ_F8_MFMA
      }
    };
    // One stage.  Pairs of row tiles first, each contracted while the next one
    // (the last one: all H others) is read.  Then every wave has read all of the
    // stage, so its buffers take stage st + 2, and stage st + 1 has landed: under
    // the MFMAs of the H row tiles, column tile by column tile, its first row
    // tiles are read, and its column tiles as the registers fall free.  Loads
    // past the last stage fetch it again, into buffers that are not read any
    // more.
    // EARLY (7 and 8 row tiles): a second barrier behind the first pair, where the
    // column tiles and row tiles 0 to 3 are done with, lets their loads go a step
    // earlier, and each load has 1.1 to 1.4 stages to arrive instead of 0.5 to 1
    // (4480 x 16384 x 6144 gated: 906 -> 860 us, its backward 943 -> 897).
    i32x8 a[2][2], h[L ? 1 : 2][H], w[FN];
    Exps e, en;
    read_exps(e, 0);
#pragma unroll
    for (int i = 0; i < FIRST; ++i) (L ? a[0][i] : h[0][i]) = read_a(0, i);
#pragma unroll
    for (int j = 0; j < FN; ++j) w[j] = read_b(0, j);
    // s: the stage's number modulo four.  No branches: the compiler would move
    // MFMAs across them.
    auto stage = [&](int st, int s) {
      const int cur = L ? 0 : s & 1, nxt = L ? 0 : cur ^ 1;   // of h
      const int ahead = min(st + 2, ST - 1);
      Rows from{};
      if (MODE == F8_GRAD && NP == 0) from = grad_rows(ahead);
      if (s == 0) load_exps(q0 + (st >> 2) + 1);
#pragma unroll
      for (int q = 0; q < NP; ++q) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if (q + 1 < NP) {
            if (j < 2) a[(q + 1) & 1][j] = read_a(s, 2 * q + 2 + j);
          } else if (j < H) {
            h[0][j] = read_a(s, L + j);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            product(2 * q + i, j, w[j], a[q & 1][i], e);
            if constexpr (PINNED) __builtin_amdgcn_sched_barrier(0);
            if (EARLY && q == 1) {
              if (i == 0) issue_b(ahead, from, s, j);
              else if (j < 4) issue_a(ahead, s, j);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
          if (EARLY && q == 0 && j == FN - 1) sync(on_way);
          if (MODE == F8_GRAD && q == 0 && j == 0) from = grad_rows(ahead);
        }
      }
      if (s == 3) put_exps(((st >> 2) + 1) & 1);
      sync(on_way);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        auto fetch = [&]() {
          if (j < FIRST) (L ? a[0][j] : h[nxt][j]) = read_a(s + 1, j);
          if (!EARLY && j * NB / FN < (j + 1) * NB / FN) issue_b(ahead, from, s, j * NB / FN);
        };
        if (!PINNED) fetch();
#pragma unroll
        for (int i = 0; i < H; ++i) {
          product(L + i, j, w[j], h[cur][i], e);
          if constexpr (PINNED) __builtin_amdgcn_sched_barrier(0);
          if (PINNED && i == 0) fetch();
          if (i == (PINNED ? 1 : 0) && j < NA && (!EARLY || j >= 4)) issue_a(ahead, s, j);
          if (i == H / 2 && j > 0) w[j - 1] = read_b(s + 1, j - 1);
          if (i == 0 && j == 1) read_exps(en, min(st + 1, ST - 1));
        }
        if constexpr (!F16 && !PINNED) {
#pragma unroll
          for (int i = 0; i < H; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      w[FN - 1] = read_b(s + 1, FN - 1);
      e = en;
    };
    int st = 0;
    for (; st + 4 <= ST; st += 4) {
      stage(st, 0);
      stage(st + 1, 1);
      stage(st + 2, 2);
      stage(st + 3, 3);
    }
    if (st < ST) stage(st, 0);
    if (st + 1 < ST) stage(st + 1, 1);
    if (st + 2 < ST) stage(st + 2, 2);
    if constexpr (PINNED) {   // in every path here, ahead of the paths' join
#pragma unroll
      for (int i = 0; i < FM; ++i) pinned_row(acc[i]);
      pinned_wait();
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

  // ---- acc[i][j][v]: row 32 i + 16 wm + fr
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if constexpr (PINNED) pinned_row(acc[i]);
    const int r = 32 * i + 16 * wm + fr;
    const bool r_out = r >= rows;   // the lanes of the gradient's exchange differ in g alone
    if (MODE != F8_GRAD && r_out) continue;
    const int64_t row = m0 + r;
    if constexpr (MODE == F8_FWD) {
#pragma unroll
      for (int q = 0; q < FN / 2; ++q) {
        const int c = 16 * FN * wn + 32 * q + 8 * g;
        float o[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) o[t] = acc[i][2 * q + (t >> 2)][t & 3];
        if constexpr (SPLIT)
          store_run<8>(p.partial, ((int64_t)split * p.m + row) * p.n + c0 + c, o, cols - c, false);
        else
          store_run<8>(p.y, row * p.n + c0 + c, o, cols - c, p.y_bf16);
      }
    } else if constexpr (MODE == F8_GATED) {
#pragma unroll
      for (int q = 0; q < FN / 4; ++q) {
        const int c = 8 * FN * wn + 32 * q + 8 * g;
        float gv[8], uv[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          gv[t] = acc[i][2 * q + (t >> 2)][t & 3];
          uv[t] = acc[i][FN / 2 + 2 * q + (t >> 2)][t & 3];
        }
        if constexpr (SPLIT) {
          const int64_t at = ((int64_t)split * p.m + row) * (2 * (int64_t)p.n) + c0 + c;
          store_run<8>(p.partial, at, gv, cols - c, false);
          store_run<8>(p.partial, at + p.n, uv, cols - c, false);
        } else {
          const int64_t at = row * p.n + c0 + c;
          // past the L2 (4480 x 16384 x 6144 with g and u: 767 -> 721 us, h alone
          // 668 -> 658, with the product that reads h 1083 -> 1047; g and u alone
          // past it 740; one product's results, either direction: no difference)
          if (p.g) {
            store_run<8, true>(p.g, at, gv, cols - c, true);
            store_run<8, true>(p.u, at, uv, cols - c, true);
          }
          float h[8];
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            float value, slope;
            act_curve<ACT>(gv[t], value, slope);
            h[t] = value * uv[t];
          }
          store_run<8, true>(p.y, at, h, cols - c, p.y_bf16);
        }
      }
    } else {
      // column 16 j + 4 g + v: lanes g and g ^ 1 exchange four columns of tile j
      // for four of tile j + 1, which leaves each eight in a row
#pragma unroll
      for (int j = 0; j < FN; j += 2) {
        const int c = 16 * FN * wn + 16 * (j + (g & 1)) + 8 * (g >> 1);
        float o[8];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[i][j][v]),
                                                          __float_as_uint(acc[i][j + 1][v]), false, false);
          o[v] = __uint_as_float(r[0]);
          o[4 + v] = __uint_as_float(r[1]);
        }
        if (r_out) continue;
        if constexpr (SPLIT)
          store_run<8>(p.partial, ((int64_t)split * p.m + row) * p.k + c0 + c, o, cols - c, false);
        else
          store_run<8>(p.y, row * p.k + c0 + c, o, cols - c, p.y_bf16);
      }
    }
  }
}

// Sum of the splits' results in order, and what the tiles' epilogue does.  A
// workgroup takes 16 rows of one group x 64 columns, a thread four columns, with
// eight splits' values on their way at once: the sums lie in L2 and the launch's
// own latency is most of it (777 x 1003 of fp32: 5 us).
template <bool GATED>
__global__ void __launch_bounds__(256) k_f8_join(const float* __restrict__ partial,
                                                 const int32_t* __restrict__ offsets, int groups,
                                                 void* __restrict__ y, uint16_t* __restrict__ g_out,
                                                 uint16_t* __restrict__ u_out, int m, int width,
                                                 int splits, int y_bf16, int act) {
  const int tid = threadIdx.x, nt = (width + 63) >> 6, tile = (int)blockIdx.x / nt;
  RowTile rt;
  if (!find_row_tile(offsets, groups, m, 16, tile, tid & 63, rt)) return;
  const int lrow = tid >> 4, c = ((int)blockIdx.x - tile * nt) * 64 + 4 * (tid & 15);
  const int left = width - c;
  if (lrow >= rt.rows || left <= 0) return;
  const int64_t row = rt.row0 + lrow, pitch = (int64_t)width * (GATED ? 2 : 1);
  auto sum = [&](int64_t col, float (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = 0.0f;
    for (int s0 = 0; s0 < splits; s0 += 8) {
      float v[8][4];
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float* src = partial + ((int64_t)min(s0 + s, splits - 1) * m + row) * pitch + col;
        if (left >= 4) {
          __builtin_memcpy(v[s], src, 16);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[s][i] = i < left ? src[i] : 0.0f;
        }
      }
#pragma unroll
      for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += s0 + s < splits ? v[s][i] : 0.0f;
    }
  };
  float o[4];
  sum(c, o);
  if constexpr (GATED) {
    float u[4];
    sum(width + c, u);
    if (g_out) {
      store_run<4>(g_out, row * width + c, o, left, true);
      store_run<4>(u_out, row * width + c, u, left, true);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = act_value(act, o[i]) * u[i];
  }
  store_run<4>(y, row * width + c, o, left, y_bf16);
}

// ---------------------------------------------------------------- few rows
// 16 rows x 16 NT weight columns per workgroup (gated: 8 NT of gate and the same
// of up), the rows rounded on the way: lane (fr, g) holds values 16 g .. 16 g + 15
// and 64 + 16 g .. of row fr's block, as the MFMA takes them, so a block's
// maximum meets in four lanes and nothing is written in between; codes come
// straight from memory in the same order.  The waves take the blocks along the
// contraction in turn and their sums meet in LDS in wave order.  With few rows the
// codes are the whole traffic; rounding x again in every workgroup takes a third
// of the time they take to arrive (130 vector instructions against 4 KB of codes).
// One row x 16384 x 6144: 18.4 us, 101 MB at 5.5 TB/s (23 us with rounding, splits
// and join as launches of their own).
// VEC: rows of x are 16-byte aligned.
template <int NT, bool GATED, bool F16, bool VEC>
__global__ void __launch_bounds__(512) k_f8_stream(const F8Args p, const uint16_t* __restrict__ x) {
  extern __shared__ __attribute__((aligned(16))) uint8_t red[];
  constexpr int WIDTH = GATED ? 8 * NT : 16 * NT, HALF = GATED ? NT / 2 : NT;
  const int tid = threadIdx.x, lane = tid & 63, fr = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = __builtin_amdgcn_readfirstlane((int)(blockDim.x >> 6));
  const int nt = (p.n + WIDTH - 1) / WIDTH;
  const int mt = row_tile_count(p.offsets, p.groups, p.m, 16, p.most_tiles, lane);
  if ((int64_t)blockIdx.x >= (int64_t)mt * nt) return;
  int64_t tm, tn;
  xcd_tile(blockIdx.x, (int64_t)mt * nt, nt, tm, tn);
  RowTile rt;
  if (!find_row_tile(p.offsets, p.groups, p.m, 16, __builtin_amdgcn_readfirstlane((int)tm), lane, rt))
    return;
  const int grp = __builtin_amdgcn_readfirstlane(rt.group);
  const int rows = __builtin_amdgcn_readfirstlane(rt.rows);
  const int64_t m0 = __builtin_amdgcn_readfirstlane(rt.row0);
  const int c0 = __builtin_amdgcn_readfirstlane((int)tn) * WIDTH;
  const int cols = min(WIDTH, p.n - c0), ldb = 128 * p.kb;
  const int64_t brow0 = (int64_t)grp * p.n + c0;
  const __amdgpu_buffer_rsrc_t w_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.b0 + brow0 * ldb), (short)0, cols * ldb, 0x00020000);
  const __amdgpu_buffer_rsrc_t u_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((GATED ? p.b1 : p.b0) + brow0 * ldb), (short)0, cols * ldb, 0x00020000);
  const int64_t ex0 = ((int64_t)grp * p.nb + (c0 >> 7)) * p.kb;
  uint32_t off_w[HALF];   // columns past the tile repeat its last one
#pragma unroll
  for (int j = 0; j < HALF; ++j)
    off_w[j] = (uint32_t)min(16 * j + fr, cols - 1) * (uint32_t)ldb + 16u * g;
  const bool live = fr < rows;
  const uint16_t* xrow = x + (m0 + min(fr, rows - 1)) * p.k;

  struct Step {
    i32x8 w[NT];
    u32x4 x[4];
    int e[2];
  };
  const int todo = (p.kb - wave + waves - 1) / waves;   // blocks of this wave
  auto load = [&](Step& f, int t) {
    const int blk = wave + waves * t;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint32_t off = off_w[j % HALF];
      u32x4 lo, hi;
      if (GATED && j >= HALF) {
        lo = __builtin_amdgcn_raw_buffer_load_b128(u_rsrc, off, 128 * blk, 0);
        hi = __builtin_amdgcn_raw_buffer_load_b128(u_rsrc, off, 128 * blk + 64, 0);
      } else {
        lo = __builtin_amdgcn_raw_buffer_load_b128(w_rsrc, off, 128 * blk, 0);
        hi = __builtin_amdgcn_raw_buffer_load_b128(w_rsrc, off, 128 * blk + 64, 0);
      }
      f.w[j] = (i32x8){(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                       (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int col = 128 * blk + 64 * (c >> 1) + 16 * g + 8 * (c & 1), left = p.k - col;
      f.x[c] = (u32x4){0u, 0u, 0u, 0u};
      if (live && left > 0) {
        if constexpr (VEC) f.x[c] = *reinterpret_cast<const u32x4*>(xrow + col);
        else f.x[c] = load8_u16(xrow + col, left);
      }
    }
    f.e[0] = p.x0[ex0 + blk];
    f.e[1] = GATED ? p.x1[ex0 + blk] : f.e[0];
  };
  f32x4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = (f32x4){0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Step& f) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = abs_max_u16(top, f.x[i >> 2][i & 3]);
    top = u16_pair_max(top);
    const auto s16 = __builtin_amdgcn_permlane16_swap(top, top, false, false);
    top = max(s16[0], s16[1]);
    const auto s32 = __builtin_amdgcn_permlane32_swap(top, top, false, false);
    top = max(s32[0], s32[1]);
    const int e = f8_exponent(top << 16);
    const float inv = f8_inverse(e);
    i32x8 a;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const u32x2 q = f8_of_bf16x8(f.x[c], inv);
      a[2 * c] = (int)q[0];
      a[2 * c + 1] = (int)q[1];
    }
    if constexpr (F16) {
      const F16Frag ah = f8_to_f16(a);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        add_scaled(acc[j], f16_block(f8_to_f16(f.w[j]), ah), f.e[GATED && j >= HALF] + e);
    } else {
#pragma unroll
      for (int j = 0; j < NT; ++j)
        acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f.w[j], a, acc[j], 0, 0, 0,
                                                                  f.e[GATED && j >= HALF], 0, e);
    }
  };
  Step f0, f1;
  if (todo > 0) load(f0, 0);
  int t = 0;
  for (; t + 2 <= todo; t += 2) {
    load(f1, t + 1);
    compute(f0);
    if (t + 2 < todo) load(f0, t + 2);
    compute(f1);
  }
  if (t < todo) compute(f0);
#pragma unroll
  for (int j = 0; j < NT; ++j)
    *reinterpret_cast<f32x4*>(red + ((wave * NT + j) * 64 + lane) * 16) = acc[j];
  __syncthreads();
  // row fr, columns 16 j + 4 g ..
  for (int j = wave; j < HALF; j += waves) {
    auto sum = [&](int tile) {
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
      for (int w = 0; w < waves; ++w)
        o += *reinterpret_cast<const f32x4*>(red + ((w * NT + tile) * 64 + lane) * 16);
      return o;
    };
    const f32x4 s = sum(j);
    const int c = 16 * j + 4 * g, left = cols - c;
    const int64_t at = (m0 + fr) * p.n + c0 + c;
    float o[4] = {s[0], s[1], s[2], s[3]};
    if constexpr (GATED) {
      const f32x4 v = sum(HALF + j);
      const float u[4] = {v[0], v[1], v[2], v[3]};
      if (p.g && live && left > 0) {
        store_run<4>(p.g, at, o, left, true);
        store_run<4>(p.u, at, u, left, true);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = act_value(p.act, o[i]) * u[i];
    }
    if (live && left > 0) store_run<4>(p.y, at, o, left, p.y_bf16);
  }
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

// Tile and splits of the contraction: each form's time (us) is modelled and the
// least chosen.  The constants are fitted to 4900 timed shapes of both result
// types and all four products, one layer and up to 64 experts, between 1 and
// 16384 rows, widths of 64 to 16384 on both sides; over them the choice takes
// 1.01 times the best form on average.  (For fp32 results they order the forms
// but are no clock: 4480 x 6144 x 16384 takes 930 us, the model has 557; the
// factor 1.35 below makes up for that beside the form of few rows.)  What decides:
//   tiles through LDS: whole rounds of 256 tiles, one stage after another; few
//     tiles split the contraction so that every CU has one (one token x 16384 x
//     6144: 23 us with four splits, 37 with one), at the price of the partial sums'
//     trip and a launch; large tiles read less per MFMA;
//   few rows (k_f8_stream, forward only): a wave's blocks one after another, or
//     all of a CU's; wide tiles round the rows less often (above: 18 us with 64
//     columns, 24 with 16), narrow ones are more (16 x 2048 x 8192: 15 us with 16
//     columns, 25 with 64); eight waves where the tiles do not fill the chip.
struct F8Tile {
  int rows;
  double fixed, stage;   // us per round, us per stage and round
};
constexpr F8Tile kF8Tiles[] = {{64, 6.9, 0.63}, {128, 7.0, 0.86}, {224, 9.0, 1.05}, {256, 9.0, 1.18}};
constexpr F8Tile kF16Tiles[] = {{64, 6.0, 0.8}, {128, 7.5, 1.03}};
struct F8Stream {
  int cols;              // MFMA column tiles
  double block, share;   // us of a wave's block, of a block among a CU's
};
constexpr F8Stream kF8Streams[] = {{1, 0.76, 0.14}, {2, 0.98, 0.215}, {4, 1.48, 0.375}};

F8Plan plan_f8(int kind, int64_t m, int64_t n, int64_t k, int groups, bool bf16) {
  F8Plan p{};
  p.kind = kind;
  p.m = m; p.n = n; p.k = k; p.groups = groups;
  const int64_t kb = (k + 127) / 128, nb = (n + 127) / 128;
  const bool grad = kind == SQ_F8_DGRAD || kind == SQ_F8_GATED_BWD;
  const bool gated = kind == SQ_F8_GATED_FWD;
  p.stages = (int)(grad ? (kind == SQ_F8_GATED_BWD ? 2 * nb : nb) : kb);
  p.lax = (p.stages + 3) & ~3;
  p.pitch = p.stages | 1;
  p.f16 = !bf16;
  p.tile_n = gated ? 128 : 256;
  const int64_t width = grad ? k : n;
  const int quads = (p.stages + 3) / 4, least = (p.stages + F8_MAX_STAGES - 1) / F8_MAX_STAGES;
  p.splits = 1;
  double best = 1e30;
  auto consider = [&](const F8Tile& t) {
    const double tiles = i8_expected_tiles(m, groups, t.rows) *
                         (double)((width + p.tile_n - 1) / p.tile_n) / 256.0;
    for (int s = least; s <= std::min(quads, std::max(16, least)); ++s) {
      const double rounds = groups > 1 ? std::max(1.0, tiles * s + 0.25) : std::ceil(tiles * s);
      double us = rounds * (t.fixed + t.stage * (double)p.stages / s);
      if (s > 1) us += 4.0 + (double)m * (double)width * (gated ? 2 : 1) * s * 8e-6 / 4.9;
      if (us < best) {
        best = us;
        p.tile_m = t.rows;
        p.splits = s;
      }
    }
  };
  if (p.f16)
    for (const F8Tile& t : kF16Tiles) consider(t);
  else
    for (const F8Tile& t : kF8Tiles) consider(t);
  const int64_t used = std::max<int64_t>(1, std::min<int64_t>(groups, m));
  if (!grad && m <= 24 * used) {
    // what the LDS form takes more: the rows' own launch; fp16 stages of few rows
    // (and 7 us of launches and joins beside the codes' way)
    const double codes = (double)used * (double)n * (double)k * (gated ? 2 : 1) / 5.6e6;
    best = std::max(best * (p.f16 ? 1.35 : 1.0) + 3.0, codes + 7.0);
    for (const F8Stream& t : kF8Streams) {
      const int cols = (gated ? 8 : 16) * t.cols;
      if (gated && t.cols < 2) continue;
      const double tiles = i8_expected_tiles(m, groups, 16) * (double)((n + cols - 1) / cols) / 256.0;
      for (int w : {4, 8}) {
        const double slow = w == 8 && tiles > 1.5 ? 1.33 : 1.0;
        const double all = tiles * (double)kb * t.share * slow;
        const double us = std::max(
            codes * slow + 1.0,
            4.9 + 0.17 * tiles + std::max(0.9 * all, t.block * (double)((kb + w - 1) / w) + 0.1 * all));
        if (us < best) {
          best = us;
          p.tile_m = 16;
          p.tile_n = cols;
          p.waves = (int)std::min<int64_t>(w, kb);
          p.splits = 1;
        }
      }
    }
  }
  // a launch has fewer than 2^32 threads
  constexpr int64_t most = (int64_t)1 << 32;
  const int64_t tiles = i8_tile_bound(m, groups, p.tile_m) * ((width + p.tile_n - 1) / p.tile_n);
  p.ok = tiles * p.splits < most / F8_MAX_THREADS;
  if (p.splits > 1) p.ok = p.ok && i8_tile_bound(m, groups, 16) * ((width + 63) / 64) < most / 256;
  if (p.tile_m > 16)
    p.ok = p.ok && f8_rows_blocks(m, grad ? n : k, kind == SQ_F8_GATED_BWD) < most / 256;
  size_t off = 0;
  const size_t held = p.tile_m == 16 ? 0 : (size_t)m;   // rows of codes between the launches
  p.off_codes = off; off = align256(off + held * p.pitch * 128);
  p.off_exps = off;  off = align256(off + held * p.lax);
  p.off_part = off;
  off = align256(off + (p.splits > 1 ? (size_t)p.splits * m * width * (gated ? 8 : 4) : 0));
  p.total = std::max<size_t>(off, 256);   // 0 says that a call is refused
  return p;
}

hipError_t launch_f8(const F8Plan& p, const F8Call& c, void* workspace, hipStream_t stream) {
  char* base = static_cast<char*>(workspace);
  uint8_t* codes = reinterpret_cast<uint8_t*>(base + p.off_codes);
  uint8_t* exps = reinterpret_cast<uint8_t*>(base + p.off_exps);
  const bool grad = p.kind == SQ_F8_DGRAD || p.kind == SQ_F8_GATED_BWD;
  F8Args a{};
  a.a = codes; a.ax = exps;
  a.b0 = c.codes[0]; a.b1 = c.codes[1];
  a.x0 = c.exps[0]; a.x1 = c.exps[1];
  a.offsets = c.offsets;
  a.y = c.y; a.g = c.g; a.u = c.u;
  a.partial = reinterpret_cast<float*>(base + p.off_part);
  a.groups = p.groups; a.m = (int)p.m; a.n = (int)p.n; a.k = (int)p.k;
  a.kb = (int)((p.k + 127) / 128); a.nb = (int)((p.n + 127) / 128);
  a.lax = p.lax; a.pitch = p.pitch; a.stages = p.stages;
  a.y_bf16 = c.y_bf16; a.act = c.act;
  a.most_tiles = (int)i8_tile_bound(p.m, p.groups, p.tile_m);
  a.splits = p.splits;
  const int64_t width = grad ? p.k : p.n;
  const int64_t tiles = a.most_tiles * ((width + p.tile_n - 1) / p.tile_n);
  if (p.tile_m == 16) {
    const size_t lds = (size_t)p.waves * (p.tile_n / (p.kind == SQ_F8_GATED_FWD ? 8 : 16)) * 1024;
#define SQ_F8_STREAM(NT, GATED, F16, VEC)                                                         \
  hipLaunchKernelGGL((k_f8_stream<NT, GATED, F16, VEC>), dim3((unsigned)tiles), dim3(64 * p.waves), \
                     lds, stream, a, c.a)
#define SQ_F8_STREAM_TYPE(NT, GATED)                                   \
  do {                                                                 \
    if (p.f16 && p.k % 8 == 0) SQ_F8_STREAM(NT, GATED, true, true);    \
    else if (p.f16) SQ_F8_STREAM(NT, GATED, true, false);              \
    else if (p.k % 8 == 0) SQ_F8_STREAM(NT, GATED, false, true);       \
    else SQ_F8_STREAM(NT, GATED, false, false);                        \
  } while (0)
    if (p.kind == SQ_F8_GATED_FWD) {
      if (p.tile_n == 16) SQ_F8_STREAM_TYPE(2, true);
      else SQ_F8_STREAM_TYPE(4, true);
    } else {
      if (p.tile_n == 16) SQ_F8_STREAM_TYPE(1, false);
      else if (p.tile_n == 32) SQ_F8_STREAM_TYPE(2, false);
      else SQ_F8_STREAM_TYPE(4, false);
    }
#undef SQ_F8_STREAM_TYPE
#undef SQ_F8_STREAM
    return hipGetLastError();
  }
  hipError_t err =
      p.kind == SQ_F8_GATED_BWD
          ? launch_f8_gated_rows(c.a, c.g_in, c.u_in, c.act, c.offsets, p.groups, codes, exps, c.dg,
                                 c.du, p.m, p.n, p.lax, p.pitch, stream)
          : launch_f8_rows(c.a, c.offsets, p.groups, codes, exps, p.m, grad ? p.n : p.k, p.lax, p.pitch,
                           stream);
  if (err != hipSuccess) return err;
  const dim3 grid((unsigned)(tiles * p.splits));
#define SQ_F8_GEMM(FM, WN, MODE, ACT, F16, SPLIT)                                              \
  hipLaunchKernelGGL((k_f8_gemm<FM, WN, MODE, ACT, F16, SPLIT>), grid, dim3(128 * WN), 0, stream, a)
#define SQ_F8_FORM(MODE, ACT, SPLIT)                                     \
  do {                                                                   \
    if (p.f16 && p.tile_m == 64) SQ_F8_GEMM(2, 4, MODE, ACT, true, SPLIT); \
    else if (p.f16) SQ_F8_GEMM(4, 4, MODE, ACT, true, SPLIT);            \
    else if (p.tile_m == 64) SQ_F8_GEMM(2, 4, MODE, ACT, false, SPLIT);  \
    else if (p.tile_m == 128) SQ_F8_GEMM(4, 4, MODE, ACT, false, SPLIT); \
    else if (p.tile_m == 224) SQ_F8_GEMM(7, 2, MODE, ACT, false, SPLIT); \
    else SQ_F8_GEMM(8, 2, MODE, ACT, false, SPLIT);                      \
  } while (0)
  // the curve is applied by the join where the contraction is split
  if (grad && p.splits > 1) SQ_F8_FORM(F8_GRAD, 0, true);
  else if (grad) SQ_F8_FORM(F8_GRAD, 0, false);
  else if (p.kind != SQ_F8_GATED_FWD && p.splits > 1) SQ_F8_FORM(F8_FWD, 0, true);
  else if (p.kind != SQ_F8_GATED_FWD) SQ_F8_FORM(F8_FWD, 0, false);
  else if (p.splits > 1) SQ_F8_FORM(F8_GATED, 0, true);
  else if (c.act == 0) SQ_F8_FORM(F8_GATED, 0, false);
  else if (c.act == 1) SQ_F8_FORM(F8_GATED, 1, false);
  else SQ_F8_FORM(F8_GATED, 2, false);
#undef SQ_F8_FORM
#undef SQ_F8_GEMM
  if (p.splits > 1) {
    if ((err = hipGetLastError()) != hipSuccess) return err;
    const dim3 jgrid((unsigned)(i8_tile_bound(p.m, p.groups, 16) * ((width + 63) / 64)));
    if (p.kind == SQ_F8_GATED_FWD)
      hipLaunchKernelGGL(k_f8_join<true>, jgrid, dim3(256), 0, stream, a.partial, c.offsets, p.groups,
                         c.y, c.g, c.u, (int)p.m, (int)width, p.splits, c.y_bf16, c.act);
    else
      hipLaunchKernelGGL(k_f8_join<false>, jgrid, dim3(256), 0, stream, a.partial, c.offsets,
                         p.groups, c.y, nullptr, nullptr, (int)p.m, (int)width, p.splits, c.y_bf16, 0);
  }
  return hipGetLastError();
}

}  // namespace sq
