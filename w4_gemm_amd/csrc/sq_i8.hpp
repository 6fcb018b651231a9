// Device helpers of the 8-bit products (forward and input gradient of the
// int8 mode, for one layer and for experts): the map from workgroups to row
// tiles of ragged groups, and the rank-r projection of the pre-phases.
#pragma once
#include "sq_device.hpp"

namespace sq {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* i8_lds_t;

// Rows and scales are floored here so that 127 / absmax and 32512 / absmax stay finite.
constexpr float I8_MIN_ABSMAX = 0x1p-100f;
// Added to a float of magnitude below 2^22 it leaves round-to-nearest-even of
// the value as an integer in the low mantissa bits (two's complement bytes).
constexpr float I8_ROUND = 12582912.0f;   // 1.5 * 2^23
constexpr uint32_t I8_NAN_BITS = 0x7FC00000u;

// ---------------------------------------------------------------- row tiles
// Rows offsets[e] .. offsets[e+1]-1 belong to group e.  The values come from
// device memory, so no host check covers them: each range is clamped into
// [0, m] here and every access derived from it stays inside the tensors.
struct RowTile {
  int group, rows;
  int row0;
};

__device__ __forceinline__ void group_range(const int32_t* __restrict__ offsets, int groups, int m,
                                            int e, int& lo, int& hi) {
  lo = hi = 0;
  if (e < groups) {
    lo = min(max(offsets[e], 0), m);
    hi = min(max(offsets[e + 1], lo), m);
  }
}

// Number of tile_m-row tiles of all groups (offsets == null: one group of m
// rows), at most `most`: what nondecreasing offsets can need, and what the
// launch and the partial sums' buffer are sized for.
__device__ __forceinline__ int row_tile_count(const int32_t* __restrict__ offsets, int groups,
                                              int m, int tile_m, int most, int lane) {
  if (!offsets) return (m + tile_m - 1) / tile_m;
  int sum = 0;
  for (int e0 = 0; e0 < groups; e0 += 64) {
    int lo, hi;
    group_range(offsets, groups, m, e0 + lane, lo, hi);
    sum += (hi - lo + tile_m - 1) / tile_m;
  }
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) sum += __shfl_xor(sum, s);
  return min(__builtin_amdgcn_readfirstlane(sum), most);
}

// Tile t in group order; false past the last one.  All 64 lanes take part.
__device__ __forceinline__ bool find_row_tile(const int32_t* __restrict__ offsets, int groups,
                                              int m, int tile_m, int t, int lane, RowTile& out) {
  if (!offsets) {
    out.group = 0;
    out.row0 = t * tile_m;
    out.rows = min(tile_m, m - out.row0);
    return out.rows > 0;
  }
  int base = 0;
  for (int e0 = 0; e0 < groups; e0 += 64) {
    int lo, hi;
    group_range(offsets, groups, m, e0 + lane, lo, hi);
    const int cnt = (hi - lo + tile_m - 1) / tile_m;
    int inc = cnt;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int v = __shfl_up(inc, s);
      if (lane >= s) inc += v;
    }
    const uint64_t past = __ballot(base + inc > t);
    if (past) {
      const int src = __builtin_ctzll(past);
      const int first = base + __builtin_amdgcn_readlane(inc - cnt, src);
      out.group = e0 + src;
      out.row0 = __builtin_amdgcn_readlane(lo, src) + (t - first) * tile_m;
      out.rows = min(tile_m, __builtin_amdgcn_readlane(hi, src) - out.row0);
      return true;
    }
    base += __builtin_amdgcn_readlane(inc, 63);
  }
  return false;
}

// Group of a row (nondecreasing offsets); -1 for a row behind the last group.
__device__ __forceinline__ int group_of_row(const int32_t* __restrict__ offsets, int groups,
                                            int row, int lane) {
  if (!offsets) return 0;
  int e = 0;
  for (int e0 = 0; e0 < groups; e0 += 64)
    e += __popcll(__ballot(e0 + lane < groups && offsets[min(e0 + lane, groups - 1) + 1] <= row));
  return e < groups ? e : -1;
}

// ---------------------------------------------------------------- last round
// Tiles run in rounds of one per CU.  The tiles past the last whole round are
// cut along the contraction into up to max_split parts each, so that they fill
// the chip too; the parts' integer sums are joined by a second kernel.
constexpr int I8_CUS = 256;
struct Tail {
  int full, splits;   // tiles before the tail; parts per tail tile (1: no split)
};
__host__ __device__ __forceinline__ Tail tile_tail(int tiles, int max_split) {
  const int rem = tiles % I8_CUS;
  int s = rem > 0 ? I8_CUS / rem : 1;
  s = s < max_split ? s : max_split;
  Tail t;
  t.splits = s > 1 ? s : 1;
  t.full = t.splits > 1 ? tiles - rem : tiles;
  return t;
}

// Eight consecutive 16-bit values from a 2-byte aligned address (one load:
// the hardware takes unaligned vector loads); values at or past `left` read
// as zero and are not touched in memory.
__device__ __forceinline__ u32x4 load8_u16(const uint16_t* __restrict__ p, int left) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (left >= 8) {
    __builtin_memcpy(&v, p, 16);
  } else {
    for (int i = 0; i < left; ++i) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  }
  return v;
}

// ---------------------------------------------------------------- rank-r projection
// t_part[slice][row][r] = sum over the slice's columns of a[row][c] fac[c][r]
// for the 16 RW rows of one tile: a bf16 [m][cols], fac bf16 [cols][rank] (the
// group's factor), exact products and fp32 sums on bf16 MFMA.  The workgroup's
// waves take the slice's 64-column units (a line of a row) in turn and their sums are added in
// wave order, so the result does not depend on timing.  Each wave stages 32
// factor rows at a time in its own LDS (64 rank bytes) and reads them
// transposed (eight consecutive c of one rank column per lane); the loads of
// the next 32 columns are in flight meanwhile.  RW = 2 reads the factor once
// for 32 rows; RW = 1 gives few rows to more workgroups.
// VEC: cols is a multiple of eight and a is 16-byte aligned.
// mem: dynamic LDS, 64 * rank bytes per wave (also holds the partial sums).
template <int RANK, int RW, bool VEC>
__device__ __forceinline__ void project_tile(const uint16_t* __restrict__ a,
                                             const uint16_t* __restrict__ fac,
                                             float* __restrict__ t_part, uint8_t* mem, int m,
                                             int cols, const RowTile& rt, int slice, int slices) {
  constexpr int RT = RANK / 16;
  const int tid = threadIdx.x, lane = tid & 63, fr = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int units = (cols + 63) >> 6;
  const int b0 = (int)((int64_t)slice * units / slices);
  const int b1 = (int)((int64_t)(slice + 1) * units / slices);
  uint8_t* stage = mem + wave * 64 * RANK;
  const uint16_t* arow[RW];   // rows past the tile repeat its last row
#pragma unroll
  for (int i = 0; i < RW; ++i)
    arow[i] = a + (int64_t)(rt.row0 + min(16 * i + fr, rt.rows - 1)) * cols;
  struct Step {
    u32x4 a[RW], f[RT];
  };
  const int steps = max(b1 - b0 - wave + waves - 1, 0) / waves * 2;   // 32 columns each
  auto load = [&](Step& st, int q) {
    const int c0 = (b0 + wave + waves * (q >> 1)) * 64 + 32 * (q & 1);
    const int ca = c0 + 8 * g;
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      if constexpr (VEC) {
        st.a[i] = (u32x4){0u, 0u, 0u, 0u};
        if (ca < cols) st.a[i] = *reinterpret_cast<const u32x4*>(arow[i] + ca);
      } else {
        st.a[i] = load8_u16(arow[i] + ca, cols - ca);
      }
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int q16 = 64 * j + lane;             // 16-byte chunk of the 32 rows
      const int c = c0 + q16 / (RANK / 8);
      st.f[j] = (u32x4){0u, 0u, 0u, 0u};
      if (c < cols)
        st.f[j] = *reinterpret_cast<const u32x4*>(fac + (int64_t)c * RANK + 8 * (q16 % (RANK / 8)));
    }
  };
  f32x4 acc[RW][RT];
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
  auto use = [&](const Step& st) {
#pragma unroll
    for (int j = 0; j < RT; ++j)
      *reinterpret_cast<u32x4*>(stage + 16 * (64 * j + lane)) = st.f[j];
    __builtin_amdgcn_s_waitcnt(SQ_WAIT_LGKM0);
    __builtin_amdgcn_wave_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    s16x8 bv[RT];
#pragma unroll
    for (int r16 = 0; r16 < RT; ++r16) {
      // transposed reads of four rows each: lane 4j + q of a 16-lane group
      // points at row j, columns 4q..4q+3; lane i receives column i
      s16x4 h[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = 8 * g + 4 * u + (fr >> 2), col = 16 * r16 + 4 * (fr & 3);
        h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(stage + 2 * (row * RANK + col)));
      }
      bv[r16] = __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
    }
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
      for (int r16 = 0; r16 < RT; ++r16)
        acc[i][r16] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, st.a[i]), __builtin_bit_cast(bf16x8, bv[r16]), acc[i][r16],
            0, 0, 0);
    __builtin_amdgcn_s_waitcnt(SQ_WAIT_LGKM0);   // the reads are done before the next write
    __builtin_amdgcn_wave_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
  };
  Step s0, s1;
  if (steps > 0) load(s0, 0);
  for (int q = 0; q < steps; q += 2) {   // an even number of steps
    load(s1, q + 1);
    use(s0);
    if (q + 2 < steps) load(s0, q + 2);
    use(s1);
  }
  // acc[i][r16][v]: row 16 i + 4g + v, rank column 16 r16 + fr
  float* red = reinterpret_cast<float*>(stage);
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int left = min(rt.rows - 16 * i, 16);
    if (left <= 0) break;
    if (i > 0) __syncthreads();   // the sums of the 16 rows before are read
#pragma unroll
    for (int r16 = 0; r16 < RT; ++r16)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[(4 * g + v) * RANK + 16 * r16 + fr] = acc[i][r16][v];
    __syncthreads();
    for (int e = tid; e < left * RANK; e += blockDim.x) {
      float t = 0.0f;
      for (int w = 0; w < waves; ++w) t += reinterpret_cast<const float*>(mem + w * 64 * RANK)[e];
      t_part[((int64_t)slice * m + rt.row0 + 16 * i) * RANK + e] = t;
    }
  }
}

// Workgroup b of the projection: row tile b / slices, slice b % slices.
template <int RANK, int RW, bool VEC>
__device__ __forceinline__ void project(const uint16_t* __restrict__ a,
                                        const uint16_t* __restrict__ fac,
                                        const int32_t* __restrict__ offsets, int groups,
                                        float* __restrict__ t_part, uint8_t* mem, int m, int cols,
                                        int b, int slices) {
  RowTile rt;
  if (!find_row_tile(offsets, groups, m, 16 * RW, b / slices, threadIdx.x & 63, rt)) return;
  const uint16_t* f = fac + (int64_t)rt.group * cols * RANK;
  project_tile<RANK, RW, VEC>(a, f, t_part, mem, m, cols, rt, b % slices, slices);
}

// t of one row, eight rank columns from r0, summed over the slices in order
// and split into three bf16 parts: hi + lo hold t to 2^-16, the third to 2^-24.
__device__ __forceinline__ void project_sum8(const float* __restrict__ t_part, int m, int rank,
                                             int slices, int row, int r0, u32x4 (&part)[3]) {
  float t[8] = {};
  const float* p = t_part + (int64_t)row * rank + r0;
  const int64_t step = (int64_t)m * rank;
  // four slices' loads in flight; a slice past the last one adds zero
  for (int s = 0; s < slices; s += 4) {
    f32x4 v[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const f32x4* q = reinterpret_cast<const f32x4*>(p + min(s + u, slices - 1) * step);
      v[u][0] = q[0];
      v[u][1] = q[1];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] += s + u < slices ? v[u][i >> 2][i & 3] : 0.0f;
  }
#pragma unroll
  for (int q = 0; q < 3; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t p = pack_bf16x2(t[2 * i], t[2 * i + 1]);
      part[q][i] = p;
      t[2 * i] -= __uint_as_float(p << 16);
      t[2 * i + 1] -= __uint_as_float(p & 0xFFFF0000u);
    }
}

}  // namespace sq
