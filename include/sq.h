/* sq.h - C ABI of libsq, the MI355X (gfx950) W4 quantized-frozen-base linear layer.
 *
 * The layer is the SquareQ v3 W4 format (SquareQ README, section "SquareQ v3 -
 * W4 (Hadamard-256 + low-rank + int4 / NVFP4)", the format formula and its
 * "Rotation", "Residual codecs" and "Low-rank branch" bullets):
 *
 *     W_hat = lora_up @ lora_down^T + dequant(R) @ H
 *
 * H is the block-diagonal normalized Hadamard-256 rotation along the input
 * dimension K (Sylvester order, entries +-1/16, symmetric and its own inverse),
 * R holds int4 codes with one fp16 scale per group of 32 or 64 consecutive
 * values along K, and lora_up / lora_down are the bf16 rank-r factors of an
 * SVD of the weight.
 *
 * Conventions for every entry point:
 *   - Tensor pointers are DEVICE pointers owned by the caller.  The library
 *     allocates no device memory and keeps no state besides a per-device
 *     architecture check.  Calls are reentrant.
 *   - Arguments are validated synchronously on the host; on any error nothing
 *     is launched and the status says why.  Kernel work is enqueued on
 *     `stream` (a hipStream_t; NULL means the null stream) and is asynchronous:
 *     the library never synchronizes.
 *   - There is exactly one device code path per call and no host fallback: a
 *     device that is not gfx950 gets SQ_E_ARCH.
 *   - All tensors are dense and row-major; every pointer must be 16-byte
 *     aligned (SQ_E_ALIGN).
 *   - *_workspace_bytes(m, ...) is what a call of exactly m rows needs.  Fewer
 *     rows can need more (they split the contraction, whose partial sums lie
 *     there), so scratch for calls of several m is the largest of their sizes.
 */
#ifndef SQ_H
#define SQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SQ_ABI_VERSION 1

typedef enum {
  SQ_OK = 0,
  SQ_E_NULL = 1,      /* a required pointer is NULL                               */
  SQ_E_SHAPE = 2,     /* K % 256 != 0, K < 256, N < 1 or M < 0; the W4 input      */
                      /* gradient also needs N % 64 == 0; the 8-bit products      */
                      /* have upper limits (stated there) and need groups >= 1;   */
                      /* the 8-bit float mode takes any N and K from 1 to 2^20    */
  SQ_E_GROUP = 3,     /* group is not 32 or 64                                    */
  SQ_E_RANK = 4,      /* rank is not 0, 32 or 64 (the int8 and MXFP4 modes also  */
                      /* take 16); see the note on ranks below                    */
  SQ_E_ALIGN = 5,     /* a pointer is not 16-byte aligned                         */
  SQ_E_WORKSPACE = 6, /* workspace smaller than the matching *_workspace_bytes()  */
  SQ_E_DTYPE = 7,     /* output dtype is not SQ_F32 or SQ_BF16                    */
  SQ_E_ARCH = 8,      /* the current device is not gfx950                         */
  SQ_E_HIP = 9,       /* a HIP runtime call or kernel launch failed               */
  SQ_E_ACT = 10       /* the gated block's activation is not one of sq_act_t      */
} sq_status_t;

typedef enum { SQ_F32 = 0, SQ_BF16 = 1 } sq_dtype_t;

/* Bits OR-ed into *dev_flags by the quantizer (read them after a sync). */
enum {
  SQ_FLAG_NONFINITE = 1,      /* a weight value, or the residual, is NaN or +-inf      */
  SQ_FLAG_SCALE_OVERFLOW = 2, /* absmax/7 of some group (int8 mode: absmax/127 of some */
                              /* row) overflows fp16                                   */
  SQ_FLAG_FP16_RANGE = 4      /* W4 only: some chosen scale exceeds 8188, so the       */
                              /* payload is outside the forward's domain (below)       */
};

/* Ranks.  The page's low-rank branch is rank 32.  The W4 entry points take
 * rank 0, 32 or 64: their kernels walk the factors in 32-wide steps and the
 * input gradient reads whole steps, so rank 16 is refused with SQ_E_RANK
 * rather than read past the factors.  The int8 and MXFP4 modes also take 16
 * (the page's v3.1 split rank).
 *
 * Domain of the W4 forward and input gradient.  Their contraction runs on
 * fp16 MFMA with the weight operand fp16(q * s), q in [-8, 7]; it is finite
 * for every payload whose scales all satisfy 8 * |s| <= 65504, that is
 * |s| <= 8188 (the largest fp16 value below 2^13).  A payload with a larger
 * scale is outside the domain: the products overflow fp16 and y (or dx) holds
 * +-inf or NaN where such a group contributes.  sq_quantize_weight never
 * emits such a payload silently: it sets SQ_FLAG_FP16_RANGE.  Scales in the
 * fp16 subnormal range are inside the domain (q * s is then exact or rounded
 * once, like any other product).  The reconstruct works in fp32 and has no
 * such limit. */

/* The W4 payload of one linear layer with N output and K input features.
 *   codes     uint8  [n][k/2]  byte b of a row = (q[2b] & 0xF) | (q[2b+1] & 0xF) << 4,
 *                              q in [-8, 7] two's complement (even k in the low nibble)
 *   scales    fp16   [n][k/group]  IEEE binary16 bit patterns
 *   lora_up   bf16   [n][rank]     (may be NULL iff rank == 0)
 *   lora_down bf16   [k][rank]     (may be NULL iff rank == 0)
 * Scale g of row n covers q[n][g*group .. g*group+group-1]; those values are
 * coordinates after the rotation, so dequant(R)[n][k] = q[n][k] * s[n][k/group]. */
typedef struct {
  int64_t n, k;
  int32_t group, rank;
  uint8_t *codes;
  uint16_t *scales;
  uint16_t *lora_up;
  uint16_t *lora_down;
} sq_w4_t;

/* Builder side (the format formula read right to left, the "Residual codecs"
 * bullet): quantize the fp32 weight w [n][k].
 *   E = w - lora_up @ lora_down^T           (fp32; the factors are read from p)
 *   R = E @ H                                (block Hadamard-256 along k)
 *   for every group of `group` values of R with absmax a and every
 *   i = 0..30: s_i = fp16(round((70+i)/100 * a / 7)),
 *   q = clamp(round_half_even(r / s_i), -8, 7) (q = 0 when s_i == 0),
 *   err_i = sum (r - q s_i)^2; the first i with the least err wins.
 * Writes p->codes, p->scales and, when fidx != NULL, fidx[n][k/group] = i
 * (uint8).  Non-finite inputs and fp16 scale overflow set bits in *dev_flags
 * (device int32, required; the library only ORs bits into it, so clear it
 * first); outputs are then unspecified but written in bounds.  A chosen scale
 * above 8188 sets SQ_FLAG_FP16_RANGE: the payload is then exact as a format
 * (reconstruct handles it) but outside the forward's domain. */
sq_status_t sq_quantize_weight(const float *w, const sq_w4_t *p, uint8_t *fidx,
                               int32_t *dev_flags, void *stream);

/* Forward (the format formula applied to x; H is symmetric so
 * x @ (dequant(R) @ H)^T = (x @ H) @ dequant(R)^T):
 *   y[m][n] = sum_k (x @ H)[m][k] * q[n][k] * s[n][k/group]
 *           + sum_r (x @ lora_down)[m][r] * lora_up[n][r]
 * x is bf16 [m][k]; y is fp32 or bf16 [m][n] (bf16 = round-to-nearest-even of
 * the fp32 result).  The contraction runs on fp16 MFMA: each row of x @ H is
 * scaled by a power of two that keeps it inside fp16 range and rounded to
 * fp16, the weight operand is fp16(q * s); accumulation is fp32.
 * `workspace` is device scratch of at least sq_linear_fwd_workspace_bytes(m, p)
 * bytes, owned by the caller and not read before it is written.  m == 0 is a
 * no-op that returns SQ_OK. */
size_t sq_linear_fwd_workspace_bytes(int64_t m, const sq_w4_t *p);
sq_status_t sq_linear_fwd(const uint16_t *x, int64_t m, const sq_w4_t *p, void *y,
                          sq_dtype_t y_dtype, void *workspace, size_t workspace_bytes,
                          void *stream);

/* The same forward in its two halves; sq_linear_fwd is exactly
 * sq_linear_fwd_rotate followed by sq_linear_fwd_contract on one stream.
 *   rotate:   reads x, p->lora_down; writes into `workspace` the fp16 rotated
 *             activations, the row powers of two and the rank-r projection
 *             x @ lora_down.
 *   contract: reads that workspace and the payload; writes y.
 * For m <= 16 the rotation and the projection run inside the contraction
 * (the whole call streams the payload once from its first cycle): there
 * rotate only copies x and p->lora_down into the workspace, and contract
 * does the rest from those copies.
 * Both take the same m, p and workspace; contract must follow a rotate of the
 * same x on the same workspace (stream order suffices). */
sq_status_t sq_linear_fwd_rotate(const uint16_t *x, int64_t m, const sq_w4_t *p, void *workspace,
                                 size_t workspace_bytes, void *stream);
sq_status_t sq_linear_fwd_contract(int64_t m, const sq_w4_t *p, void *y, sq_dtype_t y_dtype,
                                   void *workspace, size_t workspace_bytes, void *stream);

/* The forward without a workspace argument, for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation.  It computes exactly what sq_linear_fwd computes
 * (same kernels, bit-identical y) with its scratch in a library-owned static
 * device array of SQ_FWD_STATIC_SCRATCH_BYTES (64 MiB), one per device, held
 * by each device the library runs on until the process ends.  It allocates
 * nothing itself; its first call on a device looks up that device's copy of
 * the array.  A call whose sq_linear_fwd_workspace_bytes(m, p) exceeds the
 * array returns SQ_E_WORKSPACE and launches nothing (every m <= 16 forward
 * fits, and so does 4480 x 16384 x 6144).  All calls on one device share the
 * array: calls ordered on one stream are fine, calls that overlap in time on
 * one device (different streams, no ordering) race and give undefined y.
 * Nothing in the array needs to be zero: each call writes what it reads. */
#define SQ_FWD_STATIC_SCRATCH_BYTES ((size_t)64 << 20)
sq_status_t sq_linear_fwd_static(const uint16_t *x, int64_t m, const sq_w4_t *p, void *y,
                                 sq_dtype_t y_dtype, void *stream);

/* Backward side: rebuild the dense bf16 weight from the same payload
 *   w_hat[n][k] = bf16_round_nearest_even( lora_up @ lora_down^T + dequant(R) @ H )
 * with every intermediate in fp32 and one rounding at the end. */
sq_status_t sq_reconstruct_bf16(const sq_w4_t *p, uint16_t *w_hat, void *stream);

/* Input gradient (the format formula transposed: dx = dy @ W_hat; where the
 * page's backward first rebuilds the dense bf16 weight, this contracts the
 * packed codes directly, and H H = I moves the rotation to the end):
 *   dx = (dy @ dequant(R)) @ H + (dy @ lora_up) @ lora_down^T, that is
 *   dx[m][k] = sum_j ( sum_n dy[m][n] q[n][j] s[n][j/group] ) H[j][k]
 *            + sum_r (dy @ lora_up)[m][r] lora_down[k][r].
 * dy is bf16 [m][n]; dx is fp32 or bf16 [m][k] (bf16 = round-to-nearest-even
 * of the fp32 result).  N must be a multiple of 64.  The int4 contraction runs
 * on fp16 MFMA with the same operand treatment as the forward: each row of dy
 * is scaled by a power of two and rounded to fp16, the weight operand is
 * fp16(q * s), accumulation is fp32; the rank-r term is carried as bf16 hi +
 * lo parts.  `workspace` is device scratch of at least
 * sq_linear_dgrad_workspace_bytes(m, p) bytes (0 for unsupported shapes),
 * owned by the caller and not read before it is written.  m == 0 is a no-op
 * that returns SQ_OK. */
size_t sq_linear_dgrad_workspace_bytes(int64_t m, const sq_w4_t *p);
sq_status_t sq_linear_dgrad(const uint16_t *dy, int64_t m, const sq_w4_t *p, void *dx,
                            sq_dtype_t dx_dtype, void *workspace, size_t workspace_bytes,
                            void *stream);

/* ------------------------------------------------------------------------
 * int8-residual mode (SquareQ README, section "v3.1 - int8-residual mode": the
 * same format formula with an int8 residual left by a rank-16 split).  The
 * page names the mode without its details; this library reads it as the W4
 * sweep on the int8 grid with one scale per output row:
 *   W_hat = lora_up @ lora_down^T + dequant(R) @ H,  dequant(R)[n][k] = q[n][k] * s[n]
 * The payload of one layer:
 *   codes     int8   [n][k]     q in [-128, 127], coordinates after the rotation
 *   scales    fp16   [n]        one scale per output row (IEEE binary16 bits)
 *   lora_up   bf16   [n][rank]  rank 0, 16, 32 or 64 (16 is the page's)
 *   lora_down bf16   [k][rank]
 * `reserved` must be 0.  Shapes, alignment, streams and errors follow the W4
 * conventions above. */
typedef struct {
  int64_t n, k;
  int32_t rank, reserved;
  int8_t *codes;
  uint16_t *scales;
  uint16_t *lora_up;
  uint16_t *lora_down;
} sq_w8_t;

/* Builder side of the int8 mode: quantize the fp32 weight w [n][k].
 *   E = w - lora_up @ lora_down^T ;  R = E @ H
 *   per row with absmax a and for i = 0..30: s_i = fp16(round((70+i)/100 * a / 127)),
 *   q = clamp(round_half_even(r / s_i), -128, 127) (q = 0 when s_i == 0),
 *   err_i = sum over the row of (r - q s_i)^2; the first i with the least err wins.
 * Writes p->codes, p->scales and, when fidx != NULL, fidx[n] = i (uint8).
 * `workspace` (device, caller-owned, at least
 * sq_quantize_weight_w8_workspace_bytes(p) bytes) holds the rotated residual
 * in fp32 between the rotation and the sweep.  dev_flags as for
 * sq_quantize_weight. */
size_t sq_quantize_weight_w8_workspace_bytes(const sq_w8_t *p);
sq_status_t sq_quantize_weight_w8(const float *w, const sq_w8_t *p, uint8_t *fidx,
                                  int32_t *dev_flags, void *workspace, size_t workspace_bytes,
                                  void *stream);

/* Rebuild the dense bf16 weight of an int8-mode payload:
 *   w_hat[n][k] = bf16_round_nearest_even( lora_up @ lora_down^T + (q * s[n]) @ H )
 * with the rotation summed exactly on integers, one fp32 rounding for the
 * scale, the rank-r term added in fp32 and one rounding at the end. */
sq_status_t sq_reconstruct_bf16_w8(const sq_w8_t *p, uint16_t *w_hat, void *stream);

/* Forward of an int8-mode payload:
 *   y[m][n] = s[n] * sum_k (x @ H)[m][k] q[n][k] + sum_r (x @ lora_down)[m][r] lora_up[n][r]
 * x bf16 [m][k], y fp32 or bf16 [m][n].  The contraction runs on fp16 MFMA
 * with the activations treated as in sq_linear_fwd (a power of two per row,
 * rounded to fp16) and the codes exact in fp16; the row scale multiplies the
 * fp32 sum.  `workspace` is caller-owned device scratch of at least
 * sq_linear_fwd_w8_workspace_bytes(m, p) bytes; m == 0 is a no-op. */
size_t sq_linear_fwd_w8_workspace_bytes(int64_t m, const sq_w8_t *p);
sq_status_t sq_linear_fwd_w8(const uint16_t *x, int64_t m, const sq_w8_t *p, void *y,
                             sq_dtype_t y_dtype, void *workspace, size_t workspace_bytes,
                             void *stream);

/* 8-bit forward of an int8-mode payload (W8A8: 8-bit tokens, 8-bit weights;
 * half the matrix time of sq_linear_fwd_w8, with the error of 8-bit tokens):
 *   y[m][n] = s[m] * p->scales[n] * sum_k q[m][k] * codes[n][k]
 *           + sum_r (x @ lora_down)[m][r] lora_up[n][r]
 * with q and s the 8-bit integers and the scale of row m of x @ H:
 *   each block of 256 values with absmax below 2^e (e as small as that allows,
 *   at least -125) is held as integers X = trunc(x 2^(23 - e)); R = X S with S
 *   the +-1 Sylvester matrix, exact in int32; r = fp32(R) 2^(e - 27);
 *   a = max(max_k |r|, 2^-100); s = fp32(a / 127); i = fp32(127 / a);
 *   q = round_half_even(fp32(r i)), |q| <= 127.
 * Every step is one correctly rounded operation, so q and s depend on the row
 * alone.  The integer sum is exact; the scales and the rank-r term (t = x @
 * lora_down summed in fp32, carried as a sum of two bf16 parts for bf16 results
 * and three for fp32 ones) are applied in fp32.  A row of x that holds inf or
 * NaN, or whose x @ H overflows fp32, gives a row of NaN and touches no other
 * row.
 * x bf16 [m][k], y fp32 or bf16 [m][n] (bf16 = RNE of the fp32 result).
 * K <= 65536 (SQ_E_SHAPE).  `workspace`: caller-owned device scratch of at
 * least sq_linear_fwd_w8a8_workspace_bytes(m, p) bytes (0 for unsupported
 * shapes), not read before it is written; m == 0 is a no-op. */
size_t sq_linear_fwd_w8a8_workspace_bytes(int64_t m, const sq_w8_t *p);
sq_status_t sq_linear_fwd_w8a8(const uint16_t *x, int64_t m, const sq_w8_t *p, void *y,
                               sq_dtype_t y_dtype, void *workspace, size_t workspace_bytes,
                               void *stream);

/* Input gradient of the int8 mode (dx = dy @ W_hat; the backward of both
 * int8-mode forwards, the tokens' rounding passed straight through):
 *   dx = (t / 16) * ((d @ codes) S) + (dy @ lora_up) @ lora_down^T
 * with d and t the 16-bit integers and the scale of each row of
 * v = fp32(dy[m][n] * scales[n]):
 *   a = max(max_n |v|, 2^-100); t = fp32(a / 32512); i = fp32(32512 / a);
 *   d = round_half_even(fp32(v i)), |d| <= 32512,
 * that is a step of 2^-15 of the row's largest value, for all of the row.
 * d @ codes is exact in integers; the rest is fp32.  Against dy @ W_hat a row of
 * dx is off by about 2^-16 sqrt(N / 3) max|v| / |v| of its norm (|v| the row's
 * 2-norm): 4e-5 for Gaussian rows of 4096 values, up to 6e-4 where one value
 * outweighs the others, 3e-3 at N = 131072.  An fp32 dx holds no more bits
 * than that; sq_linear_dgrad, whose rows are fp16, keeps 2^-11 of each value
 * down to 2^-25 of the row's largest.
 * A row that holds inf or NaN, or whose v overflows fp32, gives a row of NaN
 * and touches no other row.  dy bf16 [m][n], dx fp32 or bf16 [m][k].  Any
 * N <= 131072 (no multiple needed), K <= 65536, m <= 2^25 (2^23 for N > 2048).
 * Workspace and m == 0 as above. */
size_t sq_linear_dgrad_w8_workspace_bytes(int64_t m, const sq_w8_t *p);
sq_status_t sq_linear_dgrad_w8(const uint16_t *dy, int64_t m, const sq_w8_t *p, void *dx,
                               sq_dtype_t dx_dtype, void *workspace, size_t workspace_bytes,
                               void *stream);

/* The two calls above over several experts: `groups` int8-mode payloads of one
 * shape, stacked in p (codes [groups][n][k], scales [groups][n], lora_up
 * [groups][n][rank], lora_down [groups][k][rank]; p->n and p->k are one
 * expert's).  Rows are sorted by expert: expert e takes rows
 * offsets[e] .. offsets[e+1]-1 of x and y (dy and dx).  offsets is a device
 * array of groups + 1 nondecreasing int32, read when the kernels run, so a
 * captured graph follows new contents.  An expert may have no rows.  Rows
 * before offsets[0] and from offsets[groups] on are left as they were.  Each
 * value is clamped into [0, m] on the device, so wrong offsets give wrong
 * rows but no access outside the tensors.  groups >= 1, m < 2^31 and
 * ceil(m / 16) * groups < 2^31 (the device counts tiles in 32 bits); offsets
 * is 16-byte aligned like every pointer. */
size_t sq_grouped_fwd_w8a8_workspace_bytes(int64_t m, int32_t groups, const sq_w8_t *p);
sq_status_t sq_grouped_fwd_w8a8(const uint16_t *x, int64_t m, const int32_t *offsets,
                                int32_t groups, const sq_w8_t *p, void *y, sq_dtype_t y_dtype,
                                void *workspace, size_t workspace_bytes, void *stream);
size_t sq_grouped_dgrad_w8_workspace_bytes(int64_t m, int32_t groups, const sq_w8_t *p);
sq_status_t sq_grouped_dgrad_w8(const uint16_t *dy, int64_t m, const int32_t *offsets,
                                int32_t groups, const sq_w8_t *p, void *dx, sq_dtype_t dx_dtype,
                                void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * MXFP4 mode (SquareQ README, "SquareQ v3 - W4", the "Residual codecs"
 * bullet's FP4 alternative for native FP4 matrix instructions, and the
 * op-level parity line that describes the FP4 forward as rotate +
 * block-quant of the activations + FP4 product + epilogue).  The page's
 * NVFP4 layout targets one vendor's instructions; this library uses the OCP
 * MX counterpart that gfx950's scaled MFMA takes:
 *   element  FP4 E2M1, magnitudes {0, 0.5, 1, 1.5, 2, 3, 4, 6}, nibble
 *            s<<3 | e<<1 | m; a value that rounds to magnitude 0 is nibble 0
 *   block    32 consecutive values along K share an E8M0 byte e (scale
 *            2^(e-127)), e = floor(log2 absmax) - 2 + 127 clamped to [0, 254]
 *            (0 for an all-zero block)
 *   rounding v / 2^(e-127) to the nearest E2M1 value, ties to the even
 *            mantissa, magnitudes above 6 saturate to 6
 * The payload of one layer:
 *   codes     uint8 [n][k/2]   two nibbles per byte, even k in the low nibble,
 *                              coordinates after the rotation
 *   exps      uint8 [n][k/32]  E8M0 block exponents
 *   lora_up   bf16  [n][rank], lora_down bf16 [k][rank]  (rank 0, 16, 32, 64)
 * `reserved` must be 0.  Shapes, alignment, streams and errors follow the W4
 * conventions above. */
typedef struct {
  int64_t n, k;
  int32_t rank, reserved;
  uint8_t *codes;
  uint8_t *exps;
  uint16_t *lora_up;
  uint16_t *lora_down;
} sq_mx4_t;

/* Builder side: codes/exps = MXFP4 of R = (w - lora_up @ lora_down^T) @ H,
 * w fp32 [n][k].  Non-finite values of R set SQ_FLAG_NONFINITE in *dev_flags
 * (outputs are then unspecified but written in bounds). */
sq_status_t sq_quantize_weight_mx4(const float *w, const sq_mx4_t *p, int32_t *dev_flags,
                                   void *stream);

/* Activation half of the forward: xq [m][k/2] / xs [m][k/32] = MXFP4 of
 * x @ H, x bf16 [m][k] (device buffers owned by the caller). */
sq_status_t sq_quantize_act_mx4(const uint16_t *x, int64_t m, int64_t k, uint8_t *xq,
                                uint8_t *xs, void *stream);

/* w_hat[n][k] = bf16_round_nearest_even( lora_up @ lora_down^T + dq(codes, exps) @ H ),
 * the rotation summed in fp32 (exact before the block scales), one rounding
 * at the end. */
sq_status_t sq_reconstruct_bf16_mx4(const sq_mx4_t *p, uint16_t *w_hat, void *stream);

/* Forward: y[m][n] = sum_k dq(Q(x @ H))[m][k] dq(codes, exps)[n][k]
 *                  + sum_r (x @ lora_down)[m][r] lora_up[n][r]
 * with Q the MXFP4 quantization above (the activations are quantized inside
 * the call, as sq_quantize_act_mx4 does), the FP4 product on
 * v_mfma_scale_f32_16x16x128_f8f6f4 with fp32 accumulation, and the rank-r
 * term from the unquantized x (fp32, carried as bf16 hi + lo).  y fp32 or
 * bf16 (RNE of the fp32 result).  `workspace`: caller-owned device scratch
 * of at least sq_linear_fwd_mx4_workspace_bytes(m, p) bytes; m == 0 is a
 * no-op. */
size_t sq_linear_fwd_mx4_workspace_bytes(int64_t m, const sq_mx4_t *p);
sq_status_t sq_linear_fwd_mx4(const uint16_t *x, int64_t m, const sq_mx4_t *p, void *y,
                              sq_dtype_t y_dtype, void *workspace, size_t workspace_bytes,
                              void *stream);

/* ------------------------------------------------------------------------
 * 8-bit float mode: layers held as they are, without rotation and without a
 * low-rank branch, in OCP FP8 E4M3 codes with a power of two per block of 128
 * (floating codes keep the same relative precision for small and for large
 * values, which is what the other modes' rotation buys integers).  Powers of
 * two because gfx950's scaled MFMA applies them, and because the codes then
 * depend on the values alone:
 *   block     weight: 128 x 128 values of [n][k]; rows of a product's input: 128
 *             consecutive values along the contraction (the last ones shorter)
 *   exponent  byte e + 127 with the least e >= -127 for which the block's
 *             absmax <= 448 * 2^e (0 for a block of zeros); 255 where the block
 *             holds inf or NaN
 *   code      v / 2^e to the nearest E4M3 value, ties to the even mantissa
 * The payload of one layer with N output and K input features, 1 <= N, K <=
 * SQ_F8_MAX, kp = K rounded up to 128:
 *   codes     uint8 [n][kp]   E4M3 (no infinities, 0x7F and 0xFF NaN); columns
 *                             from k on must be zero
 *   exps      uint8 [ceil(n/128)][kp/128]
 * Alignment, streams, workspaces and errors follow the W4 conventions above. */
#define SQ_F8_MAX ((int64_t)1 << 20)
typedef struct {
  int64_t n, k;
  uint8_t *codes;
  uint8_t *exps;
} sq_f8_t;

/* Builder side: codes and exponents of w [n][k], fp32 or bf16 (dense, no
 * padding).  A block that holds inf or NaN sets SQ_FLAG_NONFINITE in *dev_flags
 * (as for sq_quantize_weight) and gets exponent 255, NaN codes for those values
 * and zeros for the others; every result that the block takes part in is then
 * unspecified.  At most 2^24 - 1 blocks (SQ_E_SHAPE). */
sq_status_t sq_quantize_weight_f8(const void *w, sq_dtype_t w_dtype, const sq_f8_t *p,
                                  int32_t *dev_flags, void *stream);

/* Products.  With Q the rounding above of a row's blocks and W the values that
 * codes and exps stand for:
 *   sq_linear_fwd_f8     y  = Q(x) W^T        x  bf16 [m][k], y  [m][n]
 *   sq_linear_dgrad_f8   dx = Q(dy) W         dy bf16 [m][n], dx [m][k]
 * (the input gradient of the layer, the rows' rounding passed straight through;
 * blocks of dy lie along n).  The gated block, for two layers of one shape and
 * act(g) = g s(g) (SiLU, s the logistic function), g Phi(g) (GELU) or its tanh
 * form g s(2 sqrt(2/pi) (g + 0.044715 g^3)):
 *   sq_gated_fwd_f8      h = act(g) u, g = Q(x) Wgate^T, u = Q(x) Wup^T
 *   sq_gated_bwd_f8      dg = dh u act'(g), du = dh act(g),
 *                        dx = Q(dg) Wgate + Q(du) Wup
 * The forward writes g and u in bf16 [m][n] where the pointers are given (both
 * or neither); h comes from the unrounded sums.  The backward reads them, writes
 * dx [m][k] and, where given, dg and du in bf16 [m][n] (what adapters on the two
 * projections train on); Q takes the unrounded dg and du.
 * Results are fp32 or bf16 (round to nearest even of the fp32 result).  Products
 * of codes are exact.  Results in fp32 sum them in fp32: at most (128 + T) 2^-23
 * of the sum of the products' magnitudes, T the number of 128-value blocks along
 * the contraction.  Results in bf16 are summed by gfx950's 8-bit matrix
 * instructions, which in each group of eight consecutive products along the
 * contraction (blocks start at multiples of 128) drop what lies below 2^-13 of
 * the largest of their codes' powers of two multiplied, where a subnormal code
 * counts as 2^-6 (opposite a large code it can cost the others their low bits)
 * and a product with a zero does not count; between groups sums are fp32.
 * Against the exact sum that is about 2^-17 of the sum of the products'
 * magnitudes, and at most 7 * 2^-13 of the sum over the groups of their largest,
 * counted so, beside what fp32 sums lose.
 * A row of x or dy that holds inf or NaN (of dh, g and u: whose dg or du does)
 * gives a row of NaN and touches no other row.  m < 2^31, and every launch has
 * fewer than 2^32 threads (SQ_E_SHAPE; *_workspace_bytes is 0 for what is
 * refused).  `workspace`: caller-owned device scratch of at least
 * *_workspace_bytes(m, p) bytes, which are enough for either type of the result,
 * not read before they are written; m == 0 is a no-op. */
typedef enum { SQ_ACT_SILU = 0, SQ_ACT_GELU = 1, SQ_ACT_GELU_TANH = 2 } sq_act_t;
size_t sq_linear_fwd_f8_workspace_bytes(int64_t m, const sq_f8_t *p);
sq_status_t sq_linear_fwd_f8(const uint16_t *x, int64_t m, const sq_f8_t *p, void *y,
                             sq_dtype_t y_dtype, void *workspace, size_t workspace_bytes,
                             void *stream);
size_t sq_linear_dgrad_f8_workspace_bytes(int64_t m, const sq_f8_t *p);
sq_status_t sq_linear_dgrad_f8(const uint16_t *dy, int64_t m, const sq_f8_t *p, void *dx,
                               sq_dtype_t dx_dtype, void *workspace, size_t workspace_bytes,
                               void *stream);
size_t sq_gated_fwd_f8_workspace_bytes(int64_t m, const sq_f8_t *gate);
sq_status_t sq_gated_fwd_f8(const uint16_t *x, int64_t m, const sq_f8_t *gate, const sq_f8_t *up,
                            sq_act_t act, void *h, sq_dtype_t h_dtype, uint16_t *g, uint16_t *u,
                            void *workspace, size_t workspace_bytes, void *stream);
size_t sq_gated_bwd_f8_workspace_bytes(int64_t m, const sq_f8_t *gate);
sq_status_t sq_gated_bwd_f8(const uint16_t *dh, const uint16_t *g, const uint16_t *u, int64_t m,
                            const sq_f8_t *gate, const sq_f8_t *up, sq_act_t act, void *dx,
                            sq_dtype_t dx_dtype, uint16_t *dg, uint16_t *du, void *workspace,
                            size_t workspace_bytes, void *stream);

/* The four calls above over several experts: `groups` payloads of one shape
 * stacked (codes [groups][n][kp], exps [groups][ceil(n/128)][kp/128]; n and k are
 * one expert's), rows sorted by expert, offsets as for sq_grouped_fwd_w8a8: a
 * device array of groups + 1 nondecreasing int32, read when the kernels run and
 * clamped into [0, m] there; rows before offsets[0] and from offsets[groups] on
 * are left as they were in every output.  groups >= 1 and ceil(m / 16) * groups
 * < 2^31. */
size_t sq_grouped_fwd_f8_workspace_bytes(int64_t m, int32_t groups, const sq_f8_t *p);
sq_status_t sq_grouped_fwd_f8(const uint16_t *x, int64_t m, const int32_t *offsets, int32_t groups,
                              const sq_f8_t *p, void *y, sq_dtype_t y_dtype, void *workspace,
                              size_t workspace_bytes, void *stream);
size_t sq_grouped_dgrad_f8_workspace_bytes(int64_t m, int32_t groups, const sq_f8_t *p);
sq_status_t sq_grouped_dgrad_f8(const uint16_t *dy, int64_t m, const int32_t *offsets,
                                int32_t groups, const sq_f8_t *p, void *dx, sq_dtype_t dx_dtype,
                                void *workspace, size_t workspace_bytes, void *stream);
size_t sq_grouped_gated_fwd_f8_workspace_bytes(int64_t m, int32_t groups, const sq_f8_t *gate);
sq_status_t sq_grouped_gated_fwd_f8(const uint16_t *x, int64_t m, const int32_t *offsets,
                                    int32_t groups, const sq_f8_t *gate, const sq_f8_t *up,
                                    sq_act_t act, void *h, sq_dtype_t h_dtype, uint16_t *g,
                                    uint16_t *u, void *workspace, size_t workspace_bytes,
                                    void *stream);
size_t sq_grouped_gated_bwd_f8_workspace_bytes(int64_t m, int32_t groups, const sq_f8_t *gate);
sq_status_t sq_grouped_gated_bwd_f8(const uint16_t *dh, const uint16_t *g, const uint16_t *u,
                                    int64_t m, const int32_t *offsets, int32_t groups,
                                    const sq_f8_t *gate, const sq_f8_t *up, sq_act_t act, void *dx,
                                    sq_dtype_t dx_dtype, uint16_t *dg, uint16_t *du,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* Static description of a status code; never NULL. */
const char *sq_status_str(sq_status_t status);
int sq_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SQ_H */
