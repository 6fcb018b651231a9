// C ABI of libsq: argument validation, device check and kernel launches.
// Every entry point validates synchronously and launches nothing on error;
// work is enqueued on the caller's stream and never synchronized here.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "../../include/sq.h"
#include "sq_kernels.h"

namespace {

constexpr int kMaxDevices = 64;
int g_arch_ok[kMaxDevices];   // 0 unknown, 1 gfx950, -1 other
std::mutex g_arch_mu;

sq_status_t check_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return SQ_E_HIP;
  std::lock_guard<std::mutex> lock(g_arch_mu);
  if (g_arch_ok[dev] == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return SQ_E_HIP;
    g_arch_ok[dev] = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
  }
  return g_arch_ok[dev] == 1 ? SQ_OK : SQ_E_ARCH;
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

sq_status_t check_payload(const sq_w4_t* p, bool need_codes) {
  if (!p) return SQ_E_NULL;
  if (p->k < 256 || p->k % 256 != 0 || p->n < 1) return SQ_E_SHAPE;
  if (p->group != 32 && p->group != 64) return SQ_E_GROUP;
  if (p->rank != 0 && p->rank != 32 && p->rank != 64) return SQ_E_RANK;
  if (!p->codes || !p->scales) return SQ_E_NULL;
  if (p->rank > 0 && (!p->lora_up || !p->lora_down)) return SQ_E_NULL;
  if (!aligned16(p->codes) || !aligned16(p->scales)) return SQ_E_ALIGN;
  if (p->rank > 0 && (!aligned16(p->lora_up) || !aligned16(p->lora_down))) return SQ_E_ALIGN;
  (void)need_codes;
  return SQ_OK;
}

sq_status_t check_payload_w8(const sq_w8_t* p) {
  if (!p) return SQ_E_NULL;
  if (p->k < 256 || p->k % 256 != 0 || p->n < 1) return SQ_E_SHAPE;
  if ((p->rank != 0 && p->rank != 16 && p->rank != 32 && p->rank != 64) || p->reserved != 0)
    return SQ_E_RANK;
  if (!p->codes || !p->scales) return SQ_E_NULL;
  if (p->rank > 0 && (!p->lora_up || !p->lora_down)) return SQ_E_NULL;
  if (!aligned16(p->codes) || !aligned16(p->scales)) return SQ_E_ALIGN;
  if (p->rank > 0 && (!aligned16(p->lora_up) || !aligned16(p->lora_down))) return SQ_E_ALIGN;
  return SQ_OK;
}

sq_status_t check_payload_mx(const sq_mx4_t* p) {
  if (!p) return SQ_E_NULL;
  if (p->k < 256 || p->k % 256 != 0 || p->n < 1) return SQ_E_SHAPE;
  if ((p->rank != 0 && p->rank != 16 && p->rank != 32 && p->rank != 64) || p->reserved != 0)
    return SQ_E_RANK;
  if (!p->codes || !p->exps) return SQ_E_NULL;
  if (p->rank > 0 && (!p->lora_up || !p->lora_down)) return SQ_E_NULL;
  if (!aligned16(p->codes) || !aligned16(p->exps)) return SQ_E_ALIGN;
  if (p->rank > 0 && (!aligned16(p->lora_up) || !aligned16(p->lora_down))) return SQ_E_ALIGN;
  return SQ_OK;
}

sq_status_t from_hip(hipError_t e) { return e == hipSuccess ? SQ_OK : SQ_E_HIP; }

// Scratch of the allocation-free forward: one copy per device, part of the
// code object's zero-initialised data, held until the process ends.  In host
// code its name is a host-side stand-in; the device address comes from
// hipGetSymbolAddress, once per device, and only that address is used.
static __device__ __align__(256) uint8_t scratch[SQ_FWD_STATIC_SCRATCH_BYTES];
void* g_scratch_ptr[kMaxDevices];
std::mutex g_scratch_mu;

sq_status_t scratch_address(void** out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return SQ_E_HIP;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* ptr = nullptr;
    if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess || !ptr) return SQ_E_HIP;
    g_scratch_ptr[dev] = ptr;
  }
  *out = g_scratch_ptr[dev];
  return SQ_OK;
}

}  // namespace

extern "C" {

int sq_abi_version(void) { return SQ_ABI_VERSION; }

const char* sq_status_str(sq_status_t s) {
  switch (s) {
    case SQ_OK: return "ok";
    case SQ_E_NULL: return "a required pointer is NULL";
    case SQ_E_SHAPE:
      return "bad shape: need K % 256 == 0, K >= 256, N >= 1, M >= 0 (W4 input gradient: N % 64 == 0; "
             "8-bit products: K <= 65536, M < 2^31, groups >= 1, their input gradient N <= 131072, "
             "M <= 2^25 (2^23 for N > 2048))";
    case SQ_E_GROUP: return "group must be 32 or 64";
    case SQ_E_RANK: return "rank must be 0, 32 or 64 (int8 mode: 0, 16, 32 or 64; reserved 0)";
    case SQ_E_ALIGN: return "every pointer must be 16-byte aligned";
    case SQ_E_WORKSPACE: return "workspace smaller than the entry point's *_workspace_bytes()";
    case SQ_E_DTYPE: return "output dtype must be SQ_F32 or SQ_BF16";
    case SQ_E_ARCH: return "the current device is not gfx950 (MI355X)";
    case SQ_E_HIP: return "a HIP runtime call or kernel launch failed";
  }
  return "unknown status";
}

sq_status_t sq_quantize_weight(const float* w, const sq_w4_t* p, uint8_t* fidx,
                               int32_t* dev_flags, void* stream) {
  sq_status_t st = check_payload(p, true);
  if (st != SQ_OK) return st;
  if (!w || !dev_flags) return SQ_E_NULL;
  if (!aligned16(w) || (fidx && !aligned16(fidx)) || !aligned16(dev_flags)) return SQ_E_ALIGN;
  if ((st = check_device()) != SQ_OK) return st;
  return from_hip(sq::launch_quantize(w, p->lora_up, p->lora_down, p->codes, p->scales, fidx,
                                      dev_flags, p->n, p->k, p->group, p->rank,
                                      static_cast<hipStream_t>(stream)));
}

static sq::FwdPlan make_fwd_plan(int64_t m, const sq_w4_t* p) {
  if (sq::decode_eligible(m, p->n, p->k, p->rank))
    return sq::plan_decode(m, p->n, p->k, p->group, p->rank);
  return sq::plan_fwd(m, p->n, p->k, p->group, p->rank);
}

size_t sq_linear_fwd_workspace_bytes(int64_t m, const sq_w4_t* p) {
  if (!p || m <= 0 || p->k < 256 || p->k % 256 || p->n < 1) return 0;
  return make_fwd_plan(m, p).total;
}

static sq_status_t check_fwd(int64_t m, const sq_w4_t* p, void* workspace, size_t ws_bytes,
                             sq::FwdPlan* plan) {
  sq_status_t st = check_payload(p, true);
  if (st != SQ_OK) return st;
  if (m < 0) return SQ_E_SHAPE;
  if (m == 0) return SQ_OK;
  if (!workspace) return SQ_E_NULL;
  if (!aligned16(workspace)) return SQ_E_ALIGN;
  *plan = make_fwd_plan(m, p);
  if (ws_bytes < plan->total) return SQ_E_WORKSPACE;
  return SQ_OK;
}

sq_status_t sq_linear_fwd_rotate(const uint16_t* x, int64_t m, const sq_w4_t* p, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  sq::FwdPlan plan{};
  sq_status_t st = check_fwd(m, p, workspace, workspace_bytes, &plan);
  if (st != SQ_OK || m == 0) return st;
  if (!x) return SQ_E_NULL;
  if (!aligned16(x)) return SQ_E_ALIGN;
  if ((st = check_device()) != SQ_OK) return st;
  if (plan.dec)
    return from_hip(sq::launch_decode_prep(plan, x, p->lora_down, workspace,
                                           static_cast<hipStream_t>(stream)));
  return from_hip(sq::launch_fwd_rotate(plan, x, p->lora_down, workspace,
                                        static_cast<hipStream_t>(stream)));
}

sq_status_t sq_linear_fwd_contract(int64_t m, const sq_w4_t* p, void* y, sq_dtype_t y_dtype,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  sq::FwdPlan plan{};
  if (y_dtype != SQ_F32 && y_dtype != SQ_BF16) return SQ_E_DTYPE;
  sq_status_t st = check_fwd(m, p, workspace, workspace_bytes, &plan);
  if (st != SQ_OK || m == 0) return st;
  if (!y) return SQ_E_NULL;
  if (!aligned16(y)) return SQ_E_ALIGN;
  if ((st = check_device()) != SQ_OK) return st;
  if (plan.dec)
    return from_hip(sq::launch_decode_contract(plan, nullptr, nullptr, p->codes, p->scales,
                                               p->lora_up, y, y_dtype == SQ_BF16, workspace,
                                               static_cast<hipStream_t>(stream)));
  return from_hip(sq::launch_fwd_contract(plan, p->codes, p->scales, p->lora_up, y,
                                          y_dtype == SQ_BF16, workspace,
                                          static_cast<hipStream_t>(stream)));
}

sq_status_t sq_linear_fwd(const uint16_t* x, int64_t m, const sq_w4_t* p, void* y,
                          sq_dtype_t y_dtype, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (y_dtype != SQ_F32 && y_dtype != SQ_BF16) return SQ_E_DTYPE;
  sq::FwdPlan plan{};
  sq_status_t st = check_fwd(m, p, workspace, workspace_bytes, &plan);
  if (st != SQ_OK || m == 0) return st;
  if (!x || !y) return SQ_E_NULL;
  if (!aligned16(x) || !aligned16(y)) return SQ_E_ALIGN;
  if ((st = check_device()) != SQ_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (plan.dec)
    return from_hip(sq::launch_decode_contract(plan, x, p->lora_down, p->codes, p->scales,
                                               p->lora_up, y, y_dtype == SQ_BF16, workspace, s));
  if ((st = from_hip(sq::launch_fwd_rotate(plan, x, p->lora_down, workspace, s))) != SQ_OK)
    return st;
  return from_hip(sq::launch_fwd_contract(plan, p->codes, p->scales, p->lora_up, y,
                                          y_dtype == SQ_BF16, workspace, s));
}

sq_status_t sq_linear_fwd_static(const uint16_t* x, int64_t m, const sq_w4_t* p, void* y,
                                 sq_dtype_t y_dtype, void* stream) {
  if (y_dtype != SQ_F32 && y_dtype != SQ_BF16) return SQ_E_DTYPE;
  sq_status_t st = check_payload(p, true);
  if (st != SQ_OK) return st;
  if (m < 0) return SQ_E_SHAPE;
  if (m == 0) return SQ_OK;
  if (!x || !y) return SQ_E_NULL;
  if (!aligned16(x) || !aligned16(y)) return SQ_E_ALIGN;
  const sq::FwdPlan plan = make_fwd_plan(m, p);
  if (plan.total > SQ_FWD_STATIC_SCRATCH_BYTES) return SQ_E_WORKSPACE;
  if ((st = check_device()) != SQ_OK) return st;
  void* ws = nullptr;
  if ((st = scratch_address(&ws)) != SQ_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (plan.dec)
    return from_hip(sq::launch_decode_contract(plan, x, p->lora_down, p->codes, p->scales,
                                               p->lora_up, y, y_dtype == SQ_BF16, ws, s));
  if ((st = from_hip(sq::launch_fwd_rotate(plan, x, p->lora_down, ws, s))) != SQ_OK) return st;
  return from_hip(sq::launch_fwd_contract(plan, p->codes, p->scales, p->lora_up, y,
                                          y_dtype == SQ_BF16, ws, s));
}

size_t sq_linear_dgrad_workspace_bytes(int64_t m, const sq_w4_t* p) {
  if (!p || m <= 0 || p->k < 256 || p->k % 256 || p->n < 64 || p->n % 64) return 0;
  if (p->rank != 0 && p->rank != 32 && p->rank != 64) return 0;
  return sq::plan_dgrad(m, p->n, p->k, p->group, p->rank).total;
}

sq_status_t sq_linear_dgrad(const uint16_t* dy, int64_t m, const sq_w4_t* p, void* dx,
                            sq_dtype_t dx_dtype, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (dx_dtype != SQ_F32 && dx_dtype != SQ_BF16) return SQ_E_DTYPE;
  sq_status_t st = check_payload(p, true);
  if (st != SQ_OK) return st;
  if (m < 0 || p->n % 64 != 0) return SQ_E_SHAPE;
  if (m == 0) return SQ_OK;
  if (!dy || !dx || !workspace) return SQ_E_NULL;
  if (!aligned16(dy) || !aligned16(dx) || !aligned16(workspace)) return SQ_E_ALIGN;
  const sq::DgradPlan plan = sq::plan_dgrad(m, p->n, p->k, p->group, p->rank);
  if (workspace_bytes < plan.total) return SQ_E_WORKSPACE;
  if ((st = check_device()) != SQ_OK) return st;
  return from_hip(sq::launch_dgrad(plan, dy, p->codes, p->scales, p->lora_up, p->lora_down, dx,
                                   dx_dtype == SQ_BF16, workspace,
                                   static_cast<hipStream_t>(stream)));
}

sq_status_t sq_reconstruct_bf16(const sq_w4_t* p, uint16_t* w_hat, void* stream) {
  sq_status_t st = check_payload(p, true);
  if (st != SQ_OK) return st;
  if (!w_hat) return SQ_E_NULL;
  if (!aligned16(w_hat)) return SQ_E_ALIGN;
  if ((st = check_device()) != SQ_OK) return st;
  return from_hip(sq::launch_reconstruct(p->codes, p->scales, p->lora_up, p->lora_down, w_hat,
                                         p->n, p->k, p->group, p->rank,
                                         static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- int8-residual mode
size_t sq_quantize_weight_w8_workspace_bytes(const sq_w8_t* p) {
  if (!p || p->k < 256 || p->k % 256 || p->n < 1) return 0;
  return sq::quantize_w8_workspace(p->n, p->k);
}

sq_status_t sq_quantize_weight_w8(const float* w, const sq_w8_t* p, uint8_t* fidx,
                                  int32_t* dev_flags, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  sq_status_t st = check_payload_w8(p);
  if (st != SQ_OK) return st;
  if (!w || !dev_flags || !workspace) return SQ_E_NULL;
  if (!aligned16(w) || (fidx && !aligned16(fidx)) || !aligned16(dev_flags) ||
      !aligned16(workspace))
    return SQ_E_ALIGN;
  if (workspace_bytes < sq::quantize_w8_workspace(p->n, p->k)) return SQ_E_WORKSPACE;
  if ((st = check_device()) != SQ_OK) return st;
  return from_hip(sq::launch_quantize_w8(w, p->lora_up, p->lora_down, p->codes, p->scales, fidx,
                                         dev_flags, p->n, p->k, p->rank, workspace,
                                         static_cast<hipStream_t>(stream)));
}

sq_status_t sq_reconstruct_bf16_w8(const sq_w8_t* p, uint16_t* w_hat, void* stream) {
  sq_status_t st = check_payload_w8(p);
  if (st != SQ_OK) return st;
  if (!w_hat) return SQ_E_NULL;
  if (!aligned16(w_hat)) return SQ_E_ALIGN;
  if ((st = check_device()) != SQ_OK) return st;
  return from_hip(sq::launch_reconstruct(reinterpret_cast<const uint8_t*>(p->codes), p->scales,
                                         p->lora_up, p->lora_down, w_hat, p->n, p->k, 0, p->rank,
                                         static_cast<hipStream_t>(stream)));
}

// group 0 selects the int8 payload in the forward kernels
static sq::FwdPlan make_fwd_plan_w8(int64_t m, const sq_w8_t* p) {
  if (sq::decode_eligible(m, p->n, p->k, p->rank, true))
    return sq::plan_decode(m, p->n, p->k, 0, p->rank);
  return sq::plan_fwd(m, p->n, p->k, 0, p->rank);
}

size_t sq_linear_fwd_w8_workspace_bytes(int64_t m, const sq_w8_t* p) {
  if (!p || m <= 0 || p->k < 256 || p->k % 256 || p->n < 1) return 0;
  return make_fwd_plan_w8(m, p).total;
}

sq_status_t sq_linear_fwd_w8(const uint16_t* x, int64_t m, const sq_w8_t* p, void* y,
                             sq_dtype_t y_dtype, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (y_dtype != SQ_F32 && y_dtype != SQ_BF16) return SQ_E_DTYPE;
  sq_status_t st = check_payload_w8(p);
  if (st != SQ_OK) return st;
  if (m < 0) return SQ_E_SHAPE;
  if (m == 0) return SQ_OK;
  if (!x || !y || !workspace) return SQ_E_NULL;
  if (!aligned16(x) || !aligned16(y) || !aligned16(workspace)) return SQ_E_ALIGN;
  const sq::FwdPlan plan = make_fwd_plan_w8(m, p);
  if (workspace_bytes < plan.total) return SQ_E_WORKSPACE;
  if ((st = check_device()) != SQ_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (plan.dec)
    return from_hip(sq::launch_decode_contract(
        plan, x, p->lora_down, reinterpret_cast<const uint8_t*>(p->codes), p->scales, p->lora_up,
        y, y_dtype == SQ_BF16, workspace, s));
  if ((st = from_hip(sq::launch_fwd_rotate(plan, x, p->lora_down, workspace, s))) != SQ_OK)
    return st;
  return from_hip(sq::launch_fwd_contract(plan, reinterpret_cast<const uint8_t*>(p->codes),
                                          p->scales, p->lora_up, y, y_dtype == SQ_BF16, workspace,
                                          s));
}

// ---------------------------------------------------------------- 8-bit products
// Sizes that the 8-bit products take: a row of x on one workgroup (K <= 65536),
// exact int32 sums, 32-bit row numbers and a launch of fewer than 2^31 workgroups.
constexpr int64_t kI8MaxK = 65536, kI8MaxN = sq::I8_DGRAD_MAX_N;

static bool i8_shape_ok(int64_t m, int32_t groups, const sq_w8_t* p, bool dgrad) {
  if (m < 0 || m > INT32_MAX || groups < 1 || p->k > kI8MaxK || p->n > INT32_MAX) return false;
  // a gradient row takes a wave up to N = 2048 and a workgroup beyond; one launch has fewer
  // than 2^32 threads
  if (dgrad && (p->n > kI8MaxN || m > (p->n <= 2048 ? int64_t{1} << 25 : int64_t{1} << 23)))
    return false;
  // offsets that are not ordered can name up to ceil(m / 16) tiles per group,
  // which the device counts in 32 bits
  if ((m + 15) / 16 > INT32_MAX / groups) return false;
  const int64_t tiles = sq::i8_tile_bound(m, groups, 16);
  return tiles <= INT32_MAX / ((p->n + 15) / 16) && tiles <= INT32_MAX / (p->k / 16);
}

static size_t i8_workspace_bytes(int64_t m, int32_t groups, const sq_w8_t* p, bool dgrad) {
  if (!p || m <= 0 || p->k < 256 || p->k % 256 || p->n < 1) return 0;
  if (p->rank != 0 && p->rank != 16 && p->rank != 32 && p->rank != 64) return 0;
  if (!i8_shape_ok(m, groups, p, dgrad)) return 0;
  return dgrad ? sq::plan_w8_dgrad(m, p->n, p->k, groups, p->rank).total
               : sq::plan_w8a8(m, p->n, p->k, groups, p->rank).total;
}

// in is x [m][k] (forward) or dy [m][n] (input gradient); offsets is null for one layer
static sq_status_t i8_product(const uint16_t* in, int64_t m, const int32_t* offsets, bool grouped,
                              int32_t groups, const sq_w8_t* p, void* out, sq_dtype_t out_dtype,
                              void* workspace, size_t workspace_bytes, void* stream, bool dgrad) {
  if (out_dtype != SQ_F32 && out_dtype != SQ_BF16) return SQ_E_DTYPE;
  sq_status_t st = check_payload_w8(p);
  if (st != SQ_OK) return st;
  if (!i8_shape_ok(m, groups, p, dgrad)) return SQ_E_SHAPE;
  if (m == 0) return SQ_OK;
  if (!in || !out || !workspace || (grouped && !offsets)) return SQ_E_NULL;
  if (!aligned16(in) || !aligned16(out) || !aligned16(workspace) || !aligned16(offsets))
    return SQ_E_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int bf16 = out_dtype == SQ_BF16;
  if (dgrad) {
    const sq::W8DgradPlan plan = sq::plan_w8_dgrad(m, p->n, p->k, groups, p->rank);
    if (workspace_bytes < plan.total) return SQ_E_WORKSPACE;
    if ((st = check_device()) != SQ_OK) return st;
    return from_hip(sq::launch_w8_dgrad(plan, in, offsets, p->codes, p->scales, p->lora_up,
                                        p->lora_down, out, bf16, workspace, s));
  }
  const sq::W8A8Plan plan = sq::plan_w8a8(m, p->n, p->k, groups, p->rank);
  if (workspace_bytes < plan.total) return SQ_E_WORKSPACE;
  if ((st = check_device()) != SQ_OK) return st;
  return from_hip(sq::launch_w8a8(plan, in, offsets, p->codes, p->scales, p->lora_up,
                                  p->lora_down, out, bf16, workspace, s));
}

size_t sq_linear_fwd_w8a8_workspace_bytes(int64_t m, const sq_w8_t* p) {
  return i8_workspace_bytes(m, 1, p, false);
}

sq_status_t sq_linear_fwd_w8a8(const uint16_t* x, int64_t m, const sq_w8_t* p, void* y,
                               sq_dtype_t y_dtype, void* workspace, size_t workspace_bytes,
                               void* stream) {
  return i8_product(x, m, nullptr, false, 1, p, y, y_dtype, workspace, workspace_bytes, stream,
                    false);
}

size_t sq_linear_dgrad_w8_workspace_bytes(int64_t m, const sq_w8_t* p) {
  return i8_workspace_bytes(m, 1, p, true);
}

sq_status_t sq_linear_dgrad_w8(const uint16_t* dy, int64_t m, const sq_w8_t* p, void* dx,
                               sq_dtype_t dx_dtype, void* workspace, size_t workspace_bytes,
                               void* stream) {
  return i8_product(dy, m, nullptr, false, 1, p, dx, dx_dtype, workspace, workspace_bytes, stream,
                    true);
}

size_t sq_grouped_fwd_w8a8_workspace_bytes(int64_t m, int32_t groups, const sq_w8_t* p) {
  return i8_workspace_bytes(m, groups, p, false);
}

sq_status_t sq_grouped_fwd_w8a8(const uint16_t* x, int64_t m, const int32_t* offsets,
                                int32_t groups, const sq_w8_t* p, void* y, sq_dtype_t y_dtype,
                                void* workspace, size_t workspace_bytes, void* stream) {
  return i8_product(x, m, offsets, true, groups, p, y, y_dtype, workspace, workspace_bytes, stream,
                    false);
}

size_t sq_grouped_dgrad_w8_workspace_bytes(int64_t m, int32_t groups, const sq_w8_t* p) {
  return i8_workspace_bytes(m, groups, p, true);
}

sq_status_t sq_grouped_dgrad_w8(const uint16_t* dy, int64_t m, const int32_t* offsets,
                                int32_t groups, const sq_w8_t* p, void* dx, sq_dtype_t dx_dtype,
                                void* workspace, size_t workspace_bytes, void* stream) {
  return i8_product(dy, m, offsets, true, groups, p, dx, dx_dtype, workspace, workspace_bytes,
                    stream, true);
}

// Which form of the kernels a call takes, for callers that must know (the tests
// of every form); not part of the ABI.  form: rows and columns of the product's
// tile, K splits (forward) or parts of a tail tile at most (gradient), rows of a
// projection tile, projection slices.  Sizes as the entry points check them.
sq_status_t sqi_i8_form(int64_t m, int32_t groups, const sq_w8_t* p, int32_t dgrad,
                        int32_t form[5]) {
  if (!form) return SQ_E_NULL;
  if (i8_workspace_bytes(m, groups, p, dgrad != 0) == 0) return SQ_E_SHAPE;
  if (dgrad) {
    const sq::W8DgradPlan plan = sq::plan_w8_dgrad(m, p->n, p->k, groups, p->rank);
    const int32_t f[5] = {plan.tile_m, 256, plan.max_split, plan.t_rows, plan.slices};
    memcpy(form, f, sizeof f);
  } else {
    const sq::W8A8Plan plan = sq::plan_w8a8(m, p->n, p->k, groups, p->rank);
    const int32_t f[5] = {plan.tile_m, plan.tile_n, plan.splits, plan.t_rows, plan.slices};
    memcpy(form, f, sizeof f);
  }
  return SQ_OK;
}

// ---------------------------------------------------------------- MXFP4 mode
sq_status_t sq_quantize_weight_mx4(const float* w, const sq_mx4_t* p, int32_t* dev_flags,
                                   void* stream) {
  sq_status_t st = check_payload_mx(p);
  if (st != SQ_OK) return st;
  if (!w || !dev_flags) return SQ_E_NULL;
  if (!aligned16(w) || !aligned16(dev_flags)) return SQ_E_ALIGN;
  if ((st = check_device()) != SQ_OK) return st;
  return from_hip(sq::launch_quantize_mx(w, p->lora_up, p->lora_down, p->codes, p->exps, dev_flags,
                                         p->n, p->k, p->rank, static_cast<hipStream_t>(stream)));
}

sq_status_t sq_quantize_act_mx4(const uint16_t* x, int64_t m, int64_t k, uint8_t* xq, uint8_t* xs,
                                void* stream) {
  if (m < 0 || k < 256 || k % 256 != 0) return SQ_E_SHAPE;
  if (m == 0) return SQ_OK;
  if (!x || !xq || !xs) return SQ_E_NULL;
  if (!aligned16(x) || !aligned16(xq) || !aligned16(xs)) return SQ_E_ALIGN;
  sq_status_t st = check_device();
  if (st != SQ_OK) return st;
  return from_hip(sq::launch_quantize_act_mx(x, m, k, xq, xs, static_cast<hipStream_t>(stream)));
}

sq_status_t sq_reconstruct_bf16_mx4(const sq_mx4_t* p, uint16_t* w_hat, void* stream) {
  sq_status_t st = check_payload_mx(p);
  if (st != SQ_OK) return st;
  if (!w_hat) return SQ_E_NULL;
  if (!aligned16(w_hat)) return SQ_E_ALIGN;
  if ((st = check_device()) != SQ_OK) return st;
  return from_hip(sq::launch_reconstruct_mx(p->codes, p->exps, p->lora_up, p->lora_down, w_hat,
                                            p->n, p->k, p->rank,
                                            static_cast<hipStream_t>(stream)));
}

size_t sq_linear_fwd_mx4_workspace_bytes(int64_t m, const sq_mx4_t* p) {
  if (!p || m <= 0 || p->k < 256 || p->k % 256 || p->n < 1) return 0;
  return sq::plan_mx(m, p->n, p->k, p->rank).total;
}

sq_status_t sq_linear_fwd_mx4(const uint16_t* x, int64_t m, const sq_mx4_t* p, void* y,
                              sq_dtype_t y_dtype, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (y_dtype != SQ_F32 && y_dtype != SQ_BF16) return SQ_E_DTYPE;
  sq_status_t st = check_payload_mx(p);
  if (st != SQ_OK) return st;
  if (m < 0) return SQ_E_SHAPE;
  if (m == 0) return SQ_OK;
  if (!x || !y || !workspace) return SQ_E_NULL;
  if (!aligned16(x) || !aligned16(y) || !aligned16(workspace)) return SQ_E_ALIGN;
  const sq::MxPlan plan = sq::plan_mx(m, p->n, p->k, p->rank);
  if (workspace_bytes < plan.total) return SQ_E_WORKSPACE;
  if ((st = check_device()) != SQ_OK) return st;
  return from_hip(sq::launch_fwd_mx(plan, x, p->codes, p->exps, p->lora_up, p->lora_down, y,
                                    y_dtype == SQ_BF16, workspace,
                                    static_cast<hipStream_t>(stream)));
}

}  // extern "C"
