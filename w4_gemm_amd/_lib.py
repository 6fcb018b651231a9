"""ctypes binding of libsq (include/sq.h).  Argument marshalling only.

The library must have been built (``python -m w4_gemm_amd.build``); there is
no fallback of any kind when it is missing.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsq.so")

SQ_OK = 0
SQ_F32, SQ_BF16 = 0, 1
SQ_FLAG_NONFINITE, SQ_FLAG_SCALE_OVERFLOW, SQ_FLAG_FP16_RANGE = 1, 2, 4
STATUS_NAMES = {0: "SQ_OK", 1: "SQ_E_NULL", 2: "SQ_E_SHAPE", 3: "SQ_E_GROUP", 4: "SQ_E_RANK",
                5: "SQ_E_ALIGN", 6: "SQ_E_WORKSPACE", 7: "SQ_E_DTYPE", 8: "SQ_E_ARCH",
                9: "SQ_E_HIP", 10: "SQ_E_ACT"}
SQ_ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
SQ_F8_MAX = 1 << 20

# every symbol include/sq.h declares
EXPORTS = ("sq_quantize_weight", "sq_linear_fwd_workspace_bytes", "sq_linear_fwd",
           "sq_linear_fwd_rotate", "sq_linear_fwd_contract", "sq_reconstruct_bf16",
           "sq_linear_dgrad_workspace_bytes", "sq_linear_dgrad", "sq_status_str",
           "sq_abi_version", "sq_quantize_weight_w8_workspace_bytes", "sq_quantize_weight_w8",
           "sq_reconstruct_bf16_w8", "sq_linear_fwd_w8_workspace_bytes", "sq_linear_fwd_w8",
           "sq_quantize_weight_mx4", "sq_quantize_act_mx4", "sq_reconstruct_bf16_mx4",
           "sq_linear_fwd_mx4_workspace_bytes", "sq_linear_fwd_mx4", "sq_linear_fwd_static",
           "sq_linear_fwd_w8a8_workspace_bytes", "sq_linear_fwd_w8a8",
           "sq_linear_dgrad_w8_workspace_bytes", "sq_linear_dgrad_w8",
           "sq_grouped_fwd_w8a8_workspace_bytes", "sq_grouped_fwd_w8a8",
           "sq_grouped_dgrad_w8_workspace_bytes", "sq_grouped_dgrad_w8",
           "sq_quantize_weight_f8", "sq_linear_fwd_f8_workspace_bytes", "sq_linear_fwd_f8",
           "sq_linear_dgrad_f8_workspace_bytes", "sq_linear_dgrad_f8",
           "sq_gated_fwd_f8_workspace_bytes", "sq_gated_fwd_f8",
           "sq_gated_bwd_f8_workspace_bytes", "sq_gated_bwd_f8",
           "sq_grouped_fwd_f8_workspace_bytes", "sq_grouped_fwd_f8",
           "sq_grouped_dgrad_f8_workspace_bytes", "sq_grouped_dgrad_f8",
           "sq_grouped_gated_fwd_f8_workspace_bytes", "sq_grouped_gated_fwd_f8",
           "sq_grouped_gated_bwd_f8_workspace_bytes", "sq_grouped_gated_bwd_f8")
SQ_FWD_STATIC_SCRATCH_BYTES = 64 << 20


class SqW4(ctypes.Structure):
    """Mirror of sq_w4_t."""
    _fields_ = [
        ("n", ctypes.c_int64),
        ("k", ctypes.c_int64),
        ("group", ctypes.c_int32),
        ("rank", ctypes.c_int32),
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("lora_up", ctypes.c_void_p),
        ("lora_down", ctypes.c_void_p),
    ]


class SqW8(ctypes.Structure):
    """Mirror of sq_w8_t (int8-residual mode)."""
    _fields_ = [
        ("n", ctypes.c_int64),
        ("k", ctypes.c_int64),
        ("rank", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("lora_up", ctypes.c_void_p),
        ("lora_down", ctypes.c_void_p),
    ]


class SqMx4(ctypes.Structure):
    """Mirror of sq_mx4_t (MXFP4 mode)."""
    _fields_ = [
        ("n", ctypes.c_int64),
        ("k", ctypes.c_int64),
        ("rank", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("codes", ctypes.c_void_p),
        ("exps", ctypes.c_void_p),
        ("lora_up", ctypes.c_void_p),
        ("lora_down", ctypes.c_void_p),
    ]


class SqF8(ctypes.Structure):
    """Mirror of sq_f8_t (8-bit float mode)."""
    _fields_ = [
        ("n", ctypes.c_int64),
        ("k", ctypes.c_int64),
        ("codes", ctypes.c_void_p),
        ("exps", ctypes.c_void_p),
    ]


class SqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({status_str(status)})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libsq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m w4_gemm_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        L.sq_quantize_weight.argtypes = [vp, ctypes.POINTER(SqW4), vp, vp, vp]
        L.sq_quantize_weight.restype = ctypes.c_int
        L.sq_linear_fwd_workspace_bytes.argtypes = [i64, ctypes.POINTER(SqW4)]
        L.sq_linear_fwd_workspace_bytes.restype = ctypes.c_size_t
        L.sq_linear_fwd.argtypes = [vp, i64, ctypes.POINTER(SqW4), vp, ctypes.c_int, vp,
                                    ctypes.c_size_t, vp]
        L.sq_linear_fwd.restype = ctypes.c_int
        L.sq_linear_fwd_rotate.argtypes = [vp, i64, ctypes.POINTER(SqW4), vp, ctypes.c_size_t, vp]
        L.sq_linear_fwd_rotate.restype = ctypes.c_int
        L.sq_linear_fwd_contract.argtypes = [i64, ctypes.POINTER(SqW4), vp, ctypes.c_int, vp,
                                             ctypes.c_size_t, vp]
        L.sq_linear_fwd_contract.restype = ctypes.c_int
        L.sq_linear_dgrad_workspace_bytes.argtypes = [i64, ctypes.POINTER(SqW4)]
        L.sq_linear_dgrad_workspace_bytes.restype = ctypes.c_size_t
        L.sq_linear_dgrad.argtypes = [vp, i64, ctypes.POINTER(SqW4), vp, ctypes.c_int, vp,
                                      ctypes.c_size_t, vp]
        L.sq_linear_dgrad.restype = ctypes.c_int
        L.sq_linear_fwd_static.argtypes = [vp, i64, ctypes.POINTER(SqW4), vp, ctypes.c_int, vp]
        L.sq_linear_fwd_static.restype = ctypes.c_int
        L.sq_reconstruct_bf16.argtypes = [ctypes.POINTER(SqW4), vp, vp]
        L.sq_reconstruct_bf16.restype = ctypes.c_int
        P8 = ctypes.POINTER(SqW8)
        L.sq_quantize_weight_w8_workspace_bytes.argtypes = [P8]
        L.sq_quantize_weight_w8_workspace_bytes.restype = ctypes.c_size_t
        L.sq_quantize_weight_w8.argtypes = [vp, P8, vp, vp, vp, ctypes.c_size_t, vp]
        L.sq_quantize_weight_w8.restype = ctypes.c_int
        L.sq_reconstruct_bf16_w8.argtypes = [P8, vp, vp]
        L.sq_reconstruct_bf16_w8.restype = ctypes.c_int
        L.sq_linear_fwd_w8_workspace_bytes.argtypes = [i64, P8]
        L.sq_linear_fwd_w8_workspace_bytes.restype = ctypes.c_size_t
        L.sq_linear_fwd_w8.argtypes = [vp, i64, P8, vp, ctypes.c_int, vp, ctypes.c_size_t, vp]
        L.sq_linear_fwd_w8.restype = ctypes.c_int
        for name in ("sq_linear_fwd_w8a8", "sq_linear_dgrad_w8"):
            f = getattr(L, name)
            f.argtypes = [vp, i64, P8, vp, ctypes.c_int, vp, ctypes.c_size_t, vp]
            f.restype = ctypes.c_int
            f = getattr(L, name + "_workspace_bytes")
            f.argtypes = [i64, P8]
            f.restype = ctypes.c_size_t
        for name in ("sq_grouped_fwd_w8a8", "sq_grouped_dgrad_w8"):
            f = getattr(L, name)
            f.argtypes = [vp, i64, vp, i32, P8, vp, ctypes.c_int, vp, ctypes.c_size_t, vp]
            f.restype = ctypes.c_int
            f = getattr(L, name + "_workspace_bytes")
            f.argtypes = [i64, i32, P8]
            f.restype = ctypes.c_size_t
        L.sqi_i8_form.argtypes = [i64, i32, P8, i32, ctypes.POINTER(i32)]
        L.sqi_i8_form.restype = ctypes.c_int
        PX = ctypes.POINTER(SqMx4)
        L.sq_quantize_weight_mx4.argtypes = [vp, PX, vp, vp]
        L.sq_quantize_weight_mx4.restype = ctypes.c_int
        L.sq_quantize_act_mx4.argtypes = [vp, i64, i64, vp, vp, vp]
        L.sq_quantize_act_mx4.restype = ctypes.c_int
        L.sq_reconstruct_bf16_mx4.argtypes = [PX, vp, vp]
        L.sq_reconstruct_bf16_mx4.restype = ctypes.c_int
        L.sq_linear_fwd_mx4_workspace_bytes.argtypes = [i64, PX]
        L.sq_linear_fwd_mx4_workspace_bytes.restype = ctypes.c_size_t
        L.sq_linear_fwd_mx4.argtypes = [vp, i64, PX, vp, ctypes.c_int, vp, ctypes.c_size_t, vp]
        L.sq_linear_fwd_mx4.restype = ctypes.c_int
        PF, ci, sz = ctypes.POINTER(SqF8), ctypes.c_int, ctypes.c_size_t
        L.sqi_f8_form.argtypes = [i32, i64, i32, PF, ci, ctypes.POINTER(i32)]
        L.sqi_f8_form.restype = ci
        L.sq_quantize_weight_f8.argtypes = [vp, ci, PF, vp, vp]
        L.sq_quantize_weight_f8.restype = ci
        for grouped, offs in (("", []), ("grouped_", [vp, i32])):
            plain = grouped or "linear_"
            for name, args in ((f"sq_{plain}fwd_f8", [vp, i64, *offs, PF, vp, ci]),
                               (f"sq_{plain}dgrad_f8", [vp, i64, *offs, PF, vp, ci]),
                               (f"sq_{grouped}gated_fwd_f8", [vp, i64, *offs, PF, PF, ci, vp, ci, vp, vp]),
                               (f"sq_{grouped}gated_bwd_f8",
                                [vp, vp, vp, i64, *offs, PF, PF, ci, vp, ci, vp, vp])):
                f = getattr(L, name)
                f.argtypes = [*args, vp, sz, vp]
                f.restype = ci
                f = getattr(L, name + "_workspace_bytes")
                f.argtypes = [i64, *offs[1:], PF]
                f.restype = sz
        L.sq_status_str.argtypes = [ctypes.c_int]
        L.sq_status_str.restype = ctypes.c_char_p
        L.sq_abi_version.argtypes = []
        L.sq_abi_version.restype = ctypes.c_int
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().sq_status_str(status).decode()


def abi_version() -> int:
    return lib().sq_abi_version()


def sq_quantize_weight(w, p: SqW4, fidx, dev_flags, stream) -> int:
    return lib().sq_quantize_weight(w, ctypes.byref(p), fidx, dev_flags, stream)


def sq_linear_fwd_workspace_bytes(m: int, p: SqW4) -> int:
    return lib().sq_linear_fwd_workspace_bytes(m, ctypes.byref(p))


def sq_linear_fwd(x, m: int, p: SqW4, y, y_dtype: int, workspace, workspace_bytes: int,
                  stream) -> int:
    return lib().sq_linear_fwd(x, m, ctypes.byref(p), y, y_dtype, workspace, workspace_bytes,
                               stream)


def sq_linear_fwd_rotate(x, m: int, p: SqW4, workspace, workspace_bytes: int, stream) -> int:
    return lib().sq_linear_fwd_rotate(x, m, ctypes.byref(p), workspace, workspace_bytes, stream)


def sq_linear_fwd_contract(m: int, p: SqW4, y, y_dtype: int, workspace, workspace_bytes: int,
                           stream) -> int:
    return lib().sq_linear_fwd_contract(m, ctypes.byref(p), y, y_dtype, workspace,
                                        workspace_bytes, stream)


def sq_linear_fwd_static(x, m: int, p: SqW4, y, y_dtype: int, stream) -> int:
    return lib().sq_linear_fwd_static(x, m, ctypes.byref(p), y, y_dtype, stream)


def sq_reconstruct_bf16(p: SqW4, w_hat, stream) -> int:
    return lib().sq_reconstruct_bf16(ctypes.byref(p), w_hat, stream)


def sq_linear_dgrad_workspace_bytes(m: int, p: SqW4) -> int:
    return lib().sq_linear_dgrad_workspace_bytes(m, ctypes.byref(p))


def sq_linear_dgrad(dy, m: int, p: SqW4, dx, dx_dtype: int, workspace, workspace_bytes: int,
                    stream) -> int:
    return lib().sq_linear_dgrad(dy, m, ctypes.byref(p), dx, dx_dtype, workspace,
                                 workspace_bytes, stream)


def sq_quantize_weight_w8_workspace_bytes(p: SqW8) -> int:
    return lib().sq_quantize_weight_w8_workspace_bytes(ctypes.byref(p))


def sq_quantize_weight_w8(w, p: SqW8, fidx, dev_flags, workspace, workspace_bytes: int,
                          stream) -> int:
    return lib().sq_quantize_weight_w8(w, ctypes.byref(p), fidx, dev_flags, workspace,
                                       workspace_bytes, stream)


def sq_reconstruct_bf16_w8(p: SqW8, w_hat, stream) -> int:
    return lib().sq_reconstruct_bf16_w8(ctypes.byref(p), w_hat, stream)


def sq_linear_fwd_w8_workspace_bytes(m: int, p: SqW8) -> int:
    return lib().sq_linear_fwd_w8_workspace_bytes(m, ctypes.byref(p))


def sq_linear_fwd_w8(x, m: int, p: SqW8, y, y_dtype: int, workspace, workspace_bytes: int,
                     stream) -> int:
    return lib().sq_linear_fwd_w8(x, m, ctypes.byref(p), y, y_dtype, workspace, workspace_bytes,
                                  stream)


def sq_linear_fwd_w8a8_workspace_bytes(m: int, p: SqW8) -> int:
    return (_lib or lib()).sq_linear_fwd_w8a8_workspace_bytes(m, p)


def sq_linear_fwd_w8a8(x, m: int, p: SqW8, y, y_dtype: int, workspace, workspace_bytes: int,
                       stream) -> int:
    return (_lib or lib()).sq_linear_fwd_w8a8(x, m, p, y, y_dtype, workspace, workspace_bytes,
                                              stream)


def sq_linear_dgrad_w8_workspace_bytes(m: int, p: SqW8) -> int:
    return (_lib or lib()).sq_linear_dgrad_w8_workspace_bytes(m, p)


def sq_linear_dgrad_w8(dy, m: int, p: SqW8, dx, dx_dtype: int, workspace, workspace_bytes: int,
                       stream) -> int:
    return (_lib or lib()).sq_linear_dgrad_w8(dy, m, p, dx, dx_dtype, workspace, workspace_bytes,
                                              stream)


def sq_grouped_fwd_w8a8_workspace_bytes(m: int, groups: int, p: SqW8) -> int:
    return (_lib or lib()).sq_grouped_fwd_w8a8_workspace_bytes(m, groups, p)


def sq_grouped_fwd_w8a8(x, m: int, offsets, groups: int, p: SqW8, y, y_dtype: int, workspace,
                        workspace_bytes: int, stream) -> int:
    return (_lib or lib()).sq_grouped_fwd_w8a8(x, m, offsets, groups, p, y, y_dtype, workspace,
                                               workspace_bytes, stream)


def sq_grouped_dgrad_w8_workspace_bytes(m: int, groups: int, p: SqW8) -> int:
    return (_lib or lib()).sq_grouped_dgrad_w8_workspace_bytes(m, groups, p)


def sq_grouped_dgrad_w8(dy, m: int, offsets, groups: int, p: SqW8, dx, dx_dtype: int, workspace,
                        workspace_bytes: int, stream) -> int:
    return (_lib or lib()).sq_grouped_dgrad_w8(dy, m, offsets, groups, p, dx, dx_dtype,
                                               workspace, workspace_bytes, stream)


def i8_form(m: int, n: int, k: int, groups: int = 1, rank: int = 0, dgrad: bool = False) -> tuple:
    """Form of the kernels that an 8-bit product of these sizes takes: tile rows, tile columns, K
    splits (input gradient: parts of a tail tile at most), projection tile rows, projection slices."""
    form = (ctypes.c_int32 * 5)()
    p = SqW8(n, k, rank, 0, None, None, None, None)
    status = lib().sqi_i8_form(m, groups, p, dgrad, form)
    if status != SQ_OK:
        raise ValueError(status_str(status))
    return tuple(form)


def sq_quantize_weight_mx4(w, p: SqMx4, dev_flags, stream) -> int:
    return lib().sq_quantize_weight_mx4(w, ctypes.byref(p), dev_flags, stream)


def sq_quantize_act_mx4(x, m: int, k: int, xq, xs, stream) -> int:
    return lib().sq_quantize_act_mx4(x, m, k, xq, xs, stream)


def sq_reconstruct_bf16_mx4(p: SqMx4, w_hat, stream) -> int:
    return lib().sq_reconstruct_bf16_mx4(ctypes.byref(p), w_hat, stream)


def sq_linear_fwd_mx4_workspace_bytes(m: int, p: SqMx4) -> int:
    return lib().sq_linear_fwd_mx4_workspace_bytes(m, ctypes.byref(p))


def sq_linear_fwd_mx4(x, m: int, p: SqMx4, y, y_dtype: int, workspace, workspace_bytes: int,
                      stream) -> int:
    return lib().sq_linear_fwd_mx4(x, m, ctypes.byref(p), y, y_dtype, workspace, workspace_bytes,
                                   stream)


def sq_quantize_weight_f8(w, w_dtype: int, p: SqF8, dev_flags, stream) -> int:
    return lib().sq_quantize_weight_f8(w, w_dtype, p, dev_flags, stream)


def sq_linear_fwd_f8_workspace_bytes(m: int, p: SqF8) -> int:
    return (_lib or lib()).sq_linear_fwd_f8_workspace_bytes(m, p)


def sq_linear_fwd_f8(x, m: int, p: SqF8, y, y_dtype: int, workspace, workspace_bytes: int,
                     stream) -> int:
    return (_lib or lib()).sq_linear_fwd_f8(x, m, p, y, y_dtype, workspace, workspace_bytes, stream)


def sq_linear_dgrad_f8_workspace_bytes(m: int, p: SqF8) -> int:
    return (_lib or lib()).sq_linear_dgrad_f8_workspace_bytes(m, p)


def sq_linear_dgrad_f8(dy, m: int, p: SqF8, dx, dx_dtype: int, workspace, workspace_bytes: int,
                       stream) -> int:
    return (_lib or lib()).sq_linear_dgrad_f8(dy, m, p, dx, dx_dtype, workspace, workspace_bytes,
                                              stream)


def sq_grouped_fwd_f8_workspace_bytes(m: int, groups: int, p: SqF8) -> int:
    return (_lib or lib()).sq_grouped_fwd_f8_workspace_bytes(m, groups, p)


def sq_grouped_fwd_f8(x, m: int, offsets, groups: int, p: SqF8, y, y_dtype: int, workspace,
                      workspace_bytes: int, stream) -> int:
    return (_lib or lib()).sq_grouped_fwd_f8(x, m, offsets, groups, p, y, y_dtype, workspace,
                                             workspace_bytes, stream)


def sq_grouped_dgrad_f8_workspace_bytes(m: int, groups: int, p: SqF8) -> int:
    return (_lib or lib()).sq_grouped_dgrad_f8_workspace_bytes(m, groups, p)


def sq_grouped_dgrad_f8(dy, m: int, offsets, groups: int, p: SqF8, dx, dx_dtype: int, workspace,
                        workspace_bytes: int, stream) -> int:
    return (_lib or lib()).sq_grouped_dgrad_f8(dy, m, offsets, groups, p, dx, dx_dtype, workspace,
                                               workspace_bytes, stream)


def sq_gated_fwd_f8_workspace_bytes(m: int, gate: SqF8) -> int:
    return (_lib or lib()).sq_gated_fwd_f8_workspace_bytes(m, gate)


def sq_gated_fwd_f8(x, m: int, gate: SqF8, up: SqF8, act: int, h, h_dtype: int, g, u, workspace,
                    workspace_bytes: int, stream) -> int:
    return (_lib or lib()).sq_gated_fwd_f8(x, m, gate, up, act, h, h_dtype, g, u, workspace,
                                           workspace_bytes, stream)


def sq_gated_bwd_f8_workspace_bytes(m: int, gate: SqF8) -> int:
    return (_lib or lib()).sq_gated_bwd_f8_workspace_bytes(m, gate)


def sq_gated_bwd_f8(dh, g, u, m: int, gate: SqF8, up: SqF8, act: int, dx, dx_dtype: int, dg, du,
                    workspace, workspace_bytes: int, stream) -> int:
    return (_lib or lib()).sq_gated_bwd_f8(dh, g, u, m, gate, up, act, dx, dx_dtype, dg, du,
                                           workspace, workspace_bytes, stream)


def sq_grouped_gated_fwd_f8_workspace_bytes(m: int, groups: int, gate: SqF8) -> int:
    return (_lib or lib()).sq_grouped_gated_fwd_f8_workspace_bytes(m, groups, gate)


def sq_grouped_gated_fwd_f8(x, m: int, offsets, groups: int, gate: SqF8, up: SqF8, act: int, h,
                            h_dtype: int, g, u, workspace, workspace_bytes: int, stream) -> int:
    return (_lib or lib()).sq_grouped_gated_fwd_f8(x, m, offsets, groups, gate, up, act, h, h_dtype,
                                                   g, u, workspace, workspace_bytes, stream)


def sq_grouped_gated_bwd_f8_workspace_bytes(m: int, groups: int, gate: SqF8) -> int:
    return (_lib or lib()).sq_grouped_gated_bwd_f8_workspace_bytes(m, groups, gate)


def sq_grouped_gated_bwd_f8(dh, g, u, m: int, offsets, groups: int, gate: SqF8, up: SqF8, act: int,
                            dx, dx_dtype: int, dg, du, workspace, workspace_bytes: int,
                            stream) -> int:
    return (_lib or lib()).sq_grouped_gated_bwd_f8(dh, g, u, m, offsets, groups, gate, up, act, dx,
                                                   dx_dtype, dg, du, workspace, workspace_bytes,
                                                   stream)


F8_KINDS = {"fwd": 0, "dgrad": 1, "gated_fwd": 2, "gated_bwd": 3}


def f8_form(kind: str, m: int, n: int, k: int, groups: int = 1, bf16: bool = True) -> tuple:
    """Form of the kernels that an 8-bit float product of these sizes takes: tile rows (16: the form
    that streams the codes), tile columns, waves of that form's workgroups, splits."""
    form = (ctypes.c_int32 * 4)()
    status = lib().sqi_f8_form(F8_KINDS[kind], m, groups, SqF8(n, k, None, None),
                               SQ_BF16 if bf16 else SQ_F32, form)
    if status != SQ_OK:
        raise ValueError(status_str(status))
    return tuple(form)
