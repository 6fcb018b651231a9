"""Workspace sizes of the 8-bit float products over the row counts that share one buffer."""
import pytest
import torch

from w4_gemm_amd import _lib

# the addresses are not memory: where a device is there, a call that is not refused would run on them
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
E_WORKSPACE = 6

SIZES = {
    "fwd": lambda m, p: _lib.sq_linear_fwd_f8_workspace_bytes(m, p),
    "dgrad": lambda m, p: _lib.sq_linear_dgrad_f8_workspace_bytes(m, p),
    "gated_fwd": lambda m, p: _lib.sq_gated_fwd_f8_workspace_bytes(m, p),
    "gated_bwd": lambda m, p: _lib.sq_gated_bwd_f8_workspace_bytes(m, p),
}


def _call(kind, m, p, nb, bf16):
    """The status of a call with a workspace of nb bytes."""
    a, g, u, y, ws, dt = 0x8000, 0xC000, 0xD000, 0x9000, 0xA000, _lib.SQ_BF16 if bf16 else _lib.SQ_F32
    if kind == "fwd":
        return _lib.sq_linear_fwd_f8(a, m, p, y, dt, ws, nb, None)
    if kind == "dgrad":
        return _lib.sq_linear_dgrad_f8(a, m, p, y, dt, ws, nb, None)
    if kind == "gated_fwd":
        return _lib.sq_gated_fwd_f8(a, m, p, p, 0, y, dt, g, u, ws, nb, None)
    return _lib.sq_gated_bwd_f8(a, g, u, m, p, p, 0, y, dt, None, None, ws, nb, None)


@pytest.mark.parametrize("kind,n,k", [("fwd", 2051, 4099), ("fwd", 16384, 6144), ("dgrad", 2048, 4096),
                                      ("gated_fwd", 1024, 2304), ("gated_bwd", 1024, 2304)])
def test_a_size_is_that_of_exactly_its_rows(kind, n, k):
    """A buffer for many rows need not do for fewer, which split the contraction: such a call is refused
    with SQ_E_WORKSPACE before anything is launched (its larger size is the split's partial sums)."""
    p = _lib.SqF8(n, k, 0x1000, 0x2000)
    rows = range(17, 6000, 61)
    sizes = [SIZES[kind](m, p) for m in rows]
    assert all(sizes)
    seen = 0
    for i, m in enumerate(rows):
        later = min(sizes[i:])
        if later < sizes[i]:
            seen += 1
            assert max(_lib.f8_form(kind, m, n, k, 1, bf16)[3] for bf16 in (False, True)) > 1
            # the size is the larger of both result types': at least that one's call is refused
            assert E_WORKSPACE in [_call(kind, m, p, later, bf16) for bf16 in (False, True)]
    assert seen > 0


@pytest.mark.parametrize("kind", SIZES)
def test_one_byte_less_is_refused(kind):
    p = _lib.SqF8(1024, 2304, 0x1000, 0x2000)
    for m in (1, 17, 300, 777, 1024, 2048):
        size = SIZES[kind](m, p)
        assert E_WORKSPACE in [_call(kind, m, p, size - 1, bf16) for bf16 in (False, True)]
