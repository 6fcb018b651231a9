"""The planner of the 8-bit float products: the sizes of the forms' tests take the forms they are
listed with, and between them every kernel is reached."""
import pytest

from tests.f8_forms import FORMS
from w4_gemm_amd import _lib


@pytest.mark.parametrize("kind,m,n,k,e,bits,rows,cols,splits", FORMS)
def test_form(kind, m, n, k, e, bits, rows, cols, splits):
    form = _lib.f8_form(kind, m, n, k, e, bits == 16)
    assert (form[0], form[1], form[3]) == (rows, cols, splits)


def test_every_form_is_listed():
    got = {(kind, bits, rows, cols if rows == 16 else 0, splits > 1)
           for kind, _, _, _, _, bits, rows, cols, splits in FORMS}
    for kind in _lib.F8_KINDS:
        for bits in (16, 32):
            for rows in (64, 128, 224, 256) if bits == 16 else (64, 128):
                assert (kind, bits, rows, 0, False) in got
                if rows < 224:
                    assert (kind, bits, rows, 0, True) in got
            if kind in ("fwd", "gated_fwd"):
                for cols in (16, 32, 64) if kind == "fwd" else (16, 32):
                    assert (kind, bits, 16, cols, False) in got
    for kind, rows in (("dgrad", 224), ("gated_bwd", 224), ("gated_bwd", 256), ("fwd", 224), ("gated_fwd", 224)):
        assert (kind, 16, rows, 0, True) in got


def test_form_refuses_what_the_calls_refuse():
    for args in (("fwd", 0, 8, 8), ("fwd", 4, 0, 8), ("dgrad", 4, 8, (1 << 20) + 1), ("gated_fwd", 1 << 31, 8, 8)):
        with pytest.raises(ValueError):
            _lib.f8_form(*args)


@pytest.mark.parametrize("kind,n,k", [("fwd", 24, 140000), ("dgrad", 140000, 24), ("gated_bwd", 70000, 24),
                                      ("gated_fwd", 24, 1 << 20)])
def test_long_contractions_are_split(kind, n, k):
    """A workgroup holds the weight's exponents of 1024 blocks."""
    blocks = -(-(n if kind in ("dgrad", "gated_bwd") else k) // 128) * (2 if kind == "gated_bwd" else 1)
    for bf16 in (False, True):
        form = _lib.f8_form(kind, 600, n, k, 1, bf16)
        assert form[0] > 16 and form[3] >= -(-blocks // 1024)
