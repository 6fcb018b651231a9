"""The sizes of f8_deep_forms.py take the forms that they are listed with, and every kernel of the 8-bit
float products that the planner can choose is run by a test: with its curve, and where its contraction is
not split with more than two rounds of the four-stage loop."""
import pytest

from tests.f8_deep_forms import CURVES, DEEP, SPLIT, stages, with_curves
from tests.f8_forms import FORMS
from w4_gemm_amd import _lib


@pytest.mark.parametrize("kind,m,n,k,e,bits,rows,cols,splits", DEEP + SPLIT)
def test_form(kind, m, n, k, e, bits, rows, cols, splits):
    form = _lib.f8_form(kind, m, n, k, e, bits == 16)
    assert (form[0], form[1], form[3]) == (rows, cols, splits)


def test_deep_forms_are_deep():
    for kind, m, n, k, e, bits, rows, cols, splits in DEEP:
        assert splits == 1 and stages(kind, n, k) >= 9 and stages(kind, n, k) % 4 > 0
        if e == 1 and rows >= 128:   # the last tile contracts half of its row tiles
            assert 1 <= m % rows <= 32 * ((rows // 32 + 1) // 2)
        if e > 1:                    # and so does one of an expert's
            assert m >= 2 * rows + 9


def test_every_kernel_is_run():
    """Tiles through LDS: kind, bits of the result, rows, split or not, curve (of the gated forward)."""
    got = {(kind, bits, rows, splits > 1, act)
           for kind, _, _, _, _, bits, rows, _, splits, act in with_curves(DEEP + SPLIT)}
    got |= {(kind, bits, rows, splits > 1, CURVES[0]) for kind, _, _, _, _, bits, rows, _, splits in FORMS
            if kind != "gated_fwd"}
    got |= {(kind, bits, rows, True, None) for kind, _, _, _, _, bits, rows, _, splits in FORMS if splits > 1}
    for kind in _lib.F8_KINDS:
        for bits, heights in ((16, (64, 128, 224, 256)), (32, (64, 128))):
            for rows in heights:
                for act in CURVES if kind == "gated_fwd" else CURVES[:1]:
                    assert (kind, bits, rows, False, act) in got
                # split: the product's kernel knows no curve, the join is told it
                assert any((kind, bits, rows, True, act) in got for act in (*CURVES, None))
    for bits in (16, 32):
        for act in CURVES:
            assert ("gated_fwd", bits, 64, True, act) in got
    deep = {(kind, bits, rows) for kind, _, _, _, _, bits, rows, _, _ in DEEP}
    assert deep == {(kind, bits, rows) for kind in _lib.F8_KINDS
                    for bits, heights in ((16, (64, 128, 224, 256)), (32, (64, 128))) for rows in heights}
    # every way out of the four-stage loop, in the kernels that hold their accumulators in place
    for kind in ("fwd", "dgrad", "gated_fwd"):
        for rows in (224, 256):
            ways = {stages(f[0], f[2], f[3]) % 4 for f in DEEP if (f[0], f[6]) == (kind, rows)}
            assert ways == {1, 2, 3}
