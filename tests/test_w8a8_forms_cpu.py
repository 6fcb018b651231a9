"""Every form of the 8-bit products' kernels is reached by the GPU tests: the planners run on the host,
so a refit of their models that moves a tested shape to another form shows here."""
import pytest

from tests import test_gpu_w8a8 as T
from tests import w8a8_forms as F
from w4_gemm_amd import _lib

RANKS = (0, 16, 32, 64)


@pytest.mark.parametrize("rank", RANKS)
def test_shapes_have_their_form(rank):
    for want, shape in F.FWD.items():
        assert F.form(*shape, rank=rank) == want
    for want, shape in F.GRAD.items():
        assert F.form(*shape, rank=rank, dgrad=True) == want
    for rows, shape in F.FWD_SPLIT.items():
        assert F.form(*shape, rank=rank) == (rows, 256, True)
    for rows, shape in F.GRAD_SPLIT.items():
        assert F.form(*shape, rank=rank, dgrad=True) == (rows, True)
    for shape in F.GRAD_SPLIT_MANY:
        assert F.form(*shape, rank=rank, dgrad=True) == (64, True)


def test_tiled_shapes_reach_every_form():
    """The shape lists of the comparisons with 64 bits, one layer and experts."""
    small = {F.form(m, n, k, 1, rank) for m, n, k, rank in T.FWD}
    assert {F.form(*s) for s in T.TILED_FWD} | small == set(F.FWD)
    assert {F.form(*s, dgrad=True) for s in T.TILED_GRAD} == set(F.GRAD)
    several = [s for s in T.TILED_FWD if s[3] > 1]
    assert {F.form(*s) for s in several} | {(16, 16, False)} == set(F.FWD)
    assert {F.form(*s, dgrad=True) for s in T.TILED_GRAD if s[3] > 1} == set(F.GRAD)


def test_no_other_form_is_planned():
    """A walk over the sizes finds no form that the tables do not name."""
    fwd, grad = set(), set()
    for groups in (1, 3, 64):
        for m in (1, 5, 16, 40, 65, 130, 300, 700, 1500, 4480, 16384):
            for n in (1, 70, 300, 1000, 2816, 5000, 16384):
                for k in (256, 512, 2048, 6144, 16384, 65536):
                    fwd.add(F.form(m, n, k, groups))
                    grad.add(F.form(m, n, k, groups, dgrad=True))
    assert fwd <= set(F.FWD) and grad <= set(F.GRAD)


def test_form_of_refused_sizes():
    for bad in (dict(m=0), dict(k=300), dict(n=0), dict(groups=0), dict(rank=8), dict(k=65792)):
        args = dict(m=4, n=16, k=256, groups=1, rank=16) | bad
        for dgrad in (False, True):
            with pytest.raises(ValueError):
                _lib.i8_form(*args.values(), dgrad)
    assert len(_lib.i8_form(4, 16, 256)) == 5
