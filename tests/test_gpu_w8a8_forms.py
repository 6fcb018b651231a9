"""The int8 mode's 8-bit products in each form of their kernels (tests/w8a8_forms.py): what only one
form can get wrong."""
import numpy as np
import pytest
import torch

from tests import w8a8_forms as F
from tests import w8a8_reference as R
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4_gemm_amd  # noqa: F401


def _sides():
    import w4_gemm_amd as W
    return {False: (W.grouped_fwd_w8a8, W.grouped_fwd_w8a8_workspace_bytes, R.forward, 1.0),
            True: (W.grouped_dgrad_w8, W.grouped_dgrad_w8_workspace_bytes, R.gradient, 1e-3)}


def _rows(rng, m, n, k, dgrad, scale):
    return R.make_rows(rng, m, n if dgrad else k, dev(), scale)


# ------------------------------------------------------------------ splits and offsets
ONE = [(False, F.FWD[64, 256, True]), (False, F.FWD[128, 256, True]), (True, F.GRAD[64, True]),
       (True, F.GRAD[128, True])]


@pytest.mark.parametrize("dgrad,shape", ONE, ids=[f"{'grad' if d else 'fwd'}-{s}" for d, s in ONE])
@pytest.mark.parametrize("part", [(0.0, 1.0), (0.01, 0.1), (0.3, 0.55), (0.97, 1.0), (0.5, 0.5)])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_split_plan_with_some_of_the_rows(dgrad, shape, part, dt):
    """The plan cuts the contraction for all rows; the offsets, read on the device, leave fewer tiles,
    which are cut into other parts (the gradient's number of parts follows from the tiles), or none."""
    import w4_gemm_amd as W
    m, n, k = shape
    assert F.form(m, n, k, 1, 16, dgrad)[-1]
    lo, hi = (int(p * m) for p in part)
    rng = np.random.default_rng(m + lo)
    call, size, ref, scale = _sides()[dgrad]
    lay = R.make_layer(rng, n, k, 16, dev(), groups=1)
    p = W.GroupedW8Payload(*lay)
    a = _rows(rng, m, n, k, dgrad, scale)
    nbytes = size(m, p)
    ws = torch.full((nbytes + 4096,), 255, dtype=torch.uint8, device=dev())
    out = torch.full((m, k if dgrad else n), -77.0, dtype=dt, device=dev())
    call(a, torch.tensor([lo, hi], dtype=torch.int32, device=dev()), p, out=out,
         workspace=ws[:nbytes])
    want = torch.full(out.shape, -77.0, dtype=torch.float64, device=dev())
    tol = torch.zeros_like(want)
    if hi > lo:
        want[lo:hi], tol[lo:hi] = ref(a[lo:hi], *(t[0] for t in lay), dt)
    R.check(out, want, tol)
    assert bool((ws[nbytes:] == 255).all())


WRONG = [(False, s) for s in F.FWD_SPLIT.values()] + [(True, s) for s in F.GRAD_SPLIT.values()] \
    + [(True, s) for s in F.GRAD_SPLIT_MANY]


@pytest.mark.parametrize("dgrad,shape", WRONG, ids=[f"{'grad' if d else 'fwd'}-{s}" for d, s in WRONG])
def test_split_plan_with_wrong_offsets_stays_inside(dgrad, shape):
    """Offsets out of order, out of range and claiming rows again and again: rows may be wrong, but
    nothing in front of or behind the result and the workspace with its partial sums is touched."""
    import w4_gemm_amd as W
    m, n, k, groups = shape
    assert F.form(m, n, k, groups, 16, dgrad)[-1]
    rng = np.random.default_rng(m + groups)
    call, size, _, scale = _sides()[dgrad]
    p = W.GroupedW8Payload(*R.make_layer(rng, n, k, 16, dev(), groups=groups))
    a = _rows(rng, m, n, k, dgrad, scale)
    nbytes, cols = size(m, p), k if dgrad else n
    orders = [[0, m] * groups,                                   # every second expert claims all rows
              [m, 0] * groups,
              list(rng.integers(-m, 2 * m, groups + 1)),
              [0, 2 ** 31 - 1, -2 ** 31, m // 2] * groups,
              list(np.linspace(m, 0, groups + 1).astype(int))]
    for bad in orders:
        print(f"offsets {bad[:5]}", flush=True)
        offsets = torch.tensor(bad[:groups + 1], dtype=torch.int32, device=dev())
        whole = torch.full((m + 40, cols), 5.0, dtype=F32, device=dev())
        ws = torch.full((4096 + nbytes + (1 << 22),), 7, dtype=torch.uint8, device=dev())
        call(a, offsets, p, out=whole[20:20 + m], workspace=ws[4096:4096 + nbytes])
        torch.cuda.synchronize()
        assert bool((whole[:20] == 5.0).all()) and bool((whole[m + 20:] == 5.0).all())
        assert bool((ws[:4096] == 7).all()) and bool((ws[4096 + nbytes:] == 7).all())


@pytest.mark.parametrize("dgrad,shape", WRONG, ids=[f"{'grad' if d else 'fwd'}-{s}" for d, s in WRONG])
def test_split_plan_gives_the_same_bits(dgrad, shape):
    """Joined sums do not depend on which workgroup ends first; uneven experts in order."""
    import w4_gemm_amd as W
    m, n, k, groups = shape
    assert F.form(m, n, k, groups, 32, dgrad)[-1]
    rng = np.random.default_rng(m + groups + 1)
    call, _, ref, scale = _sides()[dgrad]
    lay = R.make_layer(rng, n, k, 32, dev(), groups=groups)
    p = W.GroupedW8Payload(*lay)
    a = _rows(rng, m, n, k, dgrad, scale)
    share = rng.exponential(size=groups) + 0.05
    off = np.concatenate([[0], np.cumsum(rng.multinomial(m, share / share.sum()))])
    offsets = torch.from_numpy(off.astype(np.int32)).to(dev())
    first = call(a, offsets, p)
    for _ in range(4):
        assert torch.equal(call(a, offsets, p), first)
    for e in range(groups):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            R.check(first[lo:hi], *ref(a[lo:hi], *(t[e] for t in lay), F32))
