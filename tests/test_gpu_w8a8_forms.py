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


# ------------------------------------------------------------------ the rank-r branch alone
def _exact_branch(rng, m, cols_in, cols_out, rank):
    """Rows a and factors (first [cols_in][rank], second [cols_out][rank]) whose product t = a first
    is exact in fp32 in any order of summation, and outputs that are u (t[2j] - t[2j + 1]).

    a row of a holds +-1, +-2^-8 and +-2^-16 times a power of two at one even and two odd columns;
    first's values are k / 128, 128 <= k <= 240, so every sum is a multiple of 2^-23 below 2 and fits
    24 bits.  Even columns are alike in rank columns 2j and 2j + 1: the leading part of t cancels in
    the output and what is left is the lower parts'."""
    first = rng.integers(128, 241, (cols_in, rank)) / 128.0 * rng.choice([-1.0, 1.0], (cols_in, rank))
    first[0::2, 1::2] = first[0::2, 0::2]
    a = np.zeros((m, cols_in))
    row = np.arange(m)
    scale = 2.0 ** rng.integers(-20, 11, m)
    odd = np.stack([rng.choice(cols_in // 2, 2, replace=False) for _ in row]) * 2 + 1
    a[row, rng.integers(0, (cols_in + 1) // 2, m) * 2] = rng.choice([-1.0, 1.0], m) * scale
    a[row, odd[:, 0]] = rng.choice([-1.0, 1.0], m) * 2.0 ** -8 * scale
    a[row, odd[:, 1]] = rng.choice([-1.0, 1.0], m) * 2.0 ** -16 * scale
    second = np.zeros((cols_out, rank))
    out, pair = np.arange(cols_out), rng.integers(0, rank // 2, cols_out)
    u = rng.integers(128, 256, cols_out) / 128.0
    second[out, 2 * pair], second[out, 2 * pair + 1] = u, -u
    bf = lambda v: torch.from_numpy(v).to(BF16).to(dev())   # noqa: E731
    for v in (a, first, second):
        assert torch.equal(torch.from_numpy(v).to(BF16).double(), torch.from_numpy(v))
    return bf(a), bf(first), bf(second)


BRANCH = [(False, s) for s in F.FWD.values()] + [(True, s) for s in F.GRAD.values()]


@pytest.mark.parametrize("dgrad,shape", BRANCH, ids=[f"{'grad' if d else 'fwd'}-{s}" for d, s in BRANCH])
@pytest.mark.parametrize("rank", [16, 32, 64])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_parts_of_the_rank_branch(dgrad, shape, rank, dt):
    """Codes of zero leave the rank-r term alone.  With an exact t an fp32 result is off by its sums
    only: t's three bf16 parts hold its 24 bits, and an output adds six products, each sum off by at
    most 2^-23 of |u t| (the matrix unit may truncate).  A bf16 result takes two parts, which hold t
    to 2^-17 (two halves of a step), and rounds once by 2^-8.  Either bound is far below what a part
    that is lost or in the wrong place costs: 2^-17 of t for the third, 2^-9 for the second."""
    import w4_gemm_amd as W
    m, n, k = shape
    rng = np.random.default_rng(m + n + k + rank)
    into, out = (n, k) if dgrad else (k, n)
    a, first, second = _exact_branch(rng, m, into, out, rank)
    up, down = (first, second) if dgrad else (second, first)
    p = W.W8Payload(torch.zeros((n, k), dtype=torch.int8, device=dev()),
                    torch.ones(n, dtype=torch.float16, device=dev()), up, down)
    got = (W.linear_dgrad_w8 if dgrad else W.linear_fwd_w8a8)(a, p, out_dtype=dt).double()
    t = a.double() @ first.double()
    assert torch.equal(t.float().double(), t)
    s2 = second.double().t()
    want, size = t @ s2, t.abs() @ s2.abs()
    tol = 6 * 2.0 ** -23 * size
    if dt is BF16:
        tol = tol + 2.0 ** -17 * size
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    R.check(got, want, tol)
    # the bound sees a missing part
    held, parts = torch.zeros_like(t), 2 if dt is F32 else 1
    for _ in range(parts):
        held = held + (t - held).float().bfloat16().double()
    assert float((((held @ s2) - want).abs() > tol).double().mean()) > 0.3


# ------------------------------------------------------------------ rows that are not finite
@pytest.mark.parametrize("rank", [16, 32, 64])
@pytest.mark.parametrize("dgrad", [False, True], ids=["fwd", "grad"])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_rows_that_are_not_finite_with_factors(rank, dgrad, dt):
    """inf and NaN in every form: such a row is NaN throughout and the rows that share its tiles,
    projection tiles and matrix instructions keep their values, the rank-r term included."""
    import w4_gemm_amd as W
    for key, (m, n, k) in (F.GRAD if dgrad else F.FWD).items():
        print(f"form {key}", flush=True)
        rng = np.random.default_rng(m + rank)
        lay = R.make_layer(rng, n, k, rank, dev())
        a = _rows(rng, m, n, k, dgrad, 1.0)
        bad = [r for r in (0, 3, m // 2, m - 1) if m > 1 or r == 0]
        for i, r in enumerate(dict.fromkeys(bad)):
            a[r, (37 * i + 5) % a.shape[1]] = (float("inf"), float("nan"), -float("inf"), 3.3e38)[i]
        last_is_large = len(set(bad)) == 4        # finite itself
        call, ref = ((W.linear_dgrad_w8, R.gradient) if dgrad else (W.linear_fwd_w8a8, R.forward))
        got = call(a, W.W8Payload(*lay), out_dtype=dt)
        finite = torch.isfinite(a).all(1)
        assert bool(torch.isnan(got[~finite]).all())
        keep = finite.clone()
        if last_is_large:
            keep[m - 1] = False                   # a value that may overflow on the way
        if bool(keep.any()):
            R.check(got[keep], *ref(a[keep], *lay, dt))


# ------------------------------------------------------------------ captured
@pytest.mark.parametrize("dgrad,shape", WRONG, ids=[f"{'grad' if d else 'fwd'}-{s}" for d, s in WRONG])
def test_split_plan_in_a_graph(dgrad, shape):
    """A captured call whose sums are joined follows new rows and new offsets, which leave other
    numbers of tiles and parts each time, eager calls with another workspace between the replays."""
    import w4_gemm_amd as W
    m, n, k, groups = shape
    assert F.form(m, n, k, groups, 16, dgrad)[-1]
    rng = np.random.default_rng(m + groups + 2)
    call, size, ref, scale = _sides()[dgrad]
    lay = R.make_layer(rng, n, k, 16, dev(), groups=groups)
    p = W.GroupedW8Payload(*lay)
    a = _rows(rng, m, n, k, dgrad, scale)
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device=dev())
    out = torch.empty((m, k if dgrad else n), dtype=F32, device=dev())
    ws = torch.full((size(m, p),), 255, dtype=torch.uint8, device=dev())
    call(a, offsets, p, out=out, workspace=ws)           # loads the kernels
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            call(a, offsets, p, out=out, workspace=ws)
    torch.cuda.synchronize()
    for rows in (m, max(1, m // 9), 0, m - 1, m // 2):
        share = rng.exponential(size=groups) + 0.05
        off = np.concatenate([[0], np.cumsum(rng.multinomial(rows, share / share.sum()))])
        offsets.copy_(torch.from_numpy(off.astype(np.int32)))
        a.copy_(_rows(rng, m, n, k, dgrad, scale))
        out.fill_(-77.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        eager = torch.full_like(out, -77.0)
        call(a, offsets, p, out=eager)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), rows
        e = int(np.argmax(np.diff(off)))                 # the fullest expert against 64 bits
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            R.check(out[lo:hi], *ref(a[lo:hi], *(t[e] for t in lay), F32))
        assert bool((out[rows:] == -77.0).all())
