"""The int8 mode's 8-bit forward and input gradient, for one layer and for experts, against the
64-bit reference (SquareQ README, "v3.1 - int8-residual mode", with 8-bit tokens)."""
import numpy as np
import pytest
import torch

from tests import w8a8_reference as R
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4_gemm_amd  # noqa: F401


def _workspace(nbytes):
    """A caller's workspace full of 0xFF (NaN in every float format)."""
    return torch.full((max(nbytes, 16),), 255, dtype=torch.uint8, device=dev())


def _forward(x, lay, dt):
    import w4_gemm_amd as W
    p = W.W8Payload(*lay)
    ws = _workspace(W.fwd_w8a8_workspace_bytes(x.shape[0], p))
    out = torch.full((x.shape[0], p.n), float("nan"), dtype=dt, device=dev())
    return W.linear_fwd_w8a8(x, p, out=out, workspace=ws)


def _gradient(dy, lay, dt):
    import w4_gemm_amd as W
    p = W.W8Payload(*lay)
    ws = _workspace(W.dgrad_w8_workspace_bytes(dy.shape[0], p))
    out = torch.full((dy.shape[0], p.k), float("nan"), dtype=dt, device=dev())
    return W.linear_dgrad_w8(dy, p, out=out, workspace=ws)


# ------------------------------------------------------------------ one layer
FWD = [  # m, n, k, rank
    (1, 1, 256, 0), (1, 16, 256, 16), (2, 33, 512, 32), (1, 520, 6144, 16), (3, 300, 2048, 64),
    (15, 65, 768, 0), (16, 512, 512, 32), (17, 129, 1280, 16), (31, 256, 256, 64), (33, 48, 4096, 16),
    (48, 96, 16384, 16), (64, 512, 512, 32), (65, 255, 768, 16), (127, 257, 2304, 0), (129, 1003, 1536, 32),
    (255, 64, 256, 16), (257, 513, 512, 0), (300, 260, 4352, 64), (700, 1024, 768, 16), (2, 24, 65536, 16),
]


@pytest.mark.parametrize("m,n,k,rank", FWD)
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_forward(m, n, k, rank, dt):
    rng = np.random.default_rng(m + n + k + rank)
    lay = R.make_layer(rng, n, k, rank, dev())
    x = R.make_rows(rng, m, k, dev())
    R.check(_forward(x, lay, dt), *R.forward(x, *lay, dt))


GRAD = [
    (1, 1, 256, 0), (1, 63, 256, 16), (2, 64, 512, 32), (4, 65, 768, 64), (16, 1, 1024, 16),
    (16, 512, 512, 32), (33, 200, 256, 0), (64, 2049, 256, 16), (127, 700, 1280, 32), (129, 2051, 512, 64),
    (130, 2048, 768, 16), (257, 320, 2304, 0), (300, 4099, 512, 16), (1, 16384, 256, 16), (2, 131072, 256, 0),
]


@pytest.mark.parametrize("m,n,k,rank", GRAD)
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_gradient(m, n, k, rank, dt):
    rng = np.random.default_rng(m + n + k + rank)
    lay = R.make_layer(rng, n, k, rank, dev())
    dy = R.make_rows(rng, m, n, dev(), 1e-3)
    R.check(_gradient(dy, lay, dt), *R.gradient(dy, *lay, dt))


def test_gradient_is_that_of_the_layer():
    """dx against differences of the unrounded layer: <dx, u> = (f(x + u) - f(x - u)) / 2 for
    f(x) = <dy, x W_hat^T>, which is linear, in 64 bits.  The 16-bit rows of dy w round to half a
    step, 2^-16 of the row's largest value each."""
    import w4_gemm_amd as W
    rng = np.random.default_rng(5)
    m, n, k, rank = 40, 300, 512, 32
    lay = R.make_layer(rng, n, k, rank, dev())
    codes, w, up, down = lay
    dy = R.make_rows(rng, m, n, dev(), 1e-3)
    dx = _gradient(dy, lay, F32).double()
    h = R.sylvester(dev()) / 16.0
    what = ((codes.double() * w.double()[:, None]).view(n, -1, 256) @ h).view(n, k) \
        + up.double() @ down.double().t()
    x = torch.from_numpy(rng.standard_normal((m, k))).to(dev())
    for _ in range(5):
        u = torch.from_numpy(rng.standard_normal((m, k))).to(dev())
        f = lambda z: (dy.double() * (z @ what.t())).sum()   # noqa: E731
        diff = (f(x + u) - f(x - u)) / 2
        _, tol = R.gradient(dy, *lay, F32)
        v = (dy.double() * w.double()).abs().amax(1, keepdim=True)
        step = (v * 2.0 ** -16 * 1.01) @ codes.double().abs().sum(0, keepdim=True)   # |d error| |c|
        step = step.view(m, -1, 256).sum(2, keepdim=True).expand(-1, -1, 256).reshape(m, k) / 16.0
        bound = ((tol + step) * u.abs()).sum() + 1e-12 * (dy.double().abs() @ what.abs()).sum()
        assert abs(float((dx * u).sum() - diff)) <= float(bound)
    # and it differentiates both int8-mode forwards: y of linear_fwd_w8 is x W_hat^T
    xb = x.bfloat16()
    p = W.W8Payload(*lay)
    y = W.linear_fwd_w8(xb, p).double()
    ref = xb.double() @ what.t()
    assert float((y - ref).norm() / ref.norm()) < 2e-3


# one shape for each tile form of the contractions (few rows and split K, 16 to 256 rows, tails cut
# into parts), one layer and experts; odd widths where the form allows
TILED_FWD = [
    (4584, 781, 256, 1), (433, 5955, 256, 7), (3800, 17, 11776, 1), (1219, 55, 12800, 4),
    (1, 10947, 1792, 1), (4, 4140, 512, 6), (1029, 7545, 256, 1), (659, 8211, 256, 4),
    (3000, 4701, 256, 1), (608, 9170, 256, 4), (21, 4507, 2048, 1), (2502, 49, 1792, 2),
    (65, 10276, 256, 1), (107, 4840, 256, 7), (17, 2381, 12544, 1), (26, 1519, 14592, 2),
    (34, 10247, 1536, 1), (4869, 70, 1792, 9),
]
TILED_GRAD = [
    (395, 1, 9728, 1), (107, 1, 13056, 5), (68, 4602, 11008, 1), (49, 8922, 15360, 2),
    (1637, 1323, 5120, 1), (4657, 1329, 1792, 4), (1, 771, 256, 1), (1, 836, 256, 6),
    (548, 2864, 14592, 1), (274, 3040, 14080, 9), (700, 2500, 1024, 1), (3678, 2684, 2304, 1),
    (4498, 4748, 2048, 4),
]


def _uneven(rng, m, groups):
    share = rng.exponential(size=groups) + 0.05
    return np.concatenate([[0], np.cumsum(rng.multinomial(m, share / share.sum()))])


@pytest.mark.parametrize("m,n,k,groups", TILED_FWD)
@pytest.mark.parametrize("rank,dt", [(0, F32), (16, BF16), (16, F32), (64, F32)])
def test_forward_tiles(m, n, k, groups, rank, dt):
    import w4_gemm_amd as W
    rng = np.random.default_rng(m + n + k + rank)
    x = R.make_rows(rng, m, k, dev())
    if groups == 1:
        lay = R.make_layer(rng, n, k, rank, dev())
        R.check(_forward(x, lay, dt), *R.forward(x, *lay, dt))
        return
    lay = R.make_layer(rng, n, k, rank, dev(), groups=groups)
    off = _uneven(rng, m, groups)
    p = W.GroupedW8Payload(*lay)
    out = torch.full((m, n), float("nan"), dtype=dt, device=dev())
    W.grouped_fwd_w8a8(x, torch.from_numpy(off.astype(np.int32)).to(dev()), p, out=out,
                       workspace=_workspace(W.grouped_fwd_w8a8_workspace_bytes(m, p)))
    R.check(out, *_experts(R.forward, x, off, lay, dt, n))


@pytest.mark.parametrize("m,n,k,groups", TILED_GRAD)
@pytest.mark.parametrize("rank,dt", [(0, F32), (16, BF16), (16, F32), (64, F32)])
def test_gradient_tiles(m, n, k, groups, rank, dt):
    import w4_gemm_amd as W
    rng = np.random.default_rng(m + n + k + rank)
    dy = R.make_rows(rng, m, n, dev(), 1e-3)
    if groups == 1:
        lay = R.make_layer(rng, n, k, rank, dev())
        R.check(_gradient(dy, lay, dt), *R.gradient(dy, *lay, dt))
        return
    lay = R.make_layer(rng, n, k, rank, dev(), groups=groups)
    off = _uneven(rng, m, groups)
    p = W.GroupedW8Payload(*lay)
    out = torch.full((m, k), float("nan"), dtype=dt, device=dev())
    W.grouped_dgrad_w8(dy, torch.from_numpy(off.astype(np.int32)).to(dev()), p, out=out,
                       workspace=_workspace(W.grouped_dgrad_w8_workspace_bytes(m, p)))
    R.check(out, *_experts(R.gradient, dy, off, lay, dt, k))


def test_same_call_gives_the_same_bits():
    """Forms that join split sums included: nothing depends on which workgroup ends first."""
    rng = np.random.default_rng(9)
    for m, n, k in ((17, 2381, 12544), (68, 4602, 11008), (300, 1000, 2048)):
        lay = R.make_layer(rng, n, k, 32, dev())
        x, dy = R.make_rows(rng, m, k, dev()), R.make_rows(rng, m, n, dev(), 1e-3)
        y, dx = _forward(x, lay, F32), _gradient(dy, lay, F32)
        for _ in range(3):
            assert torch.equal(_forward(x, lay, F32), y)
            assert torch.equal(_gradient(dy, lay, F32), dx)


# ------------------------------------------------------------------ values
def _value_rows(k):
    """Rows that go wrong first: zeros, one value, subnormals, the smallest and largest, wide
    spreads inside a block and between blocks, infinities and NaN."""
    rng = np.random.default_rng(11)
    rows = [np.zeros(k), np.ones(k), np.full(k, -2.5), np.full(k, 1e-39), np.full(k, 3e-32),
            np.full(k, 1e37), np.full(k, 3.3e38)]
    one = np.zeros(k); one[k - 1] = -3.0
    rows.append(one)
    rows.append(rng.standard_normal(k) * 2.0 ** rng.integers(-40, 1, k))
    rows.append(rng.standard_normal(k) * 2.0 ** np.repeat(rng.integers(-60, 60, k // 256), 256))
    last = rng.standard_normal(k); last[:-256] = 0.0
    rows.append(last)
    for bad in (np.inf, -np.inf, np.nan):
        r = rng.standard_normal(k); r[rng.integers(0, k)] = bad
        rows.append(r)
    rows.append(rng.standard_normal(k))
    return torch.from_numpy(np.stack(rows).astype(np.float32)).bfloat16().to(dev())


@pytest.mark.parametrize("repeat", [1, 5, 20])
def test_forward_values(repeat):
    """Each kind of row beside the others; a row that is not finite spoils only itself.  (1e37 and
    3.3e38 overflow in x H: their rows are NaN, as for inf; the reference says which.)"""
    k, n = 768, 70
    rng = np.random.default_rng(3)
    lay = R.make_layer(rng, n, k, 16, dev())
    x = _value_rows(k).repeat(repeat, 1)
    lay0 = (lay[0], lay[1], None, None)
    y, tol = R.forward(x, *lay0, F32)
    got = _forward(x, lay0, F32)
    over = (x.double().abs().amax(1) >= 1e37) & torch.isfinite(x).all(1)
    # x H of a constant row is 16 x in column 0: 1.6e38 is finite, 5.3e39 is not
    nan_rows = ~torch.isfinite(x).all(1) | (x.double().abs().amax(1) > 1e38)
    assert bool(torch.isnan(got[nan_rows]).all())
    keep = ~nan_rows
    R.check(got[keep], y[keep], tol[keep] + 2.0 ** -149)
    assert bool(over.any())
    # with factors the same rows are NaN and the finite ordinary ones match
    y, tol = R.forward(x, *lay, F32)
    got = _forward(x, lay, F32)
    ordinary = keep & (x.double().abs().amax(1) < 1e30)
    R.check(got[ordinary], y[ordinary], tol[ordinary] + 2.0 ** -120)
    assert bool(torch.isnan(got[~torch.isfinite(x).all(1)]).all())


@pytest.mark.parametrize("repeat", [1, 12])
def test_gradient_values(repeat):
    n, k = 768, 512
    rng = np.random.default_rng(4)
    lay = R.make_layer(rng, n, k, 0, dev())
    dy = _value_rows(n).repeat(repeat, 1)
    y, tol = R.gradient(dy, *lay, F32)
    got = _gradient(dy, lay, F32)
    finite = torch.isfinite(dy).all(1)
    assert bool(torch.isnan(got[~finite]).all())
    small = finite & (dy.double().abs().amax(1) < 1e30)
    R.check(got[small], y[small], tol[small] + 2.0 ** -120)


def test_scale_of_a_row_that_is_not_finite():
    """An infinite payload scale spoils its own output column (forward) and every row (gradient)."""
    n, k = 40, 256
    rng = np.random.default_rng(6)
    codes, w, _, _ = R.make_layer(rng, n, k, 0, dev())
    w[7] = float("inf")
    x = R.make_rows(rng, 20, k, dev())
    y = _forward(x, (codes, w, None, None), F32)
    others = [i for i in range(n) if i != 7]
    assert not bool(torch.isfinite(y[:, 7]).any())
    assert bool(torch.isfinite(y[:, others]).all())
    dx = _gradient(R.make_rows(rng, 20, n, dev()), (codes, w, None, None), F32)
    assert bool(torch.isnan(dx).all())


def test_row_does_not_depend_on_the_batch():
    """A row's result is the same bits alone, in a small batch and in one of another kernel."""
    n, k = 300, 2048
    rng = np.random.default_rng(8)
    lay = (*R.make_layer(rng, n, k, 0, dev())[:2], None, None)
    x = R.make_rows(rng, 300, k, dev())
    full = _forward(x, lay, F32)
    for m in (1, 5, 16, 40, 100):
        assert torch.equal(_forward(x[:m].contiguous(), lay, F32), full[:m]), m


def test_extreme_integers():
    """Codes and tokens at the ends of their ranges: |sum| close to 2^30 at K = 65536."""
    n, k = 20, 65536
    codes = torch.full((n, k), -128, dtype=torch.int8, device=dev())
    codes[n // 2:] = 127
    w = torch.full((n,), 2.0 ** -10, dtype=torch.float16, device=dev())
    x = torch.zeros((3, k), dtype=BF16, device=dev())
    x[:, ::256] = 1.0                    # an impulse per block: x H is constant, every q is 127
    lay = (codes, w, None, None)
    R.check(_forward(x, lay, F32), *R.forward(x, *lay, F32))
    n, k = 131072, 256
    codes = torch.full((n, k), -128, dtype=torch.int8, device=dev())
    w = torch.full((n,), 2.0 ** -10, dtype=torch.float16, device=dev())
    lay = (codes, w, None, None)
    dy = torch.ones((2, n), dtype=BF16, device=dev())
    dy[1] = -1.0
    R.check(_gradient(dy, lay, F32), *R.gradient(dy, *lay, F32))


# ------------------------------------------------------------------ experts
def _experts(fn, a, offsets, lay, dt, cols):
    """Reference per expert; rows outside every range stay at the marker."""
    want = torch.full((a.shape[0], cols), -77.0, dtype=torch.float64, device=dev())
    tol = torch.zeros_like(want)
    for e in range(lay[0].shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            one = tuple(None if t is None else t[e] for t in lay)
            want[lo:hi], tol[lo:hi] = fn(a[lo:hi], *one, dt)
    return want, tol


COUNTS = [
    [5], [0], [0, 7, 0], [1, 1, 1, 1], [300, 0, 2, 257], [16, 32, 64, 128], [129, 1, 130],
    [3] * 70, [0] * 65 + [40] + [0] * 9, list(range(20)), [700, 3],
]


@pytest.mark.parametrize("counts", COUNTS, ids=[f"{len(c)}x{sum(c)}" for c in COUNTS])
@pytest.mark.parametrize("rank,dt", [(0, F32), (16, BF16), (32, F32), (64, F32)])
def test_experts(counts, rank, dt):
    import w4_gemm_amd as W
    rng = np.random.default_rng(len(counts) + sum(counts) + rank)
    e, n, k = len(counts), 77, 512
    lay = R.make_layer(rng, n, k, rank, dev(), groups=e)
    p = W.GroupedW8Payload(*lay)
    for before, behind in ((0, 0), (2, 9)):
        off = np.concatenate([[0], np.cumsum(counts)]) + before
        m = int(off[-1]) + behind
        offsets = torch.from_numpy(off.astype(np.int32)).to(dev())
        x = R.make_rows(rng, max(m, 1), k, dev())[:m].contiguous()
        dy = R.make_rows(rng, max(m, 1), n, dev(), 1e-3)[:m].contiguous()
        out = torch.full((m, n), -77.0, dtype=dt, device=dev())
        W.grouped_fwd_w8a8(x, offsets, p, out=out,
                           workspace=_workspace(W.grouped_fwd_w8a8_workspace_bytes(m, p)))
        R.check(out, *_experts(R.forward, x, off, lay, dt, n))
        out = torch.full((m, k), -77.0, dtype=dt, device=dev())
        W.grouped_dgrad_w8(dy, offsets, p, out=out,
                           workspace=_workspace(W.grouped_dgrad_w8_workspace_bytes(m, p)))
        R.check(out, *_experts(R.gradient, dy, off, lay, dt, k))


@pytest.mark.parametrize("lo,hi", [(3, 50), (0, 512), (64, 400), (510, 512), (7, 7)])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_one_expert_with_some_of_the_rows(lo, hi, dt):
    """The plan is made for 512 rows (the gradient's tiles cut in two parts); the offsets leave
    fewer tiles, that are cut into more parts, or none."""
    import w4_gemm_amd as W
    rng = np.random.default_rng(31)
    m, n, k = 512, 4096, 4096
    lay = R.make_layer(rng, n, k, 16, dev(), groups=1)
    p = W.GroupedW8Payload(*lay)
    offsets = torch.tensor([lo, hi], dtype=torch.int32, device=dev())
    for call, size, ref, cols, scale in (
            (W.grouped_fwd_w8a8, W.grouped_fwd_w8a8_workspace_bytes, R.forward, n, 1.0),
            (W.grouped_dgrad_w8, W.grouped_dgrad_w8_workspace_bytes, R.gradient, k, 1e-3)):
        a = R.make_rows(rng, m, k if cols == n else n, dev(), scale)
        out = torch.full((m, cols), -77.0, dtype=dt, device=dev())
        call(a, offsets, p, out=out, workspace=_workspace(size(m, p)))
        R.check(out, *_experts(ref, a, [lo, hi], lay, dt, cols))


def test_experts_equal_single_layers():
    """Each expert's rows are the bits that the one-layer calls give (no factors: the number of
    slices of the rank-r sum may differ)."""
    import w4_gemm_amd as W
    rng = np.random.default_rng(21)
    counts, n, k = [40, 0, 300, 9], 130, 768
    lay = R.make_layer(rng, n, k, 0, dev(), groups=4)
    off = np.concatenate([[0], np.cumsum(counts)])
    offsets = torch.from_numpy(off.astype(np.int32)).to(dev())
    m = int(off[-1])
    x, dy = R.make_rows(rng, m, k, dev()), R.make_rows(rng, m, n, dev(), 1e-3)
    singles = [W.W8Payload(lay[0][e], lay[1][e].clone(), None, None) for e in range(4)]
    p = W.stack_payloads_w8(singles)
    y, dx = W.grouped_fwd_w8a8(x, offsets, p), W.grouped_dgrad_w8(dy, offsets, p)
    for e in range(4):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            assert torch.equal(y[lo:hi], W.linear_fwd_w8a8(x[lo:hi].contiguous(), singles[e]))
            assert torch.equal(dx[lo:hi], W.linear_dgrad_w8(dy[lo:hi].contiguous(), singles[e]))


@pytest.mark.parametrize("bad", [[0, 50, 20, 60], [-5, 10, 30, 60], [0, 20, 90, 60], [60, 40, 20, 0],
                                 [0, 2 ** 31 - 1, -2 ** 31, 60], [0, 600] * 10, [0, 600] * 40])
@pytest.mark.parametrize("m,n,k", [(60, 70, 512), (600, 70, 512), (300, 2000, 4096)])
def test_offsets_that_are_wrong_stay_inside(bad, m, n, k):
    """Offsets that are not ordered or not in range, also many that claim the same rows: rows may be
    wrong, nothing else is touched, neither behind the result nor behind the workspace."""
    import w4_gemm_amd as W
    rng = np.random.default_rng(22)
    if len(bad) > 20 and n > 100:
        n = 300
    p = W.GroupedW8Payload(*R.make_layer(rng, n, k, 16, dev(), groups=len(bad) - 1))
    offsets = torch.tensor(bad, dtype=torch.int32, device=dev())
    x, dy = R.make_rows(rng, m, k, dev()), R.make_rows(rng, m, n, dev())
    for call, size, a, cols in ((W.grouped_fwd_w8a8, W.grouped_fwd_w8a8_workspace_bytes, x, n),
                                (W.grouped_dgrad_w8, W.grouped_dgrad_w8_workspace_bytes, dy, k)):
        whole = torch.full((m + 40, cols), 5.0, dtype=F32, device=dev())
        nbytes = size(m, p)
        ws = torch.full((nbytes + (1 << 22),), 7, dtype=torch.uint8, device=dev())
        call(a, offsets, p, out=whole[20:20 + m], workspace=ws[:nbytes])
        torch.cuda.synchronize()
        assert bool((whole[:20] == 5.0).all()) and bool((whole[m + 20:] == 5.0).all())
        assert bool((ws[nbytes:] == 7).all())


def test_offsets_past_32_bits():
    """Results, integers and stacked codes of more than 2^31 elements: the last rows and experts."""
    import w4_gemm_amd as W
    rng = np.random.default_rng(23)
    m, n, k = 140_000, 16384, 256
    lay = R.make_layer(rng, n, k, 16, dev())
    x = torch.randn(m, k, device=dev()).bfloat16()
    y = W.linear_fwd_w8a8(x, W.W8Payload(*lay), out_dtype=BF16)
    for rows in (slice(0, 40), slice(131_050, 131_110), slice(m - 50, m)):
        R.check(y[rows], *R.forward(x[rows], *lay, BF16))
    del y
    n, k = 48, 16384
    lay = R.make_layer(rng, n, k, 16, dev())
    dy = torch.randn(m, n, device=dev()).bfloat16()
    dx = W.linear_dgrad_w8(dy, W.W8Payload(*lay), out_dtype=BF16)
    for rows in (slice(0, 40), slice(131_050, 131_110), slice(m - 50, m)):
        R.check(dx[rows], *R.gradient(dy[rows], *lay, BF16))
    del dx
    groups, n, k = 36, 8192, 8192
    codes = torch.randint(-100, 101, (groups, n, k), dtype=torch.int8, device=dev())
    w = torch.full((groups, n), 1e-4, dtype=torch.float16, device=dev())
    p = W.GroupedW8Payload(codes, w, None, None)
    off = np.concatenate([np.zeros(groups - 1), [30, 70]])     # the last two experts
    offsets = torch.from_numpy(off.astype(np.int32)).to(dev())
    x, dy = R.make_rows(rng, 70, k, dev()), R.make_rows(rng, 70, n, dev(), 1e-3)
    y, dx = W.grouped_fwd_w8a8(x, offsets, p), W.grouped_dgrad_w8(dy, offsets, p)
    for e, rows in ((groups - 2, slice(0, 30)), (groups - 1, slice(30, 70))):
        R.check(y[rows], *R.forward(x[rows], codes[e], w[e], None, None, F32))
        R.check(dx[rows], *R.gradient(dy[rows], codes[e], w[e], None, None, F32))


# ------------------------------------------------------------------ calls together
def test_layers_in_sequence_and_backward():
    """A two-layer expert block (up, down) with its backward, as a training step runs it."""
    import w4_gemm_amd as W
    rng = np.random.default_rng(31)
    counts, hid, k = [70, 0, 33, 150], 512, 256
    off = np.concatenate([[0], np.cumsum(counts)])
    offsets = torch.from_numpy(off.astype(np.int32)).to(dev())
    m = int(off[-1])
    lay1, lay2 = (R.make_layer(rng, hid, k, 16, dev(), groups=4),
                  R.make_layer(rng, k, hid, 16, dev(), groups=4))
    p1, p2 = W.GroupedW8Payload(*lay1), W.GroupedW8Payload(*lay2)
    x = R.make_rows(rng, m, k, dev())
    hmid = W.grouped_fwd_w8a8(x, offsets, p1, out_dtype=BF16)
    act = torch.relu(hmid)
    y = W.grouped_fwd_w8a8(act, offsets, p2, out_dtype=F32)
    dy = R.make_rows(rng, m, k, dev(), 1e-2)
    dact = W.grouped_dgrad_w8(dy, offsets, p2, out_dtype=BF16)
    dh = torch.where(hmid > 0, dact, torch.zeros_like(dact))
    dx = W.grouped_dgrad_w8(dh, offsets, p1, out_dtype=F32)
    R.check(hmid, *_experts(R.forward, x, off, lay1, BF16, hid))
    R.check(y, *_experts(R.forward, act, off, lay2, F32, k))
    R.check(dact, *_experts(R.gradient, dy, off, lay2, BF16, hid))
    R.check(dx, *_experts(R.gradient, dh, off, lay1, F32, k))


@pytest.mark.parametrize("m", [1, 20, 300])
def test_graph(m):
    """Captured forward and gradient, one graph each and a workspace that both graphs share
    (replayed in order on one stream), follow new inputs and new offsets."""
    import w4_gemm_amd as W
    rng = np.random.default_rng(40 + m)
    e, n, k = 3, 200, 768
    lay = R.make_layer(rng, n, k, 16, dev(), groups=e)
    p = W.GroupedW8Payload(*lay)
    ws = _workspace(max(W.grouped_fwd_w8a8_workspace_bytes(m, p),
                        W.grouped_dgrad_w8_workspace_bytes(m, p)))
    x, dy = torch.empty((m, k), dtype=BF16, device=dev()), torch.empty((m, n), dtype=BF16, device=dev())
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=dev())
    y, dx = torch.empty((m, n), dtype=F32, device=dev()), torch.empty((m, k), dtype=F32, device=dev())
    side = torch.cuda.Stream()
    graphs = []
    x.zero_(); dy.zero_()
    W.grouped_fwd_w8a8(x, offsets, p, out=y, workspace=ws)   # loads the kernels
    W.grouped_dgrad_w8(dy, offsets, p, out=dx, workspace=ws)
    torch.cuda.synchronize()
    for call in (lambda: W.grouped_fwd_w8a8(x, offsets, p, out=y, workspace=ws),
                 lambda: W.grouped_dgrad_w8(dy, offsets, p, out=dx, workspace=ws)):
        with torch.cuda.stream(side):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                call()
        graphs.append(g)
    torch.cuda.synchronize()
    for rep in range(4):
        cuts = np.sort(rng.integers(0, m + 1, e - 1))
        off = np.concatenate([[0], cuts, [m]])
        x.copy_(R.make_rows(rng, m, k, dev()))
        dy.copy_(R.make_rows(rng, m, n, dev(), 1e-3))
        offsets.copy_(torch.from_numpy(off.astype(np.int32)))
        y.fill_(float("nan")); dx.fill_(float("nan"))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        ey, edx = W.grouped_fwd_w8a8(x, offsets, p), W.grouped_dgrad_w8(dy, offsets, p)
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(dx, edx), rep
        R.check(y, *_experts(R.forward, x, off, lay, F32, n))


def test_two_streams_at_once():
    """Calls on two streams with a workspace each do not meet."""
    import w4_gemm_amd as W
    rng = np.random.default_rng(50)
    n, k = 512, 2048
    p = W.W8Payload(*R.make_layer(rng, n, k, 32, dev()))
    xs = [R.make_rows(rng, m, k, dev()) for m in (300, 40)]
    dys = [R.make_rows(rng, m, n, dev(), 1e-3) for m in (300, 40)]
    want = [(W.linear_fwd_w8a8(x, p), W.linear_dgrad_w8(d, p)) for x, d in zip(xs, dys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((W.linear_fwd_w8a8(xs[i], p), W.linear_dgrad_w8(dys[i], p)))
    torch.cuda.synchronize()
    for i in range(2):
        for y, dx in got[i]:
            assert torch.equal(y, want[i][0]) and torch.equal(dx, want[i][1])


def test_refusals_on_the_device():
    import w4_gemm_amd as W
    rng = np.random.default_rng(60)
    n, k, e = 64, 512, 2
    p = W.W8Payload(*R.make_layer(rng, n, k, 16, dev()))
    gp = W.GroupedW8Payload(*R.make_layer(rng, n, k, 16, dev(), groups=e))
    x = R.make_rows(rng, 8, k, dev())
    offsets = torch.tensor([0, 3, 8], dtype=torch.int32, device=dev())
    with pytest.raises(TypeError):
        W.linear_fwd_w8a8(x.float(), p)
    with pytest.raises(ValueError):
        W.linear_fwd_w8a8(x[:, :256].contiguous(), p)
    with pytest.raises(ValueError):
        W.linear_fwd_w8a8(x.t().contiguous().t(), p)          # not row-major
    with pytest.raises(ValueError):
        W.linear_fwd_w8a8(x, p, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        W.linear_fwd_w8a8(x, p, out=torch.empty((8, n + 1), device=dev()))
    with pytest.raises(ValueError):
        W.linear_fwd_w8a8(x.cpu(), p)
    with pytest.raises(W.SqError, match="SQ_E_WORKSPACE"):
        W.linear_fwd_w8a8(x, p, workspace=torch.empty(16, dtype=torch.uint8, device=dev()))
    with pytest.raises(ValueError):
        W.linear_dgrad_w8(x, p)                               # dy is [M, N]
    with pytest.raises(TypeError):
        W.grouped_fwd_w8a8(x, offsets.long(), gp)
    with pytest.raises(ValueError):
        W.grouped_fwd_w8a8(x, offsets[:2].contiguous(), gp)
    with pytest.raises(ValueError):
        W.grouped_fwd_w8a8(x, offsets.cpu(), gp)
    with pytest.raises(W.SqError, match="SQ_E_ALIGN"):
        W.grouped_fwd_w8a8(x, torch.zeros(4, dtype=torch.int32, device=dev())[1:], gp)
    # no rows: nothing runs, the shapes are still checked
    assert W.linear_fwd_w8a8(x[:0], p).shape == (0, n)
    assert W.grouped_dgrad_w8(torch.empty((0, n), dtype=BF16, device=dev()), offsets, gp).shape == (0, k)
