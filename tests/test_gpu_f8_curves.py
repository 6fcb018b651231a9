"""The gated block's curves and their gradients at the ends of bf16's range: a finite gradient
stays finite whatever its factors are."""
import pytest
import torch

from tests import f8_reference as R
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
ACTS = ("silu", "gelu", "gelu_tanh")
TOP = float(torch.finfo(BF16).max)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4_gemm_amd  # noqa: F401


def _layers(seed, n, k):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return g, R.make_layer(g, n, k), R.make_layer(g, n, k)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_gradient_of_large_projections(act, dt):
    """Where |g| is large the slope is 0 or 1 and the value 0 or g: dg is dh u or 0, du dh g or 0.
    Products of two bf16 values are exact in fp32, so the rows that are rounded are known exactly."""
    import w4_gemm_amd as W
    n, k = 130, 70
    gen, gate, up = _layers(21, n, k)
    sizes = [20.0, 1e4, 2.0 ** 31, 2.0 ** 63, 2.0 ** 64, 1.9e19, 2.0 ** 65, 1e30, 2.0 ** 126, TOP]
    m = 2 * len(sizes)
    g = torch.tensor([s * v for v in sizes for s in (1, -1)]).to(BF16).to(dev())[:, None].expand(m, n).contiguous()
    dh = R.make_rows(gen, m, n).float().clamp(-100, 100).mul(2.0 ** -60).bfloat16()
    u = torch.randn(m, n, generator=gen, device=dev()).bfloat16()
    on = (g > 0).double()
    ds = [dh.double() * u.double() * on, dh.double() * g.double() * on]
    if act == "silu":
        # at 20 its curve is not flat yet: 20 e^-20 is 7 steps of 2^-24 and more
        ds = [torch.where(g.abs() > 20, d, torch.nan) for d in ds]
    dx, dg, du = W.gated_bwd_f8(dh, g, u, gate.payload(), up.payload(), act, out_dtype=dt)
    known = slice(2, None) if act == "silu" else slice(0, None)
    for have, want in zip((dg, du), ds):
        R.check(have[known], want[known], torch.zeros_like(want[known]) + 1e-44)
    pairs = [(R.quantize_rows(d[known]), *R.transposed(v)) for d, v in zip(ds, (gate, up))]
    want, tol, _ = R.contract(pairs, dt)
    R.check(dx[known], want, tol)
    assert bool(dx.isfinite().all())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_forward_of_large_projections(act, dt):
    """h is g u or 0 there, through layers that hand their input through (k values of a power of two)."""
    import w4_gemm_amd as W
    k = 128
    eye = R.Layer(torch.eye(k, dtype=torch.float64, device=dev()),
                  torch.full((1, 1), 127, dtype=torch.int32, device=dev()), k)
    small = R.Layer(eye.codes, torch.full((1, 1), 7, dtype=torch.int32, device=dev()), k)   # 2^-120
    values = [s * 2.0 ** e for e in (5, 31, 63, 64, 65, 100, 118, 120) for s in (1, -1)]
    x = torch.zeros(len(values), k)
    for i, v in enumerate(values):
        x[i, 7 * i] = v
    h = W.gated_fwd_f8(x.bfloat16().to(dev()), eye.payload(), small.payload(), act, out_dtype=dt)
    xd = x.double().to(dev())
    want = xd * (xd > 0) * (xd * 2.0 ** -120)
    # 32 is past the flat part's start in fp32: 32 e^-32 is below 2^-40
    R.check(h, want, 2.0 ** -40 * (xd * xd * 2.0 ** -120) + 1e-44)
    assert bool(h.isfinite().all())


@pytest.mark.parametrize("act,low", [("silu", -30.0), ("gelu", -6.0), ("gelu_tanh", -6.0)])
def test_gradient_where_its_first_factors_overflow(act, low):
    """dh u past fp32's range with a slope that brings dg back into it.  fp32 holds the slope to a
    few roundings of the exponential's argument (43, 18 and 25 here, each step of the polynomials
    adding one): below 256 of 2^-24."""
    import w4_gemm_amd as W
    m, n, k = 9, 140, 60
    gen, gate, up = _layers(22, n, k)
    rnd = lambda: (1 + torch.rand(m, n, generator=gen, device=dev())) * torch.where(   # noqa: E731
        torch.rand(m, n, generator=gen, device=dev()) < 0.5, -1.0, 1.0)
    dh, u = (rnd() * 2.0 ** 69).bfloat16(), (rnd() * 2.0 ** 68).bfloat16()
    u[:, ::3] = (u[:, ::3].float() * 2.0 ** -68).bfloat16()     # ordinary ones among them
    g = torch.full((m, n), low, dtype=BF16, device=dev())
    g[:, 1::5] = -500.0                                          # slope 0 in fp32
    dx, dg, du = W.gated_bwd_f8(dh, g, u, gate.payload(), up.payload(), act)
    v, slope = R.curve(act, g.double())
    want = dh.double() * u.double() * slope
    flat = g == -500
    assert bool((dg[flat] == 0).all()) and bool((du[flat] == 0).all())
    R.check(torch.where(flat, 0, dg), torch.where(flat, 0.0, want), 2.0 ** -16 * want.abs() + 1e-44)
    R.check(torch.where(flat, 0, du), torch.where(flat, 0.0, dh.double() * v), 2.0 ** -16 * (dh.double() * v).abs() + 1e-44)
    assert bool(dx.isfinite().all())
    # a gradient that does not fit is infinite, and one of its factors that is not finite is kept
    dh[4, 5], g[4, 5], u[4, 5] = 2.0 ** 100, 3.0, 2.0 ** 100
    dh[7, 9] = float("inf")
    dx, dg, du = W.gated_bwd_f8(dh, g, u, gate.payload(), up.payload(), act)
    assert bool(dg[4, 5].isinf()) and not bool(dg[7, 9].isfinite())
    good = torch.ones(m, dtype=torch.bool, device=dev())
    good[[4, 7]] = False
    assert bool(dx[good].isfinite().all()) and bool(dx[~good].isnan().all())
