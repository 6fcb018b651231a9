"""How the 8-bit float products sum, against the bounds that sq.h states: groups of eight products
whose largest codes lie opposite zeros and subnormals, and the distance in norm of bf16 results."""
import math

import numpy as np
import pytest
import torch

from tests import f8_reference as R
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DT = pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4_gemm_amd  # noqa: F401


def _gen(*seed):
    return torch.Generator(device=dev()).manual_seed(int(np.random.default_rng(seed).integers(1 << 30)))


def _counted(codes, byte, rows):
    """Magnitudes as the largest of a group is found by: subnormal codes at 2^-6, zeros at zero."""
    c = codes.abs()
    c = torch.where(c > 0, c.clamp(min=2.0 ** -6), c)
    return R.spread_rows(c, byte) if rows else R.spread_weight(c, byte)


def _bound(rows, weight, value, dt):
    """What sq.h allows: rows (codes, bytes), weight magnitudes as counted and weight values [N, K]."""
    tol = (128 + rows[1].shape[1]) * 2.0 ** -23 * (R.spread_rows(*rows).abs() @ value.abs().t())
    return tol + (R.group_bound(_counted(*rows, True), weight) if dt == BF16 else 0.0)


@pytest.mark.parametrize("m", [1, 40, 300])
@pytest.mark.parametrize("opposite", [0.0, 2.0 ** -9, -7 * 2.0 ** -9, 2.0 ** -6])
@DT
def test_large_codes_opposite_small_ones(m, opposite, dt):
    """In every group one code of 448 lies opposite a zero, a subnormal or the smallest normal code, and
    the other seven products are between 2^-12 and 2."""
    import w4_gemm_amd as W
    gen = _gen(m, 1)
    n = k = 256
    at = torch.arange(0, k, 8, device=dev()) + torch.randint(0, 8, (k // 8,), generator=gen, device=dev())
    small = lambda rows, hi: (torch.exp2(torch.randint(-6, hi, (rows, k), generator=gen, device=dev()).float())   # noqa: E731
                              * torch.where(torch.rand(rows, k, generator=gen, device=dev()) < 0.5, -1.0, 1.0))
    x, codes = small(m, 1), small(n, 2)
    x[:, at] = 448.0
    codes[:, at] = opposite
    if m > 8:
        x[3:7] = x[3:7].abs()            # without cancellation
    codes[5:20] = codes[5:20].abs()
    x, codes, one = x.bfloat16(), codes.double(), torch.full((2, 2), 127, dtype=torch.int32, device=dev())
    rows = R.quantize_rows(x)
    layer, turned = R.Layer(codes, one, k), R.Layer(codes.t().contiguous(), one, n)
    want = R.spread_rows(*rows) @ layer.value.t()
    tol = _bound(rows, _counted(codes, one, False), layer.value, dt)
    R.check(W.linear_fwd_f8(x, layer.payload(), out_dtype=dt), want, tol)
    R.check(W.linear_dgrad_f8(x, turned.payload(), out_dtype=dt), want, tol)


@pytest.mark.parametrize("m", [1, 40])
@DT
def test_cancelling_products_of_a_subnormal_code(m, dt):
    """448 * 2^-9 and its negative cancel; the other six products of 2^-12 are below 2^-13 of
    2^8 * 2^-6.  They are more than 7 * 2^-13 of the largest product's own magnitude, so the bound has
    to count the subnormal code as it does; fp32 results keep them."""
    import w4_gemm_amd as W
    x, codes = torch.zeros(m, 128, device=dev()), torch.zeros(16, 128, device=dev())
    x[:, 0], x[:, 1], x[:, 2:8] = 448.0, -448.0, 2.0 ** -6
    codes[:, :2], codes[:, 2:8] = 2.0 ** -9, 2.0 ** -6
    layer = R.Layer(codes.double(), torch.full((1, 1), 127, dtype=torch.int32, device=dev()), 128)
    y = W.linear_fwd_f8(x.bfloat16(), layer.payload(), out_dtype=dt).double()
    want = 6 * 2.0 ** -12
    if dt == F32:
        assert bool((y == want).all())
    else:
        assert bool(((y - want).abs() <= 7 * 2.0 ** -13 * 448 * 2.0 ** -6).all())


# few rows, split, and unsplit tiles of 64 to 256 rows; contractions of up to 512 blocks
@pytest.mark.parametrize("m,n,k", [(3, 2048, 6144), (8, 4096, 65536), (40, 1024, 16384), (300, 512, 65536),
                                   (1500, 2048, 6144), (4000, 2048, 4096)])
def test_norm_of_bf16_results(m, n, k):
    """The distance of bf16 results from 64 bits in norm, for the forward and the gradient.  Rounding
    is off by at most 2^-8 of each value.  In a group of eight, seven products lose less than 2^-13 of
    its largest L, each with the sign of its product, which for Gaussian codes is either: a walk of
    steps 2^-13 L, whose norm is sqrt(7 sum L^2) 2^-13, taken twice.  A block of 128 left out would
    move the norm by sqrt(1 / blocks): 14 % at K = 6144, 4.4 % at 65536, against the 0.5 % here."""
    import w4_gemm_amd as W
    gen = _gen(m, n, k)
    layer = R.make_layer(gen, n, k)
    x = torch.randn(m, k, generator=gen, device=dev()).bfloat16()
    y = W.linear_fwd_f8(x, layer.payload(), out_dtype=BF16)
    _norm_check(y, R.quantize_rows(x), layer.value, layer.high)
    turned = R.make_layer(gen, k, n)
    dx = W.linear_dgrad_f8(x, turned.payload(), out_dtype=BF16)
    _norm_check(dx, R.quantize_rows(x), *R.transposed(turned))


def _norm_check(got, rows, value, high):
    want = R.spread_rows(*rows) @ value.t()
    # sum over the groups of L^2, from a sample of results, for all of them
    rs = slice(0, min(64, want.shape[0]))
    cs = slice(0, min(64, want.shape[1]))
    a = R.spread_rows(*rows, 2.0 ** -6)[rs].view(-1, 1, value.shape[1] // 8, 8)
    b = high[cs].view(1, -1, value.shape[1] // 8, 8)
    tops = 0.0
    for i in range(0, a.shape[0], 4):
        tops = tops + float((a[i:i + 4] * b).amax(3).square().sum())
    tops *= want.numel() / (a.shape[0] * b.shape[1])
    bound = 2.0 ** -8 * float(want.norm()) + 2.0 * 2.0 ** -13 * math.sqrt(7.0 * tops)
    assert bound < 0.01 * float(want.norm())
    assert float((got.double() - want).norm()) <= bound
