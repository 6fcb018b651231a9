"""The int8 mode's 8-bit products at the ends of their ranges, against the 64-bit reference."""
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


# 64-row tiles: whole (256 column blocks), in parts, in parts; 128-row tiles: whole (64 x 4 tiles)
LOW_HALF = [(1, 65536), (3, 256), (40, 1024), (8192, 1024)]


@pytest.mark.parametrize("m,k", LOW_HALF)
def test_low_half_of_the_longest_gradient_rows(m, k):
    """N = 131072, every low half and every code -128: the low halves' sum is 2^31, one past int32.
    Only rows below the absmax floor can do that (an ordinary row's largest value has low half 0):
    dy = 2^-108 (1 + 2^-7) gives d = 128 = 256 - 128 throughout, its negative d = -128."""
    import w4_gemm_amd as W
    n = 131072
    codes = torch.full((n, k), -128, dtype=torch.int8, device=dev())
    w = torch.ones(n, dtype=torch.float16, device=dev())
    kinds = torch.full((4, n), 2.0 ** -108 * (1 + 2.0 ** -7), dtype=BF16, device=dev())
    kinds[1] = -kinds[1]
    kinds[2, ::2] = 0.0                  # half the sum
    kinds[3, 5] = 1.0                    # an ordinary row
    d, _ = R.gradient_levels(kinds, w)
    assert bool((d[0] == 128).all()) and bool((d[1] == -128).all())
    # every block of 256 columns has the same codes, so the same result
    want, tol = R.gradient(kinds, codes[:, :256], w, None, None, F32)
    which = torch.arange(m, device=dev()) % 4
    dx = W.linear_dgrad_w8(kinds[which].contiguous(), W.W8Payload(codes, w, None, None),
                           out_dtype=F32)
    for block in dx.view(m, k // 256, 256).unbind(1):
        R.check(block, want[which], tol[which])


@pytest.mark.parametrize("m", [1, 3, 70])
@pytest.mark.parametrize("rank", [32, 64])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_longest_forward_rows_with_the_widest_factors(m, rank, dt):
    """K = 65536: a pre-phase workgroup of 16 waves, whose projection takes 64 * rank bytes of LDS each,
    16- and 32-row projection tiles."""
    import w4_gemm_amd as W
    rng = np.random.default_rng(m + rank)
    n, k = 40, 65536
    lay = R.make_layer(rng, n, k, rank, dev())
    x = R.make_rows(rng, m, k, dev())
    R.check(W.linear_fwd_w8a8(x, W.W8Payload(*lay), out_dtype=dt), *R.forward(x, *lay, dt))


def _heavy_rows(kind, m, n):
    g = torch.Generator(device=dev()).manual_seed(12)
    v = torch.randn(m, n, generator=g, device=dev())
    if kind == "student":        # t with 2 degrees of freedom: normal / sqrt(exponential)
        v = v / torch.empty_like(v).exponential_(generator=g).sqrt()
    elif kind == "column":
        v[:, 7] *= 1000.0
    elif kind == "softmax":
        v = torch.softmax(2.0 * v, 1)
        v[torch.arange(m), torch.randint(n, (m,), generator=g, device=dev())] -= 1.0
    return (1e-2 * v).bfloat16()


@pytest.mark.parametrize("kind", ["gauss", "student", "column", "softmax"])
@pytest.mark.parametrize("n", [1000, 4096, 16384])
def test_gradient_of_heavy_tailed_rows(kind, n):
    """dx against dy W_hat itself, not against the definition that holds the 16-bit rows: each element
    within the step's worst case, and a row's error near what independent roundings give, uniform over
    a step of max / 32512 (variance step^2 / 12 each): max / 32512 sqrt(n / 12) / |v| of the norm of
    dx.  Norms over 1024 columns of a random W_hat scatter by 1 / sqrt(512) = 4.4 % (squared), so 1.25
    is more than five of their standard deviations; 1e-6 stands for the fp32 steps."""
    import w4_gemm_amd as W
    m, k = 32, 1024
    codes, w, _, _ = R.make_layer(np.random.default_rng(n), n, k, 0, dev())
    dy = _heavy_rows(kind, m, n)
    dx = W.linear_dgrad_w8(dy, W.W8Payload(codes, w, None, None)).double()
    h = R.sylvester(dev()) / 16.0
    c = codes.double()
    what = ((c * w.double()[:, None]).view(n, -1, 256) @ h).view(n, k)
    want = dy.double() @ what
    v = dy.double() * w.double()
    step = v.abs().amax(1, keepdim=True) / 32512.0
    _, tol = R.gradient(dy, codes, w, None, None, F32)
    worst = ((0.5 * step + 2.0 ** -23 * v.abs().amax(1, keepdim=True)) * c.abs().sum(0)) \
        .view(m, -1, 256).sum(2, keepdim=True).expand(-1, -1, 256).reshape(m, k) / 16.0
    R.check(dx, want, tol + worst)
    off = (dx - want).norm(dim=1) / want.norm(dim=1)
    expect = step[:, 0] * (n / 12.0) ** 0.5 / v.norm(dim=1)
    print(f"{kind} n {n}: median {float(off.median()):.2e}, expected {float(expect.median()):.2e}")
    assert bool((off <= 1.25 * expect + 1e-6).all())
