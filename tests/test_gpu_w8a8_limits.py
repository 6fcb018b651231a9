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
