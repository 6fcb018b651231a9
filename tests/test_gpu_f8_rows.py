"""The rounding of rows on their way into the 8-bit float products, bit for bit: through layers that hand
their input on (a one per row, powers of two per block) every result is one rounded value.  And what lies
beside a layer's codes in memory: padding columns and other experts."""
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


def _unit(n, shift=None):
    """The layer of size n x n that multiplies block b of its input by 2^shift[b]."""
    b = R.blocks(n)
    byte = torch.full((b, b), 127, dtype=torch.int32, device=dev())
    if shift is not None:
        byte += torch.diag(torch.tensor(shift, dtype=torch.int32, device=dev()))
    codes = torch.zeros(n, 128 * b, dtype=torch.float64, device=dev())
    codes[torch.arange(n), torch.arange(n)] = 1.0
    return R.Layer(codes, byte, n)


def _zero(n):
    layer = _unit(n)
    layer.codes.zero_()
    return layer


def _border_rows(m, n):
    """bf16 rows whose blocks are: ordinary; with a largest value at, above and below 448 * 2^e; with
    ties and subnormal codes; of bf16's smallest values (exponent byte 0); zero; near bf16's largest.
    And a power of two per block that brings each result into range."""
    gen = _gen(m, n)
    v = torch.randn(m, n, generator=gen, device=dev(), dtype=torch.float64)
    shift = []
    for b in range(R.blocks(n)):
        c = slice(128 * b, min(n, 128 * b + 128))
        w, kind = v[:, c], b % 6
        top = torch.tensor([448.0, 450.0, 446.0, 256.0, 510.0, 512.0], device=dev(), dtype=torch.float64)
        if kind == 1:
            w.mul_(30).clamp_(-200, 200)
            w[:, -1] = top[torch.randint(0, 6, (m,), generator=gen, device=dev())]
            w.mul_(torch.exp2(torch.randint(-40, 40, (m, 1), generator=gen, device=dev()).double()))
        elif kind == 2:
            # halves of the steps of subnormal and of normal codes, below a largest value of 448
            w.copy_((torch.randint(0, 64, w.shape, generator=gen, device=dev()) + 0.5) * torch.exp2(
                torch.randint(-10, 3, w.shape, generator=gen, device=dev()).double()))
            w[:, 0] = -448.0
        elif kind == 3:
            w.copy_(torch.randint(-200, 200, w.shape, generator=gen, device=dev()).double() * 2.0 ** -133)
            if m > 1:
                w[1] = w[1].sign() * 2.0 ** -133
        elif kind == 4:
            w[::2] = 0.0
        elif kind == 5:
            w.mul_(2.0 ** 124).clamp_(-3.0e38, 3.0e38)
        shift.append({3: 60, 5: -20}.get(kind, 0))
    return v.bfloat16(), shift


def _want(rows, shift):
    """Rows rounded to codes times their powers of two, in 64 bits, with each block's power of two."""
    q = R.spread_rows(*R.quantize_rows(rows))
    return (q * torch.exp2(torch.tensor(shift, device=dev()).double()).repeat_interleave(128))[:, :rows.shape[1]]


# 1 and 16 rows are rounded in the products' own launch, more in a pass of their own
@pytest.mark.parametrize("m,n", [(1, 768), (16, 896), (16, 771), (1, 1), (5, 130), (40, 896), (300, 771), (33, 129)])
@DT
def test_rows_of_the_forward_and_the_gradient(m, n, dt):
    import w4_gemm_amd as W
    x, shift = _border_rows(m, n)
    want = _want(x, shift)
    p = _unit(n, shift).payload()
    assert torch.equal(W.linear_fwd_f8(x, p, out_dtype=dt).double(), want)
    assert torch.equal(W.linear_dgrad_f8(x, p, out_dtype=dt).double(), want)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("m,n", [(1, 512), (7, 515), (300, 640)])
@DT
def test_rows_of_the_gated_backward(m, n, act, dt):
    """With g = 2^20 the slope is 1 and the value g, so dg = dh u and du = dh 2^20, both exact in fp32
    (products of two bf16 values), and each is rounded once to codes and once to bf16."""
    import w4_gemm_amd as W
    gen = _gen(m, n, 3)
    dh, _ = _border_rows(m, 256)
    dh = dh.repeat(1, R.blocks(n) // 2 + 1)[:, :n].contiguous()
    u = (torch.randn(m, n, generator=gen, device=dev()) * torch.exp2(
        torch.randint(-8, 8, (m, n), generator=gen, device=dev()).float())).bfloat16()
    g = torch.full((m, n), 2.0 ** 20, dtype=BF16, device=dev())
    one, none = _unit(n).payload(), _zero(n).payload()
    ds = [dh.double() * u.double(), dh.double() * 2.0 ** 20]
    for i, pair in enumerate(((one, none), (none, one))):
        dx, dg, du = W.gated_bwd_f8(dh, g, u, *pair, act, out_dtype=dt)
        assert torch.equal(dx.double(), _want(ds[i], [0] * R.blocks(n)))
        assert torch.equal(dg, ds[0].bfloat16()) and torch.equal(du, ds[1].bfloat16())


@pytest.mark.parametrize("m", [3, 40, 600])
@DT
def test_padding_columns_stay_out_of_the_gradient(m, dt):
    """Codes behind column K lie in the gradient's last tile: whatever they hold, NaN among it, dx is the
    same (the forward needs zeros there)."""
    import w4_gemm_amd as W
    gen = _gen(m, 5)
    n, k = 300, 200
    layer, dy = R.make_layer(gen, n, k), R.make_rows(gen, m, n)
    g, u = ((2 * torch.randn(m, n, generator=gen, device=dev())).bfloat16() for _ in range(2))
    clean, dirty = layer.payload(), layer.payload()
    bits = torch.randint(0, 256, (n, 256 - k), generator=gen, device=dev(), dtype=torch.int32).to(torch.uint8)
    bits[::3, ::5] = 0x7F
    dirty.codes.view(torch.uint8)[:, k:] = bits
    assert torch.equal(W.linear_dgrad_f8(dy, clean, out_dtype=dt), W.linear_dgrad_f8(dy, dirty, out_dtype=dt))
    for a, b in zip(W.gated_bwd_f8(dy, g, u, clean, clean, out_dtype=dt), W.gated_bwd_f8(dy, g, u, dirty, dirty, out_dtype=dt)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("counts", [[3, 2, 4], [40, 30, 50], [300, 1, 290]])
@DT
def test_other_experts_stay_out(counts, dt):
    """The codes behind an expert's last row are the next expert's: with those NaN, and with NaN rows
    of the same call beside it, its results are the same."""
    import w4_gemm_amd as W
    gen = _gen(sum(counts), 6)
    n, k, m = 70, 330, sum(counts)
    clean = W.stack_payloads_f8([R.make_layer(gen, n, k).payload() for _ in counts])
    dirty = W.GroupedF8Payload(clean.codes.clone(), clean.exps.clone(), k)
    dirty.codes.view(torch.uint8)[1] = 0x7F
    dirty.exps[1] = 255
    cuts = np.concatenate([[0], np.cumsum(counts)])
    off = torch.from_numpy(cuts.astype(np.int32)).to(dev())
    x, dy = R.make_rows(gen, m, k), R.make_rows(gen, m, n)
    g, u = ((2 * torch.randn(m, n, generator=gen, device=dev())).bfloat16() for _ in range(2))

    def all_of(p):
        return (W.grouped_fwd_f8(x, off, p, out_dtype=dt), W.grouped_dgrad_f8(dy, off, p, out_dtype=dt),
                *W.grouped_gated_fwd_f8(x, off, p, p, save=True, out_dtype=dt),
                *W.grouped_gated_bwd_f8(dy, g, u, off, p, p, out_dtype=dt))

    want = all_of(clean)
    middle = slice(cuts[1], cuts[2])
    for t in (x, dy, g, u):
        t[middle] = float("nan")
    for a, b in zip(all_of(dirty), want):
        assert torch.equal(a[:cuts[1]], b[:cuts[1]]) and torch.equal(a[cuts[2]:], b[cuts[2]:])
        assert bool(a[middle].isnan().all())
