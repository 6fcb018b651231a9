"""Every form of the 8-bit float products against the 64-bit reference: tiles of 64 to 256 rows with
and without splits, the form that streams the codes, one layer and experts, and contractions of more
than 1024 blocks."""
import numpy as np
import pytest
import torch

from tests import f8_reference as R
from tests.f8_forms import FORMS
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4_gemm_amd  # noqa: F401


def _run(kind, x, g, u, payloads, off, act, dt):
    """The call with a workspace full of NaN codes that ends in guard bytes, and NaN results."""
    import w4_gemm_amd as W
    name = ("" if off is None else "grouped_") + {"fwd": "fwd_f8", "dgrad": "dgrad_f8"}.get(kind, kind + "_f8")
    call = getattr(W, "linear_" + name if off is None and kind in ("fwd", "dgrad") else name)
    size = getattr(W, name + "_workspace_bytes")(x.shape[0], payloads[0])
    ws = torch.full((size + 256,), 255, dtype=torch.uint8, device=dev())
    p = payloads[0]
    out = torch.full((x.shape[0], p.k if kind in ("dgrad", "gated_bwd") else p.n), float("nan"), dtype=dt, device=dev())
    args = ([x, g, u] if kind == "gated_bwd" else [x]) + ([] if off is None else [off]) + payloads
    kw = dict(workspace=ws[:size], out=out)
    if kind == "gated_fwd":
        kw.update(save=True, act=act)
    if kind == "gated_bwd":
        kw.update(act=act)
    got = call(*args, **kw)
    assert bool((ws[size:] == 255).all())
    return got if isinstance(got, tuple) else (got,)


def _want(kind, x, g, u, layers, act, dt):
    if kind == "fwd":
        return [R.forward(x, layers[0], dt)]
    if kind == "dgrad":
        return [R.gradient(x, layers[0], dt)]
    if kind == "gated_fwd":
        return R.gated(x, *layers, act, dt)
    return R.gated_backward(x, g, u, *layers, act, dt)


@pytest.mark.parametrize("kind,m,n,k,e,bits,rows,cols,splits", FORMS)
def test_form(kind, m, n, k, e, bits, rows, cols, splits):
    import w4_gemm_amd as W
    print(f"form {kind} m{m} n{n} k{k} e{e} {bits} {rows}x{cols} s{splits}", flush=True)
    rng = np.random.default_rng(m + n + k + e)
    gen = torch.Generator(device=dev()).manual_seed(int(rng.integers(1 << 30)))
    dt, act = (BF16 if bits == 16 else F32), ("silu", "gelu", "gelu_tanh")[int(rng.integers(3))]
    pairs = 2 if kind.startswith("gated") else 1
    layers = [[R.make_layer(gen, n, k) for _ in range(pairs)] for _ in range(e)]
    back = kind in ("dgrad", "gated_bwd")
    x = R.make_rows(gen, m, n if back else k, 1e-3 if back else 1.0)
    g, u = ((2 * torch.randn(m, n, generator=gen, device=dev())).bfloat16() for _ in range(2)) \
        if kind == "gated_bwd" else (None, None)
    if m > 40:   # a row that is not finite, in the middle of a tile
        x[m // 2, 0] = float("inf")
    if e == 1:
        payloads, off, cuts = [v.payload() for v in layers[0]], None, [0, m]
    else:
        payloads = [W.stack_payloads_f8([v[i].payload() for v in layers]) for i in range(pairs)]
        share = rng.exponential(size=e) + 0.05
        counts = rng.multinomial(m, share / share.sum())
        cuts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        off = torch.from_numpy(cuts).to(dev())
    got = _run(kind, x, g, u, payloads, off, act, dt)
    again = _run(kind, x, g, u, payloads, off, act, dt)
    for a, b in zip(got, again):
        assert torch.equal(a.view(torch.int16) if a.dtype == BF16 else a.view(torch.int32),
                           b.view(torch.int16) if b.dtype == BF16 else b.view(torch.int32))
    for i in range(e):
        r = torch.arange(int(cuts[i]), int(cuts[i + 1]), device=dev())
        if m > 40:
            if bool((r == m // 2).any()):
                assert bool(torch.isnan(got[0][m // 2]).all())
            r = r[r != m // 2]
        if not r.numel():
            continue
        want = _want(kind, x[r], None if g is None else g[r], None if u is None else u[r], layers[i], act, dt)
        for have, w in zip(got, want):
            R.check(have[r], *w)


@pytest.mark.parametrize("kind,m,n,k", [("fwd", 600, 24, 140000), ("fwd", 3, 40, 300000), ("dgrad", 200, 140000, 24),
                                        ("gated_fwd", 100, 20, 140000), ("gated_bwd", 100, 70000, 30)])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_contractions_of_more_than_1024_blocks(kind, m, n, k, dt):
    gen = torch.Generator(device=dev()).manual_seed(m + n + k)
    layers = [R.make_layer(gen, n, k) for _ in range(2 if kind.startswith("gated") else 1)]
    back = kind in ("dgrad", "gated_bwd")
    x = R.make_rows(gen, m, n if back else k, 1e-3 if back else 1.0)
    g, u = ((2 * torch.randn(m, n, generator=gen, device=dev())).bfloat16() for _ in range(2)) \
        if kind == "gated_bwd" else (None, None)
    got = _run(kind, x, g, u, [v.payload() for v in layers], None, "silu", dt)
    for have, w in zip(got, _want(kind, x, g, u, layers, "silu", dt)):
        R.check(have, *w)
