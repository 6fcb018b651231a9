"""The 8-bit float products where the contraction's loop comes round several times without a split, with
every curve, and the split forms of the largest tiles, against the 64-bit reference."""
import numpy as np
import pytest
import torch

from tests import f8_reference as R
from tests.f8_deep_forms import DEEP, SPLIT, with_curves
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4_gemm_amd  # noqa: F401


def _cuts(m, e, rows):
    """Experts' row ranges: a whole tile and five rows, an expert without rows (of four), the others,
    and one that ends two rows short of a tile."""
    if e < 3:
        return np.array([0, m] if e == 1 else [0, rows + 5, m], np.int32)
    counts = [0] * e
    counts[0] = rows + 5
    counts[-1] = min(rows - 2, m - counts[0])
    left, middle = m - counts[0] - counts[-1], list(range(2, e - 1)) or [1]
    for i in middle:
        counts[i] = left // len(middle)
    counts[middle[0]] += left - sum(counts[i] for i in middle)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _run(kind, a, g, u, payloads, off, act, dt):
    """The call with a workspace full of NaN codes that ends in guard bytes, and NaN results."""
    import w4_gemm_amd as W
    name = ("" if off is None else "grouped_") + kind + "_f8"
    call = getattr(W, "linear_" + name if off is None and kind in ("fwd", "dgrad") else name)
    size = getattr(W, name + "_workspace_bytes")(a.shape[0], payloads[0])
    ws = torch.full((size + 256,), 255, dtype=torch.uint8, device=dev())
    p = payloads[0]
    out = torch.full((a.shape[0], p.k if kind in ("dgrad", "gated_bwd") else p.n), float("nan"), dtype=dt, device=dev())
    kw = {"gated_fwd": dict(save=True, act=act), "gated_bwd": dict(act=act)}.get(kind, {})
    got = call(a, *([g, u] if kind == "gated_bwd" else []), *([] if off is None else [off]), *payloads,
               workspace=ws[:size], out=out, **kw)
    assert bool((ws[size:] == 255).all())
    return got if isinstance(got, tuple) else (got,)


def _want(kind, a, g, u, layers, act, dt):
    if kind in ("fwd", "dgrad"):
        return [(R.forward if kind == "fwd" else R.gradient)(a, layers[0], dt)]
    if kind == "gated_fwd":
        return R.gated(a, *layers, act, dt)
    return R.gated_backward(a, g, u, *layers, act, dt)


@pytest.mark.parametrize("kind,m,n,k,e,bits,rows,cols,splits,act", with_curves(DEEP + SPLIT))
def test_form(kind, m, n, k, e, bits, rows, cols, splits, act):
    import w4_gemm_amd as W
    print(f"form {kind} m{m} n{n} k{k} e{e} {bits} {rows}x{cols} s{splits} {act}", flush=True)
    gen = torch.Generator(device=dev()).manual_seed(m + n + k + e)
    dt = BF16 if bits == 16 else F32
    pairs = 2 if kind.startswith("gated") else 1
    layers = [[R.make_layer(gen, n, k) for _ in range(pairs)] for _ in range(e)]
    back = kind in ("dgrad", "gated_bwd")
    a = R.make_rows(gen, m, n if back else k, 1e-3 if back else 1.0)
    g, u = ((2 * torch.randn(m, n, generator=gen, device=dev())).bfloat16() for _ in range(2)) \
        if kind == "gated_bwd" else (None, None)
    cuts = _cuts(m, e, rows)
    if e == 1:
        payloads, off = [v.payload() for v in layers[0]], None
    else:
        payloads = [W.stack_payloads_f8([v[i].payload() for v in layers]) for i in range(pairs)]
        off = torch.from_numpy(cuts).to(dev())
    got = _run(kind, a, g, u, payloads, off, act, dt)
    again = _run(kind, a, g, u, payloads, off, act, dt)
    for x, y in zip(got, again):
        assert torch.equal(x, y)
    for i in range(e):
        r = slice(int(cuts[i]), int(cuts[i + 1]))
        if r.start == r.stop:
            continue
        want = _want(kind, a[r], None if g is None else g[r], None if u is None else u[r], layers[i], act, dt)
        for have, w in zip(got, want):
            R.check(have[r], *w)
