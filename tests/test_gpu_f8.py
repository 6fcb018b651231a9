"""The 8-bit float mode (E4M3 codes, a power of two per block of 128) against its 64-bit reference:
quantizer, forward, input gradient, the gated block and its backward, for one layer and for experts."""
import numpy as np
import pytest
import torch

from tests import f8_reference as R
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DT = pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
ACTS = ("silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import w4_gemm_amd  # noqa: F401


def _gen(*seed):
    return torch.Generator(device=dev()).manual_seed(int(np.random.default_rng(seed).integers(1 << 30)))


def _workspace(nbytes):
    """A caller's workspace full of 0xFF (NaN codes and exponents), 256 guard bytes behind it."""
    return torch.full((nbytes + 256,), 255, dtype=torch.uint8, device=dev())


def _call(fn, size, *args, out, **kw):
    buf = _workspace(size)
    got = fn(*args, workspace=buf[:size], out=out, **kw)
    assert bool((buf[size:] == 255).all())
    return got


def _nan(m, n, dt):
    return torch.full((m, n), float("nan"), dtype=dt, device=dev())


def _forward(x, p, dt):
    import w4_gemm_amd as W
    return _call(W.linear_fwd_f8, W.fwd_f8_workspace_bytes(x.shape[0], p), x, p,
                 out=_nan(x.shape[0], p.n, dt))


def _gradient(dy, p, dt):
    import w4_gemm_amd as W
    return _call(W.linear_dgrad_f8, W.dgrad_f8_workspace_bytes(dy.shape[0], p), dy, p,
                 out=_nan(dy.shape[0], p.k, dt))


# ------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("n,k", [(1, 1), (1, 130), (127, 129), (128, 128), (129, 1), (300, 1000), (5, 4099),
                                 (257, 264), (2050, 7)])
@DT
def test_quantizer(n, k, dt):
    import w4_gemm_amd as W
    g = _gen(n, k)
    w = torch.randn(n, k, generator=g, device=dev()) * torch.exp(3 * torch.randn(n, 1, generator=g, device=dev()))
    w[:, k // 2] = 0.0
    w = w.to(dt)
    p, flags = W.quantize_weight_f8(w)
    codes, byte = R.quantize_weight(w)
    assert p.codes.shape == codes.shape and (p.n, p.k) == (n, k)
    assert torch.equal(p.codes.double(), codes)
    assert torch.equal(p.exps.int(), byte.int())
    assert int(flags[0]) == 0


def test_quantizer_at_the_borders():
    """Largest magnitudes at and next to 448 * 2^e, subnormal weights, ties, zero blocks, and the
    smallest exponent."""
    import w4_gemm_amd as W
    g = _gen(7)
    blocks = []
    for e in (-140, -126, -119, -118, -50, -1, 0, 1, 60, 119):
        for top in (448.0, np.nextafter(np.float32(448), np.float32(449)), np.nextafter(np.float32(448), np.float32(0)),
                    256.0, 511.0):
            v = torch.rand(128, 128, generator=g, device=dev(), dtype=torch.float64) * 2 - 1
            v *= torch.exp2(torch.randint(-20, 1, v.shape, generator=g, device=dev()).double())
            v[0, :64] = (torch.arange(64, device=dev()) + 0.5) / 512          # ties among the subnormal codes
            v = (v * float(top) * 2.0 ** e).float()
            v[5, 9] = float(np.float32(float(top) * 2.0 ** e))
            blocks.append(v)
    blocks.append(torch.zeros(128, 128, device=dev()))
    w = torch.cat(blocks, 1).contiguous()
    assert w.isfinite().all()
    p, flags = W.quantize_weight_f8(w)
    codes, byte = R.quantize_weight(w)
    assert torch.equal(p.codes.double(), codes) and torch.equal(p.exps.int(), byte.int())
    assert int(flags[0]) == 0 and int(p.exps[0, -1]) == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quantizer_flags_what_is_not_finite(bad):
    import w4_gemm_amd as W
    w = torch.ones(200, 300, device=dev())
    w[150, 299] = bad
    p, flags = W.quantize_weight_f8(w)
    assert int(flags[0]) == 1
    assert p.exps.tolist() == [[int(R.exponent_byte(torch.ones(1).double()))] * 3] * 1 + \
        [[int(R.exponent_byte(torch.ones(1).double()))] * 2 + [255]]
    assert torch.isnan(p.codes.float()).nonzero().tolist() == [[150, 299]]


# ------------------------------------------------------------------ one layer
FWD = [  # m, n, k
    (1, 1, 1), (1, 16, 128), (2, 33, 127), (1, 520, 6144), (3, 300, 2048), (15, 65, 769), (16, 512, 512),
    (17, 129, 1280), (31, 256, 255), (33, 48, 4096), (48, 96, 16384), (64, 512, 500), (65, 255, 768),
    (127, 257, 2311), (129, 1003, 640), (255, 64, 2), (257, 513, 513), (300, 260, 4352), (700, 1024, 896),
    (2, 24, 65536), (12, 40, 1023), (200, 7, 129), (1, 5000, 300), (9, 1, 40000),
]


@pytest.mark.parametrize("m,n,k", FWD)
@DT
def test_forward(m, n, k, dt):
    g = _gen(m, n, k)
    layer, x = R.make_layer(g, n, k), R.make_rows(g, m, k)
    R.check(_forward(x, layer.payload(), dt), *R.forward(x, layer, dt))


GRAD = [
    (1, 1, 1), (1, 63, 256), (2, 64, 511), (4, 65, 768), (16, 1, 1024), (16, 512, 512), (33, 200, 257),
    (64, 2049, 256), (127, 700, 1280), (129, 2051, 515), (130, 2048, 768), (257, 320, 2304), (300, 4099, 130),
    (1, 16384, 256), (3, 65537, 3), (7, 130, 5000),
]


@pytest.mark.parametrize("m,n,k", GRAD)
@DT
def test_gradient(m, n, k, dt):
    g = _gen(m, n, k)
    layer, dy = R.make_layer(g, n, k), R.make_rows(g, m, n, 1e-3)
    R.check(_gradient(dy, layer.payload(), dt), *R.gradient(dy, layer, dt))


@pytest.mark.parametrize("m,n,k", [(5, 70, 700), (40, 300, 1000), (130, 257, 384)])
@DT
def test_codes_of_all_exponents(m, n, k, dt):
    """Codes spread over all exponents, blocks whose powers of two differ by 2^20."""
    g = _gen(m, n, k, 1)
    layer = R.make_layer(g, n, k, wide=True)
    x = (R.make_rows(g, m, k).float() * torch.exp2(torch.randint(-30, 10, (m, k), generator=g, device=dev()).float())).bfloat16()
    R.check(_forward(x, layer.payload(), dt), *R.forward(x, layer, dt))
    dy = (R.make_rows(g, m, n).float() * torch.exp2(torch.randint(-30, 10, (m, n), generator=g, device=dev()).float())).bfloat16()
    R.check(_gradient(dy, layer.payload(), dt), *R.gradient(dy, layer, dt))


@pytest.mark.parametrize("scale", [2.0 ** -125, 2.0 ** -60, 2.0 ** 100])
@DT
def test_small_and_large_rows(scale, dt):
    """Rows near the ends of bf16's range: exponents reach their smallest byte and high ones."""
    g = _gen(3)
    m, n, k = 20, 130, 300
    layer = R.make_layer(g, n, k)
    x = (R.make_rows(g, m, k).float().clamp(-60, 60) * scale).bfloat16()
    y, tol, norm = R.forward(x, layer, dt)
    # results below the smallest normal may be flushed, in every block and in the end
    tol = tol + 4 * 2.0 ** -126
    R.check(_forward(x, layer.payload(), dt), y, tol)


def test_rows_that_are_not_finite():
    """inf or NaN anywhere gives a row of NaN and touches no other row."""
    g = _gen(4)
    m, n, k = 40, 200, 390
    layer, x = R.make_layer(g, n, k), R.make_rows(g, m, k)
    dy = R.make_rows(g, m, n)
    for dt in (F32, BF16):
        for call, a in ((_forward, x), (_gradient, dy)):
            clean = call(a, layer.payload(), dt)
            bad = a.clone()
            bad[3, 0], bad[17, a.shape[1] - 1], bad[38, 130] = float("nan"), float("inf"), float("-inf")
            got = call(bad, layer.payload(), dt)
            rows = torch.ones(m, dtype=torch.bool, device=dev())
            rows[[3, 17, 38]] = False
            assert torch.equal(got[rows], clean[rows])
            assert bool(torch.isnan(got[~rows]).all())


def test_zero_rows_and_padding():
    """Zero rows give zeros; what lies behind column K of the codes' rows takes no part, nor do row
    codes past N in the gradient."""
    g = _gen(5)
    layer = R.make_layer(g, 70, 200)
    x = R.make_rows(g, 9, 200)
    x[4] = 0
    for dt in (F32, BF16):
        assert bool((_forward(x, layer.payload(), dt)[4] == 0).all())
        dy = R.make_rows(g, 9, 70)
        dy[8] = 0
        assert bool((_gradient(dy, layer.payload(), dt)[8] == 0).all())


def test_gradient_is_that_of_the_layer():
    """dx against differences of the layer without the rows' rounding: <dx, v> for
    f(x) = <dy, x W^T>, which is linear, in 64 bits.  Q keeps each value to half a code step:
    2^-4 of it, or 2^-10 of the block's power of two, whose 448-fold is above the block's largest."""
    g = _gen(6)
    m, n, k = 40, 300, 515
    layer, dy = R.make_layer(g, n, k), R.make_rows(g, m, n, 1e-3)
    dx = _gradient(dy, layer.payload(), F32).double()
    _, tol, _ = R.gradient(dy, layer, F32)
    w = layer.value[:, :k]
    _, byte = R.quantize_rows(dy)
    half = torch.maximum(2.0 ** -4 * dy.double().abs(),
                         2.0 ** -10 * R.pow2(byte - 127).repeat_interleave(128, 1)[:, :n])
    x = torch.randn(m, k, generator=g, device=dev(), dtype=torch.float64)
    for _ in range(5):
        v = torch.randn(m, k, generator=g, device=dev(), dtype=torch.float64)
        f = lambda z: (dy.double() * (z @ w.t())).sum()   # noqa: E731
        diff = (f(x + v) - f(x - v)) / 2
        bound = ((tol + half @ w.abs()) * v.abs()).sum() + 1e-12 * (dy.double().abs() @ w.abs()).sum()
        assert abs(float((dx * v).sum() - diff)) <= float(bound)


# ------------------------------------------------------------------ gated block
def _gated(x, gate, up, act, dt):
    import w4_gemm_amd as W
    return _call(W.gated_fwd_f8, W.gated_fwd_f8_workspace_bytes(x.shape[0], gate), x, gate, up, act,
                 save=True, out=_nan(x.shape[0], gate.n, dt))


def _gated_backward(dh, g, u, gate, up, act, dt):
    import w4_gemm_amd as W
    return _call(W.gated_bwd_f8, W.gated_bwd_f8_workspace_bytes(dh.shape[0], gate), dh, g, u, gate, up, act,
                 out=_nan(dh.shape[0], gate.k, dt))


GATED = [(1, 1, 1), (1, 500, 640), (5, 33, 300), (16, 130, 1024), (17, 257, 128), (60, 64, 2050), (129, 200, 385),
         (300, 515, 260)]


@pytest.mark.parametrize("m,n,k", GATED)
@pytest.mark.parametrize("act", ACTS)
@DT
def test_gated_forward(m, n, k, act, dt):
    import w4_gemm_amd as W
    gen = _gen(m, n, k)
    gate, up, x = R.make_layer(gen, n, k), R.make_layer(gen, n, k), R.make_rows(gen, m, k)
    h, g, u = _gated(x, gate.payload(), up.payload(), act, dt)
    for got, want in zip((h, g, u), R.gated(x, gate, up, act, dt)):
        R.check(got, *want)
    # without saving: the same h
    assert torch.equal(W.gated_fwd_f8(x, gate.payload(), up.payload(), act, out_dtype=dt), h)


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 640, 500), (16, 130, 1024), (33, 257, 128), (129, 200, 385),
                                   (300, 515, 260), (4, 2050, 60)])
@pytest.mark.parametrize("act", ACTS)
@DT
def test_gated_backward(m, n, k, act, dt):
    import w4_gemm_amd as W
    gen = _gen(m, n, k)
    gate, up = R.make_layer(gen, n, k), R.make_layer(gen, n, k)
    dh = R.make_rows(gen, m, n, 1e-3)
    g, u = ((2 * torch.randn(m, n, generator=gen, device=dev())).bfloat16() for _ in range(2))
    got = _gated_backward(dh, g, u, gate.payload(), up.payload(), act, dt)
    for have, want in zip(got, R.gated_backward(dh, g, u, gate, up, act, dt)):
        R.check(have, *want)
    # dx alone: the same
    alone = W.gated_bwd_f8(dh, g, u, gate.payload(), up.payload(), act, out_dtype=dt, want_dgu=False)
    assert torch.equal(alone, got[0])


@pytest.mark.parametrize("act", ACTS)
def test_curves_over_their_range(act):
    """h and its gradients for g from -30 to 30 (past where the curves are flat), by a layer that
    hands its input through."""
    k = 128
    eye = R.Layer(torch.eye(k, dtype=torch.float64, device=dev()), torch.full((1, 1), 127, dtype=torch.int32, device=dev()), k)
    values = torch.tensor([s * m * 2.0 ** e for e in range(-6, 4) for m in (1.0, 1.25, 1.875) for s in (1, -1)]
                          + [0.0, 24.0, -24.0, 30.0, -30.0, -13.0, 13.0, -6.5])
    x = torch.zeros(1, k)
    x[0, :values.numel()] = values
    x = x.bfloat16().to(dev())
    h, g, u = _gated(x, eye.payload(), eye.payload(), act, F32)
    for have, want in zip((h, g, u), R.gated(x, eye, eye, act, F32)):
        R.check(have, *want)
    dh = torch.ones_like(x)
    for have, want in zip(_gated_backward(dh, g, u, eye.payload(), eye.payload(), act, F32),
                          R.gated_backward(dh, g, u, eye, eye, act, F32)):
        R.check(have, *want)


def test_gated_backward_is_the_gradient():
    """dg and du against central differences of h = act(g) u in 64 bits, and dx against those of the
    block without the rounding of dg and du (whose half steps bound what that moves)."""
    gen = _gen(8)
    m, n, k, step = 20, 150, 200, 1e-5
    gate, up = R.make_layer(gen, n, k), R.make_layer(gen, n, k)
    dh = R.make_rows(gen, m, n)
    g, u = ((1.5 * torch.randn(m, n, generator=gen, device=dev())).bfloat16() for _ in range(2))
    for act in ACTS:
        dx, dg, du = _gated_backward(dh, g, u, gate.payload(), up.payload(), act, F32)
        h = lambda a, b: R.curve(act, a)[0] * b   # noqa: E731
        gd, ud, d = g.double(), u.double(), dh.double()
        num_g = d * (h(gd + step, ud) - h(gd - step, ud)) / (2 * step)
        num_u = d * (h(gd, ud + step) - h(gd, ud - step)) / (2 * step)
        # differences: step^2 / 6 of a third derivative below 3, and 64-bit rounding over the step
        slack = d.abs() * (ud.abs() + gd.abs() + 1) * 1e-9
        R.check(dg, num_g, slack + (d * ud).abs() * R.curve_error(gd))
        R.check(du, num_u, slack + (d * gd).abs() * R.curve_error(gd))
        want = num_g @ gate.value[:, :k] + num_u @ up.value[:, :k]
        moved = 0.0
        for v, layer in ((num_g, gate), (num_u, up)):
            _, byte = R.quantize_rows(v)
            half = torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -9 * R.pow2(byte - 127).repeat_interleave(128, 1)[:, :n])
            moved = moved + half @ layer.value[:, :k].abs()
        assert bool(((dx.double() - want).abs() <= moved * 1.01 + 1e-9).all())


# ------------------------------------------------------------------ experts
COUNTS = {"uneven": [5, 0, 70, 1, 0, 40], "one": [37], "none": [0, 0, 0], "long": [300, 2, 129, 16],
          "many": [i % 3 for i in range(130)]}


def _stack(gen, e, n, k):
    import w4_gemm_amd as W
    layers = [R.make_layer(gen, n, k) for _ in range(e)]
    return layers, W.stack_payloads_f8([v.payload() for v in layers])


def _offsets(counts, lead):
    return torch.tensor(np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int32), device=dev())


@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("lead,tail", [(0, 0), (3, 5)])
@DT
def test_experts(name, lead, tail, dt):
    """Every product, expert by expert; rows outside the experts' ranges are left as they were in
    every output, whatever they hold."""
    import w4_gemm_amd as W
    counts = COUNTS[name]
    gen = _gen(len(counts), lead)
    n, k, e = (70, 130, len(counts)) if len(counts) > 20 else (257, 390, len(counts))
    m = lead + sum(counts) + tail
    gates, gate = _stack(gen, e, n, k)
    ups, up = _stack(gen, e, n, k)
    off = _offsets(counts, lead)
    x, dy = R.make_rows(gen, m, k), R.make_rows(gen, m, n, 1e-3)
    g, u = ((2 * torch.randn(m, n, generator=gen, device=dev())).bfloat16() for _ in range(2))
    used = torch.zeros(m, dtype=torch.bool, device=dev())
    used[lead:m - tail] = True
    for t in (x, dy, g, u):
        t[~used] = float("nan")
    mark = 7.0
    full = lambda c: torch.full((m, c), mark, dtype=dt, device=dev())   # noqa: E731
    if m == 0:
        assert W.grouped_fwd_f8(x, off, gate, out=full(n)).shape == (0, n)
        return
    y = _call(W.grouped_fwd_f8, W.grouped_fwd_f8_workspace_bytes(m, gate), x, off, gate, out=full(n))
    dx = _call(W.grouped_dgrad_f8, W.grouped_dgrad_f8_workspace_bytes(m, gate), dy, off, gate, out=full(k))
    h, gs, us = _call(W.grouped_gated_fwd_f8, W.grouped_gated_fwd_f8_workspace_bytes(m, gate), x, off, gate, up,
                      "gelu_tanh", save=True, out=full(n))
    bx, dg, du = _call(W.grouped_gated_bwd_f8, W.grouped_gated_bwd_f8_workspace_bytes(m, gate), dy, g, u, off, gate,
                       up, "silu", out=full(k))
    for out in (y, dx, h, bx):
        assert bool((out[~used] == mark).all())
    at = lead
    for i, c in enumerate(counts):
        if c and (len(counts) < 20 or i % 7 < 3):
            r = slice(at, at + c)
            R.check(y[r], *R.forward(x[r], gates[i], dt))
            R.check(dx[r], *R.gradient(dy[r], gates[i], dt))
            for have, want in zip((h[r], gs[r], us[r]), R.gated(x[r], gates[i], ups[i], "gelu_tanh", dt)):
                R.check(have, *want)
            for have, want in zip((bx[r], dg[r], du[r]), R.gated_backward(dy[r], g[r], u[r], gates[i], ups[i], "silu", dt)):
                R.check(have, *want)
        at += c


def test_rows_outside_keep_saved_and_gradient_outputs():
    """g, u, dg and du of rows outside the ranges are left as they were, through the C ABI (the
    wrapper allocates them)."""
    import w4_gemm_amd as W
    from w4_gemm_amd import _lib
    gen = _gen(9)
    m, n, k, e = 30, 140, 200, 2
    _, gate = _stack(gen, e, n, k)
    _, up = _stack(gen, e, n, k)
    off = torch.tensor([4, 9, 21], dtype=torch.int32, device=dev())
    x, dh = R.make_rows(gen, m, k), R.make_rows(gen, m, n)
    outs = [torch.full((m, n), 7.0, dtype=BF16, device=dev()) for _ in range(5)]
    dx = torch.full((m, k), 7.0, dtype=BF16, device=dev())
    ws = _workspace(max(W.grouped_gated_fwd_f8_workspace_bytes(m, gate), W.grouped_gated_bwd_f8_workspace_bytes(m, gate)))
    s = torch.cuda.current_stream().cuda_stream
    h, g, u, dg, du = outs
    assert _lib.sq_grouped_gated_fwd_f8(x.data_ptr(), m, off.data_ptr(), e, gate.abi(), up.abi(), 0, h.data_ptr(), 1,
                                        g.data_ptr(), u.data_ptr(), ws.data_ptr(), ws.numel(), s) == 0
    assert _lib.sq_grouped_gated_bwd_f8(dh.data_ptr(), g.data_ptr(), u.data_ptr(), m, off.data_ptr(), e, gate.abi(),
                                        up.abi(), 0, dx.data_ptr(), 1, dg.data_ptr(), du.data_ptr(), ws.data_ptr(),
                                        ws.numel(), s) == 0
    for t in (*outs, dx):
        assert bool((t[:4] == 7).all()) and bool((t[21:] == 7).all()) and not bool((t[4:21] == 7).all())


@DT
def test_offsets_out_of_range_stay_inside(dt):
    """Offsets are clamped into [0, m]: values below, above and falling ones touch nothing outside."""
    import w4_gemm_amd as W
    gen = _gen(10)
    m, n, k = 40, 100, 140
    layers, p = _stack(gen, 3, n, k)
    x, dy = R.make_rows(gen, m, k), R.make_rows(gen, m, n)
    off = torch.tensor([-5, 10, 25, 1000], dtype=torch.int32, device=dev())
    y, dx = W.grouped_fwd_f8(x, off, p, out_dtype=dt), W.grouped_dgrad_f8(dy, off, p, out_dtype=dt)
    for i, r in enumerate((slice(0, 10), slice(10, 25), slice(25, 40))):
        R.check(y[r], *R.forward(x[r], layers[i], dt))
        R.check(dx[r], *R.gradient(dy[r], layers[i], dt))
    wrong = torch.tensor([0, 30, 10, 2 ** 31 - 1], dtype=torch.int32, device=dev())
    size = W.grouped_fwd_f8_workspace_bytes(m, p)
    _call(W.grouped_fwd_f8, size, x, wrong, p, out=_nan(m, n, dt))
    torch.cuda.synchronize()


# ------------------------------------------------------------------ together
@DT
def test_mlp_block_forward_and_backward(dt):
    """Gated half, down projection, and the way back, as a training step runs them; every call is
    held to the reference on what the one before it returned."""
    import w4_gemm_amd as W
    gen = _gen(11)
    m, d, f = 70, 384, 515
    gate, up, down = R.make_layer(gen, f, d), R.make_layer(gen, f, d), R.make_layer(gen, d, f)
    pg, pu, pd = (v.payload() for v in (gate, up, down))
    x, dy = R.make_rows(gen, m, d), R.make_rows(gen, m, d, 1e-3)
    h, g, u = W.gated_fwd_f8(x, pg, pu, "silu", out_dtype=BF16, save=True)
    y = W.linear_fwd_f8(h, pd, out_dtype=dt)
    dh = W.linear_dgrad_f8(dy, pd, out_dtype=BF16)
    dx, dg, du = W.gated_bwd_f8(dh, g, u, pg, pu, "silu", out_dtype=dt)
    for have, want in zip((h, g, u), R.gated(x, gate, up, "silu", BF16)):
        R.check(have, *want)
    R.check(y, *R.forward(h, down, dt))
    R.check(dh, *R.gradient(dy, down, BF16))
    for have, want in zip((dx, dg, du), R.gated_backward(dh, g, u, gate, up, "silu", dt)):
        R.check(have, *want)


def test_mlp_block_of_experts_is_its_experts():
    """The same through stacked experts: bit for bit what each expert's rows give alone."""
    import w4_gemm_amd as W
    gen = _gen(12)
    counts = [33, 0, 20, 7]
    d, f, m = 260, 390, sum(counts)
    (gates, pg), (ups, pu), (downs, pd) = _stack(gen, 4, f, d), _stack(gen, 4, f, d), _stack(gen, 4, d, f)
    off = _offsets(counts, 0)
    x, dy = R.make_rows(gen, m, d), R.make_rows(gen, m, d, 1e-3)
    h, g, u = W.grouped_gated_fwd_f8(x, off, pg, pu, out_dtype=BF16, save=True)
    y = W.grouped_fwd_f8(h, off, pd, out_dtype=BF16)
    dh = W.grouped_dgrad_f8(dy, off, pd, out_dtype=BF16)
    dx, dg, du = W.grouped_gated_bwd_f8(dh, g, u, off, pg, pu, out_dtype=BF16)
    at = 0
    for i, c in enumerate(counts):
        r = slice(at, at + c)
        at += c
        if not c:
            continue
        for have, want in zip((h[r], g[r], u[r]), R.gated(x[r], gates[i], ups[i], "silu", BF16)):
            R.check(have, *want)
        R.check(y[r], *R.forward(h[r], downs[i], BF16))
        R.check(dh[r], *R.gradient(dy[r], downs[i], BF16))
        for have, want in zip((dx[r], dg[r], du[r]), R.gated_backward(dh[r], g[r], u[r], gates[i], ups[i], "silu", BF16)):
            R.check(have, *want)


# ------------------------------------------------------------------ streams, graphs, large
def test_same_bits_again_and_on_another_stream():
    import w4_gemm_amd as W
    gen = _gen(13)
    m, n, k = 150, 300, 1000
    gate, up = R.make_layer(gen, n, k).payload(), R.make_layer(gen, n, k).payload()
    x, dh = R.make_rows(gen, m, k), R.make_rows(gen, m, n)

    def all_of():
        h, g, u = W.gated_fwd_f8(x, gate, up, save=True, out_dtype=BF16)
        return [W.linear_fwd_f8(x, gate), W.linear_dgrad_f8(dh, gate, out_dtype=BF16), h, g, u,
                *W.gated_bwd_f8(dh, g, u, gate, up)]

    first = all_of()
    for a, b in zip(first, all_of()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = all_of()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [8, 200])
def test_captured_and_replayed(rows):
    """A captured training step through experts follows new rows and new offsets; two graphs share
    one workspace on one stream."""
    import w4_gemm_amd as W
    gen = _gen(14, rows)
    n, k, e = 260, 390, 5
    _, gate = _stack(gen, e, n, k)
    _, up = _stack(gen, e, n, k)
    x, dh = R.make_rows(gen, rows, k), R.make_rows(gen, rows, n)
    off = torch.zeros(e + 1, dtype=torch.int32, device=dev())
    ws = _workspace(max(W.grouped_gated_fwd_f8_workspace_bytes(rows, gate),
                        W.grouped_gated_bwd_f8_workspace_bytes(rows, gate)))
    h = torch.zeros(rows, n, dtype=BF16, device=dev())
    dx = torch.zeros(rows, k, device=dev())

    def fwd():
        return W.grouped_gated_fwd_f8(x, off, gate, up, save=True, workspace=ws, out=h)

    def bwd(g, u):
        return W.grouped_gated_bwd_f8(dh, g, u, off, gate, up, workspace=ws, out=dx)

    def set_inputs(seed):
        gs = _gen(15, seed)
        cuts = torch.sort(torch.randint(0, rows + 1, (e - 1,), generator=gs, device=dev()))[0]
        off.copy_(torch.cat([torch.zeros(1, device=dev()), cuts, torch.full((1,), rows, device=dev())]).int())
        x.copy_(R.make_rows(gs, rows, k))
        dh.copy_(R.make_rows(gs, rows, n))

    set_inputs(0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        bwd(*fwd()[1:])
    stream.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0], stream=stream):
        _, g, u = fwd()
    with torch.cuda.graph(graphs[1], stream=stream):
        _, dg, du = bwd(g, u)
    for seed in range(1, 5):
        set_inputs(seed)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (h, g, u, dx, dg, du)]
        want_f = [t.clone() for t in fwd()]
        want_b = [t.clone() for t in bwd(want_f[1], want_f[2])]
        torch.cuda.synchronize()
        for a, b in zip(got, want_f + want_b):
            assert torch.equal(a, b)


def test_results_past_two_to_the_31():
    """Results of more than 2^31 values: the last rows and the first ones."""
    import w4_gemm_amd as W
    gen = _gen(16)
    m, n, k = 70001, 32768, 128
    layer = R.make_layer(gen, n, k)
    x = R.make_rows(gen, m, k)
    y = W.linear_fwd_f8(x, layer.payload(), out_dtype=BF16)
    for r in (slice(0, 4), slice(m - 4, m)):
        R.check(y[r], *R.forward(x[r], layer, BF16))
    del y
    wide = R.make_layer(gen, k, n)
    dx = W.linear_dgrad_f8(x, wide.payload(), out_dtype=BF16)
    for r in (slice(0, 4), slice(m - 4, m)):
        R.check(dx[r], *R.gradient(x[r], wide, BF16))


def test_experts_past_two_to_the_31():
    """The last expert of a stack of more than 2^31 codes."""
    import w4_gemm_amd as W
    gen = _gen(17)
    n, k, e = 32768, 32768, 3
    last = R.make_layer(gen, 256, 256)
    p = W.GroupedF8Payload(torch.zeros((e, n, k), dtype=torch.uint8, device=dev()).view(torch.float8_e4m3fn),
                           torch.full((e, n // 128, k // 128), 127, dtype=torch.uint8, device=dev()), k)
    p.codes[2, n - 256:, k - 256:] = last.codes.float().to(torch.float8_e4m3fn)
    p.exps[2, n // 128 - 2:, k // 128 - 2:] = last.byte.to(torch.uint8)
    off = torch.tensor([0, 2, 2, 7], dtype=torch.int32, device=dev())
    x, dy = R.make_rows(gen, 7, 256), R.make_rows(gen, 7, 256)
    wide = lambda t, c: torch.cat([torch.zeros(7, c - 256, dtype=BF16, device=dev()), t], 1).contiguous()   # noqa: E731
    y = W.grouped_fwd_f8(wide(x, k), off, p)
    dx = W.grouped_dgrad_f8(wide(dy, n), off, p)
    assert bool((y[:2] == 0).all()) and bool((y[2:, :n - 256] == 0).all())
    R.check(y[2:, n - 256:].contiguous(), *R.forward(x[2:], last, F32))
    R.check(dx[2:, k - 256:].contiguous(), *R.gradient(dy[2:], last, F32))


def test_no_rows():
    import w4_gemm_amd as W
    gen = _gen(18)
    p = R.make_layer(gen, 20, 30).payload()
    x, dy = torch.zeros(0, 30, dtype=BF16, device=dev()), torch.zeros(0, 20, dtype=BF16, device=dev())
    assert W.linear_fwd_f8(x, p).shape == (0, 20) and W.linear_dgrad_f8(dy, p).shape == (0, 30)
    assert [t.shape for t in W.gated_fwd_f8(x, p, p, save=True)] == [(0, 20)] * 3
    assert [t.shape for t in W.gated_bwd_f8(dy, dy, dy, p, p)] == [(0, 30), (0, 20), (0, 20)]
