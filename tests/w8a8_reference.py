"""The int8 mode's 8-bit forward and input gradient in 64 bits (torch float64 / int64), written
from the definition in include/sq.h, with a bound on the error of the library's arithmetic.

The integers q and d and the scales s and t are part of the definition and must be met exactly,
so the bounds count only what comes after them:

forward      the integer sum is exact; its conversion and two scale products round three times
             (3 * 2^-24 of the term);
gradient     hi and lo sums convert once each, their sum rounds once, eight butterfly stages and
             one product follow: 12 * 2^-24 of the sum of magnitudes that meet in an output;
rank-r term  t is an fp32 sum of K (N) exact products: (K + 64) * 2^-24 of the sum of their
             magnitudes (twice that, as the matrix unit may truncate instead of rounding), is held
             as bf16 hi + lo (2^-16 of t), and is used in 2r more fp32 steps;
bf16 output  2^-8 of the value.
"""
import numpy as np
import torch

U = 2.0 ** -24


def sylvester(device):
    h = torch.ones(1, 1, dtype=torch.float64, device=device)
    for _ in range(8):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
    return h


def f32(t):
    return t.to(torch.float32).to(torch.float64)


def token_levels(x):
    """(q, s) of each row of bf16 x as float64; rows that are not finite get q = 0, s = NaN."""
    m, k = x.shape
    fin = torch.isfinite(x).all(1)
    b = torch.where(fin[:, None], x, torch.zeros_like(x)).double().view(m, k // 256, 256)
    e = torch.frexp(b.abs().amax(2)).exponent.clamp(min=-125).long()[:, :, None]
    two = lambda p: ((p + 1023) << 52).view(torch.float64)          # noqa: E731
    sums = torch.trunc(b * two(23 - e)) @ sylvester(x.device)       # integers below 2^31
    return _levels(f32(f32(sums) * two(e - 27)).view(m, k), 127.0, fin)


def _levels(v, top, fin):
    a = v.abs().amax(1, keepdim=True).clamp(min=2.0 ** -100)
    q = torch.round(f32(v * f32(top / a)))
    s = f32(a / top)
    return q, torch.where(fin[:, None], s, torch.full_like(s, float("nan")))


def gradient_levels(dy, w):
    """(d, t) of each row of dy (bf16) times the column scales w."""
    v = f32(dy.double() * w.double())
    fin = torch.isfinite(v).all(1)
    return _levels(torch.where(fin[:, None], v, torch.zeros_like(v)), 32512.0, fin)


def _low(a, first, second, tol):
    """The rank-r term of rows a and its error bound, added to tol."""
    if first is None:
        return 0.0
    f, s = first.double(), second.double()
    t = a.double() @ f
    mag = a.double().abs() @ f.abs()
    n, r = a.shape[1], f.shape[1]
    per = 2.0 ** -16 * t.abs() + 2 * (n + 64) * U * mag
    tol += (per + 2 * r * 2 * U * (t.abs() + per)) @ s.abs().t()
    return t @ s.t()


def forward(x, codes, w, up, down, out_dtype):
    """(y, tolerance) of one layer."""
    q, s = token_levels(x)
    main = (q @ codes.double().t()) * s * w.double()
    tol = 4 * U * main.abs()
    y = main + _low(x, down, up, tol)
    return y, _rounded(y, tol, out_dtype)


def gradient(dy, codes, w, up, down, out_dtype):
    d, t = gradient_levels(dy, w)
    lo = torch.remainder(d + 128, 256) - 128
    c = codes.double()
    acc, low = d @ c, lo @ c
    m, k = acc.shape
    h = sylvester(dy.device)
    main = (acc.view(m, -1, 256) @ h).view(m, k) * (t / 16.0)
    mag = (acc.abs() + 2 * low.abs()).view(m, -1, 256).sum(2, keepdim=True).expand(-1, -1, 256)
    tol = 12 * U * mag.reshape(m, k) * (t / 16.0) + U * main.abs()
    y = main + _low(dy, up, down, tol)
    return y, _rounded(y, tol, out_dtype)


def _rounded(y, tol, out_dtype):
    tol = tol + 2 * U * y.abs()
    return tol + (2.0 ** -8 * (y.abs() + tol) if out_dtype == torch.bfloat16 else 0.0)


def check(got, want, tol):
    """Every element within its bound; NaN where and only where the reference has it."""
    got = got.double()
    assert got.shape == want.shape
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), "NaN in other places"
    over = ((got - want).abs() - tol)[~nan]
    if over.numel():
        worst = float(over.max())
        assert worst <= 0.0, f"{int((over > 0).sum())} of {over.numel()} past the bound, by {worst:.3g}"


# ------------------------------------------------------------------ inputs
def make_layer(rng, n, k, rank, device, groups=None):
    """Random payload tensors of one layer or of `groups` experts."""
    lead = () if groups is None else (groups,)
    codes = np.clip(np.rint(rng.standard_normal(lead + (n, k)) * 30.0), -128, 127).astype(np.int8)
    w = (4.5 / np.sqrt(k) / 127.0 * np.exp(0.1 * rng.standard_normal(lead + (n,)))).astype(np.float16)
    bf = lambda a: torch.from_numpy(a.astype(np.float32)).bfloat16().to(device)   # noqa: E731
    up = bf(rng.standard_normal(lead + (n, rank)) * (1.5 / np.sqrt(n))) if rank else None
    down = bf(rng.standard_normal(lead + (k, rank)) * (1.5 / np.sqrt(k))) if rank else None
    return torch.from_numpy(codes).to(device), torch.from_numpy(w).to(device), up, down


def make_rows(rng, m, cols, device, scale=1.0):
    """Rows with a spread of magnitudes and a few outlier columns, as bf16."""
    a = rng.standard_normal((m, cols)) * np.exp(rng.standard_normal((m, 1))) * scale
    a[:, rng.choice(cols, max(1, cols // 200), replace=False)] *= 20.0
    return torch.from_numpy(a.astype(np.float32)).bfloat16().to(device)
