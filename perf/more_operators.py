"""What is measured of the 8-bit floating-point layer: cases, inputs, the plain form, 64-bit values.

The layer holds e4m3 codes with one power-of-two scale for each block of 128 x 128; rows that meet
it are rounded to e4m3 with one such scale for each 128 values along the contraction:

  Q(v)          per block of 128: the least e >= -127 with max|v| <= 448 * 2^e; codes e4m3(v / 2^e)
  quantize      codes and exponents of a weight, blocks of 128 x 128
  fwd           y = Q(x) W^T, for one layer or with rows sorted by expert
  dgrad         dx = Q(dy) W, likewise
  gated         h = act(g) * u, g = Q(x) Wg^T, u = Q(x) Wu^T, likewise; training keeps g and u
  gated_bwd     dg = dh u act'(g), du = dh act(g), dx = Q(dg) Wg + Q(du) Wu

``own`` selects the framework's calls; otherwise `run` computes the plain form from elementary torch
operations.
"""
import math

import numpy as np
import torch

own = False

OPS = ("quantize", "fwd", "dgrad", "gated", "gated_bwd")
LARGEST = 2 * 4480 * 16384 * 6144      # products of the largest listed case
MOST_WEIGHTS = 370_000_000             # codes of all experts and both projections together


def listed():
    d = dict
    return [
        # an odd projection of the builder, weights as trained
        d(name="quantize odd", op="quantize", n=1003, k=2311, w="bf16"),
        # an MLP-up weight in the builder
        d(name="quantize up", op="quantize", n=16384, k=6144, w="fp32"),
        # one token through an MLP-up projection: the latency of decoding
        d(name="fwd 1 token up", op="fwd", m=1, n=16384, k=6144, e=1, out="bf16"),
        # a short prompt, odd sizes all round, full-precision result
        d(name="fwd odd prompt", op="fwd", m=777, n=1003, k=2311, e=1, out="fp32"),
        # the prompt pass of an image or text model's MLP-down projection
        d(name="fwd prompt down", op="fwd", m=4480, n=6144, k=16384, e=1, out="bf16"),
        # an odd training batch with odd widths
        d(name="dgrad odd", op="dgrad", m=1001, n=2051, k=4099, e=1, out="fp32"),
        # the backward of a prompt through the experts' down projections, unevenly loaded
        d(name="experts gradient", op="dgrad", m=8192, n=2048, k=2816, e=32, out="bf16"),
        # a few decoded tokens through the gated half of an MLP
        d(name="gated 8 tokens", op="gated", m=8, n=16384, k=6144, e=1, act="silu", save=False,
          out="bf16"),
        # the forward of a training step through the gated half of an MLP
        d(name="gated prompt", op="gated", m=4480, n=16384, k=6144, e=1, act="silu", save=True,
          out="bf16"),
        # decoding with gated experts: few rows for each, some experts without any
        d(name="gated experts decode", op="gated", m=128, n=1408, k=2048, e=64, act="silu",
          save=False, out="bf16"),
        # the largest training step's backward
        d(name="gated gradient", op="gated_bwd", m=4480, n=16384, k=6144, e=1, act="silu",
          out="bf16"),
        # a small uneven training batch of gated experts, odd widths
        d(name="gated experts gradient odd", op="gated_bwd", m=413, n=715, k=771, e=12,
          act="gelu_tanh", out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    while True:
        op = rng.choice(OPS)
        if op == "quantize":
            n, k = _log_int(rng, 1, 16384), _log_int(rng, 1, 16384)
            if n * k <= 16384 * 6144:
                return dict(op=op, n=n, k=k, w=rng.choice(("bf16", "fp32")))
            continue
        many = rng.random() < 0.5
        m = _log_int(rng, 1, 16384 if many else 4480)
        n = _log_int(rng, 64, 4096 if many else 16384)
        k = _log_int(rng, 64, 4096 if many else 16384)
        e = _log_int(rng, 2, 64) if many else 1
        both = 2 if op.startswith("gated") else 1
        if both * m * n * k > LARGEST or both * e * n * k > MOST_WEIGHTS:
            continue
        case = dict(op=op, m=m, n=n, k=k, e=e, out=rng.choice(("bf16", "fp32")))
        if both == 2:
            case["act"] = rng.choice(("silu", "gelu", "gelu_tanh"))
        if op == "gated":
            case["save"] = rng.random() < 0.5
        if op == "gated_bwd":
            # dg and du pass exp on their way to 8 bits: only a 16-bit dx means something
            case["out"] = "bf16"
        return case


def _blocks(v):
    return -(-v // 128)


def work(case):
    op, n, k = case["op"], case["n"], case["k"]
    exps = _blocks(n) * _blocks(k)
    if op == "quantize":
        return {"bytes": (2 if case["w"] == "bf16" else 4) * n * k + n * k + exps, "flops": 0}
    m, e = case["m"], case["e"]
    used = min(e, e * (1.0 - (1.0 - 1.0 / e) ** m)) if e > 1 else 1.0   # experts that get a row
    size = 2 if case["out"] == "bf16" else 4
    both = 2 if op.startswith("gated") else 1
    into, from_ = (n, k) if op in ("dgrad", "gated_bwd") else (k, n)
    moved = 2 * m * into + size * m * from_ + both * used * (n * k + exps)
    if op == "gated" and case["save"]:
        moved += 2 * 2 * m * n
    if op == "gated_bwd":
        moved += 2 * 2 * m * n + 2 * 2 * m * n       # g and u in, dg and du out
    return {"bytes": moved, "flops": 2 * both * m * n * k}


DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def prepare(case, seed):
    op, n, k = case["op"], case["n"], case["k"]
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def weight():
        # N(0, 1/K), rows and columns of uneven size
        return randn(n, k) * torch.exp(0.3 * randn(n, 1)) * (torch.exp(0.3 * randn(1, k))
                                                             / math.sqrt(k))

    if op == "quantize":
        return dict(op=op, w=weight().to(DTYPES[case["w"]]))
    m, e = case["m"], case["e"]
    payloads = []
    for _ in range(2 if op.startswith("gated") else 1):
        codes = torch.empty(e, n, 128 * _blocks(k), dtype=torch.float8_e4m3fn, device=dev)
        exps = torch.empty(e, _blocks(n), _blocks(k), dtype=torch.uint8, device=dev)
        for i in range(e):
            codes[i], exps[i] = _plain_weight(weight())
        payloads.append((codes[0], exps[0]) if e == 1 else (codes, exps))
    s = dict(op=op, k=k, payloads=payloads, out=DTYPES[case["out"]], act=case.get("act"),
             save=case.get("save"))
    if op in ("fwd", "gated"):
        # activations: unit variance, 0.5 % outlier channels 20 times as large
        a = randn(m, k)
        a[:, torch.from_numpy(rng.choice(k, max(1, k // 200), replace=False)).to(dev)] *= 20.0
    else:
        # gradients: small, a spread of row magnitudes
        a = randn(m, n) * 1e-3 * torch.exp(randn(m, 1))
    s["a"] = a.bfloat16()
    if op == "gated_bwd":
        s["g"], s["u"] = (1.5 * randn(m, n)).bfloat16(), (1.5 * randn(m, n)).bfloat16()
    share = rng.exponential(size=e) + 0.05        # uneven experts
    counts = rng.multinomial(m, share / share.sum())
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    s["offsets"] = torch.from_numpy(offsets).to(dev) if e > 1 else None
    s["cap"] = int(counts.max())
    return s


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import w4_gemm_amd as W
    op, off, out = s["op"], s.get("offsets"), s.get("out")
    if op == "quantize":
        p, _ = W.quantize_weight_f8(s["w"])
        return p.codes, p.exps
    if off is None:
        p = [W.F8Payload(c, x, s["k"]) for c, x in s["payloads"]]
        if op == "fwd":
            return W.linear_fwd_f8(s["a"], *p, out_dtype=out)
        if op == "dgrad":
            return W.linear_dgrad_f8(s["a"], *p, out_dtype=out)
        if op == "gated":
            return W.gated_fwd_f8(s["a"], *p, act=s["act"], save=s["save"], out_dtype=out)
        return W.gated_bwd_f8(s["a"], s["g"], s["u"], *p, act=s["act"], out_dtype=out)
    p = [W.GroupedF8Payload(c, x, s["k"]) for c, x in s["payloads"]]
    if op == "fwd":
        return W.grouped_fwd_f8(s["a"], off, *p, out_dtype=out)
    if op == "dgrad":
        return W.grouped_dgrad_f8(s["a"], off, *p, out_dtype=out)
    if op == "gated":
        return W.grouped_gated_fwd_f8(s["a"], off, *p, act=s["act"], save=s["save"], out_dtype=out)
    return W.grouped_gated_bwd_f8(s["a"], s["g"], s["u"], off, *p, act=s["act"], out_dtype=out)


# ------------------------------------------------------------------ plain form
def _exponent(top):
    """Exponent byte of a block with the largest magnitude top (fp32): 448 is 1.75 * 2^8."""
    bits = top.contiguous().view(torch.int32)
    e = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    return e.clamp(min=0)


def _power_of_two(e):
    """2^(e - 127) in fp32 for exponent bytes 1 .. 254, and 2^-127 for 0."""
    return torch.where(e > 0, (e.int() << 23).view(torch.float32), 2.0 ** -127)


def _padded(v, rows, cols):
    return torch.nn.functional.pad(v, (0, cols - v.shape[1], 0, rows - v.shape[0]))


def _plain_weight(w):
    """e4m3 codes [N, K to the next 128] and exponent bytes of blocks of 128 x 128."""
    n, k = w.shape
    nb, kb = _blocks(n), _blocks(k)
    v = _padded(w.float(), 128 * nb, 128 * kb).view(nb, 128, kb, 128)
    e = _exponent(v.abs().amax((1, 3)))
    codes = (v * _power_of_two(254 - e)[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(128 * nb, 128 * kb)[:n], e.to(torch.uint8)


def _held(codes, exps):
    """The values (fp32) that codes [..., N, K] with exponents of 128 x 128 blocks stand for."""
    scale = _power_of_two(exps).repeat_interleave(128, -2)[..., :codes.shape[-2], :]
    return codes.float() * scale.repeat_interleave(128, -1)


def _rounded(v):
    """The values (fp32) that rows are rounded to, padded with zeros to blocks of 128."""
    m, c = v.shape
    b = _padded(v, m, 128 * _blocks(c)).view(m, -1, 128)
    e = _exponent(b.abs().amax(2, keepdim=True))
    q = (b * _power_of_two(254 - e)).to(torch.float8_e4m3fn).float()
    return (q * _power_of_two(e)).view(m, -1)


def _activation(act, g):
    """act(g) and act'(g)."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    slope = c * (1.0 + 3.0 * 0.044715 * g * g)
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * slope


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _plain_weight(s["w"])
    a, k, off = s["a"].float(), s["k"], s["offsets"]
    weights = [_held(*p)[..., :k] for p in s["payloads"]]
    if off is None:
        def times(v, w):
            return v @ w
    else:
        # rows of each expert side by side, padded to the fullest
        row = torch.arange(a.shape[0], device=a.device)
        gid = torch.searchsorted(off[1:].long(), row, right=True)
        at = (gid, row - off.long()[gid])

        def times(v, w):
            buf = torch.zeros(w.shape[0], s["cap"], v.shape[1], device=v.device)
            buf[at] = v
            return torch.bmm(buf, w)[at]

    def forward(x, w):
        return times(x, w.transpose(-1, -2))

    if op == "fwd":
        return forward(_rounded(a)[:, :k], weights[0]).to(s["out"])
    if op == "dgrad":
        return times(_rounded(a)[:, :a.shape[1]], weights[0]).to(s["out"])
    if op == "gated":
        x = _rounded(a)[:, :k]
        g, u = (forward(x, w) for w in weights)
        h = (_activation(s["act"], g)[0] * u).to(s["out"])
        return (h, g.bfloat16(), u.bfloat16()) if s["save"] else h
    value, slope = _activation(s["act"], s["g"].float())
    dg, du = a * s["u"].float() * slope, a * value
    dx = times(_rounded(dg)[:, :a.shape[1]], weights[0])
    dx += times(_rounded(du)[:, :a.shape[1]], weights[1])
    return dx.to(s["out"]), dg.bfloat16(), du.bfloat16()


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The operators' definition in 64 bits, expert by expert."""
    s = prepare(case, seed)
    if case["op"] == "quantize":
        w = s["w"].double()
        n, k = w.shape
        codes = torch.zeros(n, 128 * _blocks(k), dtype=torch.float64, device=w.device)
        exps = torch.zeros(_blocks(n), _blocks(k), dtype=torch.uint8, device=w.device)
        for i in range(_blocks(n)):
            rows = slice(128 * i, min(n, 128 * i + 128))
            strip = w[rows]
            for j in range(_blocks(k)):
                cols = slice(128 * j, min(k, 128 * j + 128))
                codes[rows, cols], e = _grid(strip[:, cols].reshape(1, -1), strip[:, cols].shape)
                exps[i, j] = (e + 127).to(torch.uint8)
        return codes, exps
    e, k = case["e"], case["k"]
    off = [0, s["a"].shape[0]] if e == 1 else s["offsets"].tolist()
    parts = []
    for i in range(e):
        rows = slice(off[i], off[i + 1])
        weights = [_values(*(p if e == 1 else (p[0][i], p[1][i])))[:, :k] for p in s["payloads"]]
        parts.append(_exact_rows(case, {v: s[v][rows].double() for v in "agu" if v in s}, weights))
    return tuple(torch.cat(v) for v in zip(*parts)) if isinstance(parts[0], tuple) \
        else torch.cat(parts)


def _exact_rows(case, s, weights):
    op, a = case["op"], s["a"]
    if op == "fwd":
        return _nearest(a) @ weights[0].t()
    if op == "dgrad":
        return _nearest(a) @ weights[0]
    if op == "gated":
        x = _nearest(a)
        g, u = x @ weights[0].t(), x @ weights[1].t()
        h = _curve(case["act"], g)[0] * u
        return (h, g, u) if case["save"] else h
    value, slope = _curve(case["act"], s["g"])
    dg, du = a * s["u"] * slope, a * value
    return _nearest(dg) @ weights[0] + _nearest(du) @ weights[1], dg, du


def _curve(act, g):
    if act == "silu":
        return g * torch.sigmoid(g), torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g)
    if act == "gelu":
        cdf = torch.special.ndtr(g)
        return g * cdf, cdf + g * torch.exp(-g * g / 2) * (2 * math.pi) ** -0.5
    # tanh(z) = 2 sigmoid(2 z) - 1
    z = 2 * (2 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3)
    p = torch.sigmoid(z)
    return g * p, p + g * p * torch.sigmoid(-z) * 2 * (2 / math.pi) ** 0.5 * (1 + 0.134145 * g ** 2)


def _scaled(v, e):
    """v * 2^e in 64 bits for whole e, exactly."""
    return v * (e.long() + 1023 << 52).view(torch.float64)


def _grid(v, shape=None):
    """Codes of v [blocks, values] on the e4m3 grid of each block's 2^e, and e."""
    top = v.abs().amax(1) if v.shape[1] else v.new_zeros(v.shape[0])
    mant, ex = torch.frexp(top)                       # 448 = 0.875 * 2^9
    e = torch.where(top > 0, ex - 9 + (mant > 0.875).int(), -127).clamp(min=-127)
    u = _scaled(v, -e[:, None])
    step = torch.frexp(u)[1].clamp(min=-5) - 4        # three bits behind the leading one
    q = _scaled(torch.round(_scaled(u, -step)), step)
    return (q if shape is None else q.reshape(shape)), e.squeeze()


def _nearest(v):
    """Rows of v as they are rounded, block of 128 by block of 128."""
    cols = v.shape[1]
    parts = []
    for c in range(0, cols, 128):
        q, e = _grid(v[:, c:c + 128])
        parts.append(_scaled(q, e.reshape(-1, 1)))
    return torch.cat(parts, 1)


def _values(codes, exps):
    """Codes times their blocks' powers of two, strip by strip of 128 rows."""
    strips = []
    for i, row in enumerate(exps.long()):
        c = codes[128 * i:128 * i + 128].float().double()
        strips.append(_scaled(c.view(c.shape[0], -1, 128), row[None, :, None] - 127).view(c.shape))
    return torch.cat(strips)
