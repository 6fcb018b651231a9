"""What is measured of the int8 layer's products: cases, inputs, the plain form and the 64-bit values.

Four operators on the int8-residual payload (codes c [N][K], row scales w [N], factors up [N][r]
and down [K][r]); S is the 256-point Sylvester matrix (entries +-1) on blocks of 256 columns:

  fwd           y = s w (q c^T) + (x down) up^T, q and s the 8-bit integers and scale of each
                rotated token
  dgrad         dx = (t / 16) ((d c) S) + (dy up) down^T, d and t the 16-bit integers and scale of
                each row of dy w
  grouped_fwd   fwd with one payload per expert, rows sorted by expert
  grouped_dgrad dgrad likewise

``own`` selects the framework's calls; otherwise `run` computes the plain form from elementary torch
operations.
"""
import math

import numpy as np
import torch

own = False

OPS = ("fwd", "dgrad", "grouped_fwd", "grouped_dgrad")
LARGEST = 4480 * 16384 * 6144      # rows x N x K of the largest listed case
MOST_WEIGHTS = 380_000_000         # codes of all experts together


def listed():
    d = dict
    return [
        # one token through an MLP-up projection: the latency of decoding
        d(name="fwd 1 token up", op="fwd", m=1, n=16384, k=6144, e=1, rank=16, out="bf16"),
        # a small batch of decoded tokens through the long-K projection
        d(name="fwd 48 tokens down", op="fwd", m=48, n=6144, k=16384, e=1, rank=16, out="bf16"),
        # a short prompt, odd row and column counts, full-precision result
        d(name="fwd odd prompt", op="fwd", m=777, n=1003, k=2304, e=1, rank=32, out="fp32"),
        # the prompt pass of an image or text model's MLP-up projection
        d(name="fwd prompt up", op="fwd", m=4480, n=16384, k=6144, e=1, rank=16, out="bf16"),
        # the tiny layer of the tests, in a training step
        d(name="dgrad tiny", op="dgrad", m=64, n=512, k=512, e=1, rank=32, out="fp32"),
        # an odd training batch with an odd output width
        d(name="dgrad odd", op="dgrad", m=1001, n=2051, k=4096, e=1, rank=64, out="fp32"),
        # the largest training step
        d(name="dgrad up", op="dgrad", m=4480, n=16384, k=6144, e=1, rank=16, out="bf16"),
        # decoding with experts: few rows for each, some experts without any
        d(name="experts decode", op="grouped_fwd", m=128, n=2816, k=2048, e=64, rank=16, out="bf16"),
        # a prompt through experts, unevenly loaded
        d(name="experts prompt", op="grouped_fwd", m=16384, n=2816, k=2048, e=64, rank=16, out="bf16"),
        # few experts, odd width, no low-rank branch
        d(name="experts odd", op="grouped_fwd", m=1533, n=1001, k=1280, e=7, rank=0, out="fp32"),
        # the backward of the prompt through experts
        d(name="experts gradient", op="grouped_dgrad", m=8192, n=2816, k=2048, e=32, rank=16,
          out="bf16"),
        # a small uneven training batch
        d(name="experts gradient odd", op="grouped_dgrad", m=413, n=715, k=768, e=12, rank=32,
          out="fp32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    while True:
        op = rng.choice(OPS)
        many = op.startswith("grouped")
        m = _log_int(rng, 1, 16384 if many else 4480)
        n = _log_int(rng, 64, 4096 if many else 16384)
        k = 256 * _log_int(rng, 1, 16 if many else 64)
        e = _log_int(rng, 2, 64) if many else 1
        rank, out = rng.choice((0, 16, 32, 64)), rng.choice(("bf16", "fp32"))
        if m * n * k <= LARGEST and e * n * k <= MOST_WEIGHTS:
            return dict(op=op, m=m, n=n, k=k, e=e, rank=rank, out=out)


def work(case):
    m, n, k, e, r = (case[v] for v in ("m", "n", "k", "e", "rank"))
    used = min(e, e * (1.0 - (1.0 - 1.0 / e) ** m)) if e > 1 else 1.0   # experts that get a row
    size = 2 if case["out"] == "bf16" else 4
    into, from_ = (n, k) if case["op"].endswith("dgrad") else (k, n)
    return {"bytes": 2 * m * into + size * m * from_ + used * (n * k + 2 * n + 2 * r * (n + k)),
            "flops": 2 * m * n * k + 2 * m * r * (n + k)}


def prepare(case, seed):
    m, n, k, e, r = (case[v] for v in ("m", "n", "k", "e", "rank"))
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # the payload of a quantized N(0, 1/K) weight, one for each expert
    codes = torch.cat([(randn(n, k) * 30.0).round_().clamp_(-128, 127).to(torch.int8)[None]
                       for _ in range(e)])
    scales = (4.5 / math.sqrt(k) / 127.0 * torch.exp(0.1 * randn(e, n))).to(torch.float16)
    up = (randn(e, n, r) * (1.5 / math.sqrt(n))).bfloat16() if r else None
    down = (randn(e, k, r) * (1.5 / math.sqrt(k))).bfloat16() if r else None
    if case["op"].endswith("dgrad"):
        # gradients: small, a spread of row magnitudes
        a = (randn(m, n) * 1e-3 * torch.exp(randn(m, 1))).bfloat16()
    else:
        # activations: unit variance, 0.5 % outlier channels 20 times as large
        a = randn(m, k)
        a[:, torch.from_numpy(rng.choice(k, max(1, k // 200), replace=False)).to(dev)] *= 20.0
        a = a.bfloat16()
    share = rng.exponential(size=e) + 0.05        # uneven experts
    counts = rng.multinomial(m, share / share.sum())
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    if e == 1:
        codes, scales = codes[0], scales[0]
        up, down = (None, None) if not r else (up[0], down[0])
    sylvester = torch.ones(1, 1, dtype=torch.float64, device=dev)
    for _ in range(8):
        sylvester = torch.cat([torch.cat([sylvester, sylvester], 1),
                               torch.cat([sylvester, -sylvester], 1)])
    return dict(op=case["op"], a=a, codes=codes, scales=scales, up=up, down=down,
                offsets=torch.from_numpy(offsets).to(dev), cap=int(counts.max()),
                out=torch.bfloat16 if case["out"] == "bf16" else torch.float32,
                sylvester=sylvester)


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import w4_gemm_amd as W
    if s["op"] == "fwd":
        return W.linear_fwd_w8a8(s["a"], W.W8Payload(s["codes"], s["scales"], s["up"], s["down"]),
                                 out_dtype=s["out"])
    if s["op"] == "dgrad":
        return W.linear_dgrad_w8(s["a"], W.W8Payload(s["codes"], s["scales"], s["up"], s["down"]),
                                 out_dtype=s["out"])
    p = W.GroupedW8Payload(s["codes"], s["scales"], s["up"], s["down"])
    if s["op"] == "grouped_fwd":
        return W.grouped_fwd_w8a8(s["a"], s["offsets"], p, out_dtype=s["out"])
    return W.grouped_dgrad_w8(s["a"], s["offsets"], p, out_dtype=s["out"])


# ------------------------------------------------------------------ plain form
def _power_of_two(e):
    """2^e in 64 bits for integers e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _to_grid(v, top):
    """(integers on the grid of +-top, scale) of each row of v (fp32).  Every step is one fp32
    rounding of the 64-bit value: a value next to a border between two integers must fall on the
    side that the definition puts it."""
    a = v.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100).double()
    inv = (top / a).float().double()
    return torch.round((v.double() * inv).float()), (a / top).float()


def _rotated(x, sylvester):
    """x H in fp32: each block of 256 as 24-bit integers, whose sums are exact."""
    m, k = x.shape
    b = x.double().view(m, k // 256, 256)
    e = torch.frexp(b.abs().amax(-1, keepdim=True)).exponent.clamp(min=-125)
    sums = torch.trunc(b * _power_of_two(23 - e)) @ sylvester
    return (sums.float().double() * _power_of_two(e - 27)).float().view(m, k)


def _plain(s):
    a, codes, op = s["a"], s["codes"].float(), s["op"]
    back = op.endswith("dgrad")
    w = s["scales"].float()
    first, second = (s["up"], s["down"]) if back else (s["down"], s["up"])
    if s["codes"].dim() == 3:
        # rows of each expert side by side, padded to the fullest
        row = torch.arange(a.shape[0], device=a.device)
        gid = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
        at = (gid, row - s["offsets"].long()[gid])
        w = w[gid]

        def times(v, mat, transpose):
            buf = torch.zeros(mat.shape[0], s["cap"], v.shape[1], device=v.device)
            buf[at] = v
            return torch.bmm(buf, mat.transpose(1, 2) if transpose else mat)[at]
    else:
        def times(v, mat, transpose):
            return v @ (mat.t() if transpose else mat)
    if back:
        d, t = _to_grid(a.float() * w, 32512.0)
        c = times(d, codes, False)
        h = s["sylvester"].float() / 16.0
        y = (c.view(a.shape[0], -1, 256) @ h).view_as(c) * t
    else:
        q, t = _to_grid(_rotated(a, s["sylvester"]), 127.0)
        y = times(q, codes, True) * t * w
    if first is not None:
        y = y + times(times(a.float(), first.float(), False), second.float(), True)
    return y.to(s["out"])


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The operators' definition with the products in 64 bits, expert by expert."""
    s = prepare(case, seed)
    back = case["op"].endswith("dgrad")
    n_experts = case["e"]
    off = s["offsets"].tolist()

    def of(t, e):
        return None if t is None else (t[e] if n_experts > 1 else t).double()

    parts = []
    for e in range(n_experts):
        a = s["a"][off[e]:off[e + 1]].double()
        c, w, up, down = (of(s[v], e) for v in ("codes", "scales", "up", "down"))
        if back:
            q, t = _levels(a * w, 32512)
            y = _butterflies(q @ c) * (t / 16.0)
            low = None if up is None else (a @ up) @ down.t()
        else:
            q, t = _levels(_exact_rotation(a), 127)
            y = (q @ c.t()) * t * w
            low = None if up is None else (a @ down) @ up.t()
        parts.append(y if low is None else y + low)
    return torch.cat(parts)


def _butterflies(v):
    """Unnormalized 256-point Walsh-Hadamard transform of each block of 256 columns."""
    rows, cols = v.shape
    h = 1
    while h < 256:
        p = v.reshape(rows, cols // (2 * h), 2, h)
        v = torch.stack([p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]], 2).reshape(rows, cols)
        h *= 2
    return v


def _exact_rotation(a):
    """Each block of 256 as integers below 2^23, transformed in int64, rounded to fp32."""
    rows, k = a.shape
    b = a.reshape(rows * (k // 256), 256)
    top = b.abs().amax(1).float().view(torch.int32) >> 23          # biased exponent
    unit = (1023 + (top.clamp(min=1).long() - 149) << 52).view(torch.float64)[:, None]
    ints = (b / unit).to(torch.int64)                              # toward zero
    sums = _butterflies(ints.reshape(rows, k)).reshape(-1, 256).to(torch.float32).double()
    return (sums * (unit / 16.0)).float().double().reshape(rows, k)


def _levels(v, top):
    """Integers and scale of each row: quotients in 64 bits, rounded to fp32 where the definition
    holds them in fp32."""
    a = torch.maximum(v.abs().max(dim=1, keepdim=True).values if v.shape[1] else v,
                      torch.full((1, 1), 2.0 ** -100, dtype=torch.float64, device=v.device))
    reciprocal = (torch.full_like(a, float(top)) / a).to(torch.float32).to(torch.float64)
    return (v * reciprocal).to(torch.float32).round().to(torch.float64), \
        (a / top).to(torch.float32).to(torch.float64)
