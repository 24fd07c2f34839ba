"""Inputs, 64-bit definitions and bounds for the tests of the experts' feed-forward block.

Bounds, elementwise, none of them fitted: a rounding to bf16 is off by at most 2^-8 of the value.
A sum of K products of bf16 values (each exact in fp32) is added by the tensor cores with one
truncation, 2^-23 of what has been added so far, per 16 products at least and per product at most;
what has been added so far is at most S, the sum of the products' magnitudes. So a sum is off by
at most K * 2^-23 * S. The activations' slopes are below 1.13, and their fast exponential and
reciprocal are off by less than 2^-18 of the values that they are multiplied with."""
from __future__ import annotations

import math

import torch

BF16 = 2.0 ** -8
SLOPE = 1.13
FAST = 2.0 ** -18
SENTINEL = 77.0
ACTS = {"silu": 0, "gelu": 1}


class Rows:
    """Experts' rows in slabs of R ranks: counts per expert, in order; rows past max_rows are dropped."""

    def __init__(self, counts, R, max_rows, device="cuda"):
        self.E, self.R, self.max_rows = len(counts), R, max_rows
        per = self.E // R
        self.offsets = torch.tensor([sum(counts[:e]) for e in range(self.E + 1)], dtype=torch.int32, device=device)
        self.spans = []
        for e in range(self.E):
            first = sum(counts[e // per * per:e])
            a, b = min(first, max_rows), min(first + counts[e], max_rows)
            self.spans.append((e // per, a, b))
        self.dropped = any(sum(counts[r * per:(r + 1) * per]) > max_rows for r in range(R))

    def owned(self):
        m = torch.zeros((self.R, self.max_rows), dtype=torch.bool, device=self.offsets.device)
        for r, a, b in self.spans:
            m[r, a:b] = True
        return m


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def slab(rows: Rows, seed, width, scale=1.0):
    """Random rows where experts own them, NaN everywhere else."""
    t = normal(seed, rows.R, rows.max_rows, width, scale=scale)
    t[~rows.owned()] = math.nan
    return t


def out(rows: Rows, width, dtype=torch.bfloat16):
    t = torch.full((rows.R, rows.max_rows, width), SENTINEL, dtype=torch.float32, device="cuda")
    return t.to(dtype)


def act_of(name, v):
    """An activation and its derivative."""
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s + v * s * (1 - s)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)


def product(a, b):
    """a [n][k] times b [m][k] transposed in 64 bits, and the bound of the tensor cores' sum."""
    a, b = a.double(), b.double()
    return a @ b.T, a.shape[1] * 2.0 ** -23 * (a.abs() @ b.abs().T)


def close(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - (BF16 * want.abs() + bound)
    assert over.numel() == 0 or float(over.max()) <= 0, (what, float(over.max()), float(want.abs().max()))


def untouched(t, rows: Rows, what):
    kept = t.float()[~rows.owned()]
    assert torch.equal(kept, torch.full_like(kept, float(torch.tensor(SENTINEL).to(t.dtype)))), what


def check_gate_up(x, w, rows: Rows, act, h, pre=None, pre_q=None, pre_scales=None):
    F = w.shape[1] // 2
    for e, (r, a, b) in enumerate(rows.spans):
        if a == b:
            continue
        c, err = product(x[r, a:b], w[e])
        gate, up, eg, eu = c[:, :F], c[:, F:], err[:, :F], err[:, F:]
        v, _ = act_of(act, gate)
        close(h[r, a:b], v * up, 1.01 * (SLOPE * eg * up.abs() + v.abs() * eu) + SLOPE * eg * eu + FAST * (gate * up).abs(),
              ("h", e))
        if pre is not None:
            close(pre[r, a:b], c, err, ("pre", e))
        if pre_q is not None:
            s = pre_scales[r, a:b].double()
            amax, worst = (t.view(b - a, -1, 128).amax(2) for t in (c.abs(), err))
            assert bool(((s - amax / 448).abs() <= BF16 * amax / 448 + 1.01 * worst / 448).all()), ("scales", e)
            wide = s.repeat_interleave(128, dim=1)
            got = pre_q[r, a:b].view(torch.float8_e4m3fn).double() * wide
            # half a step of E4M3: 2^-4 of the value, 2^-10 scales where codes are subnormal
            assert bool(((got - c).abs() <= 2.0 ** -4 * c.abs() + 2.0 ** -10 * wide + 1.1 * err).all()), ("codes", e)
    for name, t in (("h", h), ("pre", pre), ("pre_q", pre_q), ("pre_scales", pre_scales)):
        if t is not None:
            untouched(t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t, rows, name)


def check_down(h, w, rows: Rows, y):
    for e, (r, a, b) in enumerate(rows.spans):
        if a < b:
            close(y[r, a:b], *product(h[r, a:b], w[e]), ("y", e))
    untouched(y, rows, "y")


def decode(pre_q, pre_scales):
    return pre_q.view(torch.float8_e4m3fn).double() * pre_scales.double().repeat_interleave(128, dim=-1)


def check_down_bwd(dy, w, pre, rows: Rows, act, dpre, h=None):
    """pre: what the checkpoint stands for, in 64 bits"""
    F = w.shape[2]
    for e, (r, a, b) in enumerate(rows.spans):
        if a == b:
            continue
        dh, err = product(dy[r, a:b], w[e].T)
        gate, up = pre[r, a:b, :F].double(), pre[r, a:b, F:].double()
        v, dv = act_of(act, gate)
        # act' = s + g s (1 - s) p'(g): |g p'(g)| s (1 - s) < 2, and s is off by less than 2^-20
        close(dpre[r, a:b, :F], dh * up * dv, 1.01 * err * (up * dv).abs() + 4 * FAST * (dh * up).abs(), ("dgate", e))
        close(dpre[r, a:b, F:], dh * v, 1.01 * err * v.abs() + FAST * (dh * gate).abs(), ("dup", e))
        if h is not None:
            close(h[r, a:b], v * up, FAST * (gate * up).abs(), ("h", e))
    untouched(dpre, rows, "dpre")
    if h is not None:
        untouched(h, rows, "h")


def check_gate_up_bwd(dpre, w, rows: Rows, dx):
    for e, (r, a, b) in enumerate(rows.spans):
        if a < b:
            close(dx[r, a:b], *product(dpre[r, a:b], w[e].T), ("dx", e))
    untouched(dx, rows, "dx")


def check_wgrad(dout, x, rows: Rows, dw):
    for e, (r, a, b) in enumerate(rows.spans):
        if a == b:
            assert not dw[e].any(), ("dw", e)
        else:
            close(dw[e], *product(dout[r, a:b].T, x[r, a:b].T), ("dw", e))
