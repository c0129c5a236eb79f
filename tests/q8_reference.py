"""The 8-bit path from its definition, in 64 bits, for its tests: quantization
of rows, the root-mean-square norm, and products of codes (plain torch, on the
device of its arguments)."""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def quantize(v):
    """Codes (int8) and scales (fp32) of the rows of a float64 v."""
    top = v.abs().amax(1)
    bad = ~torch.isfinite(v).all(1)
    scale = torch.where(bad, torch.zeros_like(top), top / 127).float()
    bad |= ~torch.isfinite(scale)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    c = torch.round(v / scale.double()[:, None]).clamp(-127, 127)
    c = torch.where(bad[:, None], torch.zeros_like(c), c).to(torch.int8)
    return c, torch.where(bad, torch.full_like(scale, math.nan), scale)


def norm(x, residual, weight, eps):
    """(h as bf16, u in float64) of bf16 rows; rows without a finite u are NaN."""
    h = x if residual is None else (x.double() + residual.double()).bfloat16()
    d = h.double()
    p = d * weight.double()
    u = p / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    good = torch.isfinite(d).all(1) & torch.isfinite(p.float()).all(1)
    return h, torch.where(good[:, None], u, torch.full_like(u, math.nan))


def product(xq, xs, wq, ws, act="none"):
    """(y, tolerance of an fp32 y) in float64.

    p = fp32(fp32(fp32(sum) xs) ws) is off by 3 half steps e = 2^-24.  A gated y
    = a sigmoid(z) b has a and b (3 e each), the sigmoid of an a that is off (its
    relative change is at most |z| times z's own, which is 3 times a's: 9 |z| e),
    the sigmoid's own error (|z| 2^-21.7 < 5 |z| e, and 4 e of its reciprocal,
    addition and product) and two products: (12 + 14 |z|) e, below (20 + 16 |z|) e.
    Where the sigmoid is below 2^-126 it may be anything up to that."""
    s = xq.double() @ wq.double().t()
    p = s * xs.double()[:, None] * ws.double()
    e = HALF[torch.float32]
    if act == "none":
        return p, p.abs() * 3.01 * e
    n = wq.shape[0] // 2
    a, b = p[:, :n], p[:, n:]
    z = a if act == "silu" else 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
    y = a * torch.sigmoid(z) * b
    return y, y.abs() * (20 + 16 * z.abs().clamp(max=90)) * e + (a * b).abs() * 2.0 ** -126


def check(y, want, tol, what=""):
    """y (fp32, or bf16 with its own rounding on top) against a 64-bit value."""
    if y.dtype is torch.bfloat16:
        tol = tol + (want.abs() + tol) * HALF[torch.bfloat16]
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), (what, float((err - tol).max()), float(err.max()))
