"""Helpers of the training-step tests: tensors at odd offsets, their float64
values, and the bounds that the operators' arithmetic allows."""

from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24                       # half a unit in the last place, relative
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}   # half the smallest subnormal


def torch_dtype(name):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "u8": torch.uint8}[name]


def on_device(values, dtype, offset=0):
    """A flat tensor of these values, starting `offset` elements into its allocation."""
    import torch

    values = np.ascontiguousarray(values)
    whole = torch.zeros(values.size + offset + 3, dtype=torch_dtype(dtype), device="cuda")
    got = whole[offset:offset + values.size]
    got.copy_(torch.from_numpy(values))
    return got


def f64(t):
    return t.detach().double().cpu().numpy()


def f32(t):
    return t.detach().float().cpu().numpy()


def rounded(x, dtype):
    """How far one rounding to `dtype` moves x at most."""
    return np.abs(x) * UNIT[dtype] + TINY[dtype]


def adamw_bound(p, g, m, v, *, step, lr, betas, eps, factor):
    """Bound on a float32 AdamW step's parameter error, against float64.

    Counting half-ulp relative errors u: the factor has 5 (norm * scale, + 1e-6
    with its constant, /, * scale), g' 6, so m' is off by at most
    (6 + 3) u (|beta1 m| + |(1 - beta1) g'|) (constants, products, sum), and v',
    a sum of non-negative terms, by 2 * 6 + 4 = 16 u; its root by 8 + 1 u, times
    the correction (2 u) 11 u, plus eps 13 u; the quotient adds 1 u (3 u with
    an approximate reciprocal and root), the step size 2 u: together
    lr-scaled (9 A + 18 |m'|) / d u with A the terms' magnitudes.  The parameter
    itself has its decay (2 u) and the difference (1 u).
    """
    g = factor * g
    a = np.abs(betas[0] * m) + np.abs((1 - betas[0]) * g)
    v = betas[1] * v + (1 - betas[1]) * g * g
    d = np.sqrt(v / (1 - betas[1] ** step)) + eps
    size = lr / (1 - betas[0] ** step)
    with np.errstate(all="ignore"):
        off = np.where(d > 0, size * 27 * a / d, 0.0)
        moved = np.where(d > 0, size * a / d, 0.0)
    return U32 * (3 * (np.abs(p) + moved) + off) + 2.0 ** -149


def norm_bound(values):
    """The norm: float64 sums of n exact squares, then one rounding to float32 (and a subnormal's)."""
    return values * 2.0 ** -23 + 2.0 ** -149
