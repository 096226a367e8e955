"""The training-step operators from their definitions: global gradient norm,
AdamW with float32 or packed states, layer norm with its gradient.

Plain NumPy, sharing no code with the library.  ``*_f32`` functions round
after every operation, as the operator is specified to do, so their results
can be compared bit for bit; the others work in float64.
"""

from __future__ import annotations

import math

import numpy as np

STATE_BLOCK = 256
M32 = 0xFFFFFFFF


def grad_norm(grads) -> float:
    """sqrt of the sum of squares over every element, scaled so that no square overflows float64."""
    xs = [np.asarray(g, dtype=np.float64).ravel() for g in grads]
    x = np.concatenate(xs) if xs else np.zeros(0)
    if x.size == 0:
        return 0.0
    if np.isnan(x).any():
        return math.nan
    top = float(np.abs(x).max())
    if top == 0.0 or math.isinf(top):
        return top
    return top * math.sqrt(math.fsum((x / top) ** 2))


# --------------------------------------------------------------------------
# AdamW
# --------------------------------------------------------------------------

def factor_f32(norm, max_norm=0.0, grad_scale=1.0):
    """What the gradients are multiplied with, in float32."""
    f = np.float32
    if max_norm <= 0:
        return f(grad_scale)
    with np.errstate(all="ignore"):
        r = f(max_norm) / (f(norm) * f(grad_scale) + f(1e-6))
        return f(grad_scale) * (f(1) if r > 1 else r)


def moments_f32(g, m, v, betas, factor):
    """New float32 moments, rounded after every operation."""
    f = np.float32
    with np.errstate(all="ignore"):
        g = f(factor) * g.astype(f)
        m = m * f(betas[0]) + g * f(1 - betas[0])
        v = v * f(betas[1]) + (g * g) * f(1 - betas[1])
    return m, v


def adamw(p, g, m, v, *, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, factor=1.0):
    """One step in float64 on float64 values: (p, m, v)."""
    p, g, m, v = (np.asarray(a, dtype=np.float64) for a in (p, g, m, v))
    g = float(factor) * g
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    mhat, vhat = m / (1 - betas[0] ** step), v / (1 - betas[1] ** step)
    p = p - lr * weight_decay * p - lr * mhat / (np.sqrt(vhat) + eps)
    return p, m, v


# --------------------------------------------------------------------------
# packed states
# --------------------------------------------------------------------------

def code_values(kind: str) -> np.ndarray:
    """The 256 codes' values at scale 1, from the format's statement."""
    out = np.zeros(256)
    for c in range(256):
        if kind == "exp_avg":
            e, f = (c >> 3) & 15, c & 7
            x = (1 + f / 8) * 2.0 ** (e - 15) if e else f / 8 * 2.0 ** -14
            out[c] = -x if c & 128 else x
        else:
            e, f = c >> 3, c & 7
            out[c] = (1 + f / 8) * 2.0 ** (e - 31) if e else f / 8 * 2.0 ** -30
    return out


def blocks_of(n: int) -> int:
    return (n + STATE_BLOCK - 1) // STATE_BLOCK


def unpack(codes, scales, kind: str) -> np.ndarray:
    """float64 values of codes and scale bytes."""
    codes = np.asarray(codes)
    e = np.repeat(np.asarray(scales).astype(np.int64), STATE_BLOCK)[:codes.size]
    scale = np.where(e == 255, np.nan, np.exp2(np.maximum(e, 1).astype(np.float64) - 127))
    return code_values(kind)[codes] * scale


def _mix(x):
    x = np.asarray(x, dtype=np.uint64) & M32
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x7FEB352D)) & np.uint64(M32)
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0x846CA68B)) & np.uint64(M32)
    return x ^ (x >> np.uint64(16))


def random_bits(seed: int, tensor: int, n: int) -> np.ndarray:
    """The 32 random bits of each element of a tensor."""
    key = int(_mix((seed + 0x9E3779B9 * (tensor + 1)) & M32))
    i = np.arange(n, dtype=np.uint64) & np.uint64(M32)
    return _mix((np.uint64(key) + i * np.uint64(0x9E3779B9)) & np.uint64(M32))


def pack(x, bits, kind: str):
    """Codes and scale bytes of float32 values, with the random bits of their elements.

    In float64 arithmetic on the values' place between two codes; the place
    of a value below a code's last bit is cut to float32's 20 bits there, as
    the operator states the noise in units of it.
    """
    x = np.asarray(x, dtype=np.float32)
    n = x.size
    codes, scales = np.zeros(n, np.uint8), np.zeros(blocks_of(n), np.uint8)
    noise = ((bits & np.uint64(0xFFFF)) if kind == "exp_avg" else (bits >> np.uint64(16))).astype(np.float64)
    up = (noise * 16 + 8) / 2.0 ** 20
    bias = 15 if kind == "exp_avg" else 31
    for b in range(scales.size):
        s = slice(b * STATE_BLOCK, min(n, (b + 1) * STATE_BLOCK))
        top = float(np.abs(x[s]).max()) if not np.isnan(x[s]).any() else math.nan
        e = 255
        if math.isfinite(top):
            e = 1
            while e < 255 and 1.875 * 2.0 ** (e - 127) < top:
                e += 1
        scales[b] = e
        if e == 255:
            continue
        for i in range(s.start, s.stop):
            # a multiple of float32's smallest after scaling, as float32 keeps it
            y = float(np.float32(np.float32(abs(float(x[i])) * 2.0 ** (127 - e)) * np.float32(2.0 ** -(127 - bias))))
            if y == 0.0:
                code = 0 if kind == "exp_avg" else int(up[i] >= 1)
            else:
                place = max(math.frexp(y)[1] - 1, -126)          # exponent of y, or of the subnormals
                step = 2.0 ** (place - 3)
                units = y / step                                  # below 8: subnormal codes
                whole = math.floor(units + up[i])
                field = place + 127
                code = (field - 1) * 8 + whole if field > 1 or whole >= 8 else whole
            if kind == "exp_avg":
                code |= 128 if np.signbit(x[i]) else 0
            elif code == 0 and x[i] > 0:
                code = 1
            codes[i] = code
    return codes, scales


# --------------------------------------------------------------------------
# layer norm
# --------------------------------------------------------------------------

def layer_norm(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd) in float64."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, dtype=np.float64)
    if beta is not None:
        y = y + np.asarray(beta, dtype=np.float64)
    return y, mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta) in float64 from the given statistics."""
    dy, x, mean, rstd = (np.asarray(a, dtype=np.float64) for a in (dy, x, mean, rstd))
    h = (x - mean[:, None]) * rstd[:, None]
    w = dy if gamma is None else dy * np.asarray(gamma, dtype=np.float64)
    dx = rstd[:, None] * (w - w.mean(1, keepdims=True) - h * (w * h).mean(1, keepdims=True))
    return dx, (dy * h).sum(0), dy.sum(0)
