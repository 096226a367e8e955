"""The operators at a model's ends from their definitions: the embedding and
its gradient, activations in 8 bits.

Plain NumPy, sharing no code with the library; float64 unless a name says
otherwise.
"""

from __future__ import annotations

import math

import numpy as np

ACTIVATION_BLOCK = 32


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------

def embedding(tokens, table, scale=1.0):
    """scale * the table's row of each token; NaN for a token outside the table."""
    table = np.asarray(table, dtype=np.float64)
    out = np.full((len(tokens), table.shape[1]), np.nan)
    for i, t in enumerate(tokens):
        if 0 <= t < table.shape[0]:
            out[i] = table[t] * scale
    return out


def embedding_backward(dy, tokens, vocab, scale=1.0, padding=None, held=None):
    """(the table's gradient, the sum of its terms' magnitudes, how many terms each row has).

    `held`: what the gradient is added to; else rows without a token are 0.
    """
    dy = np.asarray(dy, dtype=np.float64)
    got = np.zeros((vocab, dy.shape[1])) if held is None else np.array(held, dtype=np.float64)
    size, terms = np.abs(got), np.zeros(vocab, np.int64)
    for i, t in enumerate(tokens):
        if 0 <= t < vocab and t != padding:
            got[t] += scale * dy[i]
            size[t] += np.abs(scale * dy[i])
            terms[t] += 1
    return got, size, terms


# --------------------------------------------------------------------------
# activations in 8 bits
# --------------------------------------------------------------------------

def pack_activations(x):
    """(codes int8, scale bytes) of [rows, cols] values that float32 holds."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    blocks = -(-cols // ACTIVATION_BLOCK)
    codes, scales = np.zeros((rows, cols), np.int8), np.zeros((rows, blocks), np.uint8)
    for r in range(rows):
        for b in range(blocks):
            part = x[r, b * ACTIVATION_BLOCK:(b + 1) * ACTIVATION_BLOCK]
            top = np.abs(part).max()
            e = 255
            if math.isfinite(top):
                e = 1
                while e < 255 and 127 * 2.0 ** (e - 133) < top:
                    e += 1
            scales[r, b] = e
            if e < 255:
                # np.rint rounds ties to even; the quotient by a power of two is exact
                codes[r, b * ACTIVATION_BLOCK:(b + 1) * ACTIVATION_BLOCK] = np.rint(part / 2.0 ** (e - 133))
    return codes, scales


def unpack_activations(codes, scales):
    """float64 values of codes and scale bytes."""
    e = np.repeat(np.asarray(scales).astype(np.int64), ACTIVATION_BLOCK, axis=1)[:, :codes.shape[1]]
    scale = np.where(e == 255, np.nan, np.exp2(np.maximum(e, 1).astype(np.float64) - 133))
    return codes.astype(np.float64) * scale


# --------------------------------------------------------------------------
# cross entropy
# --------------------------------------------------------------------------

def cross_entropy(x, weight, targets, ignore=-100):
    """(loss, lse) of every row's logits x W^T."""
    z = np.asarray(x, dtype=np.float64) @ np.asarray(weight, dtype=np.float64).T
    with np.errstate(all="ignore"):
        top = z.max(1)
        lse = top + np.log(np.exp(z - top[:, None]).sum(1))
    loss = np.full(len(targets), np.nan)
    for i, t in enumerate(targets):
        if t == ignore:
            loss[i] = 0.0
        elif 0 <= t < z.shape[1]:
            loss[i] = lse[i] - z[i, t]
    return loss, lse


def cross_entropy_backward(g, x, weight, targets, lse, ignore=-100):
    """(dx, dweight, dz) with dz = g (exp(z - lse) - onehot); ignored rows and rows of g = 0 take no part."""
    x, weight = np.array(x, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    g = np.asarray(g, dtype=np.float64)
    live = np.array([t != ignore for t in targets], dtype=bool) & (g != 0)
    x[~live] = 0
    dz = np.zeros((x.shape[0], weight.shape[0]))
    with np.errstate(all="ignore"):
        dz[live] = np.exp(x[live] @ weight.T - np.asarray(lse, dtype=np.float64)[live, None])
    for i, t in enumerate(targets):
        if live[i]:
            if 0 <= t < weight.shape[0]:
                dz[i, t] -= 1
            else:
                dz[i] = np.nan
    dz[live] *= g[live, None]
    return dz @ weight, dz.T @ x, dz
