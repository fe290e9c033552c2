"""Plain 64-bit implementation (numpy) of the operators around the attention
half: norms on both sides of a block, log probabilities of next tokens.  Shares
no code with libpw; test-only.  16-bit inputs come as float64 arrays.
"""
from __future__ import annotations

import numpy as np


def norm_add_norm(x, residual, eps, post_weight=None, weight=None, gate=None, residual_scale=1.0, block_scale=1.0):
    """(r, y, the sum of the magnitudes of r's two terms); y is None without a weight."""
    u = x
    if post_weight is not None:
        u = x / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps) * post_weight
    u = block_scale * u * (1.0 if gate is None else gate)
    r = residual_scale * residual + u
    y = None
    if weight is not None:
        y = r / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps) * weight
    return r, y, np.abs(residual_scale * residual) + np.abs(u)


def token_logprobs(logits, targets, top, scale):
    """(logprobs, lse, entropy, top_ids, top_logprobs) of rows without NaN or +inf."""
    rows, vocab = logits.shape
    z = scale * logits
    m = z.max(axis=1, keepdims=True)
    safe = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(z - safe)
    s = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = safe + np.log(s)
    lp = np.where(np.isneginf(z), -np.inf, z - np.where(np.isneginf(lse), 0.0, lse))
    p = np.exp(lp)
    entropy = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum(axis=1)
    out = np.full(targets.shape, np.nan)
    for i in range(rows):
        for j, t in enumerate(targets[i]):
            out[i, j] = 0.0 if t < 0 else lp[i, t] if t < vocab else np.nan
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top]
    return out, lse[:, 0], entropy, ids, np.take_along_axis(lp, ids, axis=1)


def activation(g, kind):
    """(act(g), the magnitude of its exponent's argument)"""
    t = g if kind == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    e = np.exp(-np.abs(t))
    return g * np.where(t >= 0, 1, e) / (1 + e), np.abs(t)
