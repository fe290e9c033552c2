"""Plain 64-bit implementation (numpy) of the attention half of a decoder
layer: residual norm, e4m3 quantisation and product, rotary positions, the
paged cache and attention over it.  Shares no code with libpw; test-only.

16-bit inputs come as float64 arrays (their values are exact there), 8-bit
codes as uint8.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -100
GROUP = 128


# ---------------------------------------------------------------- e4m3
def e4m3_values() -> np.ndarray:
    """The 256 values: sign, 4 exponent bits with bias 7, 3 mantissa bits;
    0x7F and 0xFF are NaN, there are no infinities."""
    out = np.empty(256)
    for code in range(256):
        s, e, m = code >> 7, (code >> 3) & 15, code & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[code] = math.nan if e == 15 and m == 7 else (-v if s else v)
    return out


def e4m3_decode(codes: np.ndarray) -> np.ndarray:
    return e4m3_values()[codes]


def e4m3_step(v: np.ndarray) -> np.ndarray:
    """Distance of neighbouring e4m3 values at magnitude |v| (<= 448)."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    return 2.0 ** (e - 3)


def group_scales(y: np.ndarray, block_rows: int) -> np.ndarray:
    rows, cols = y.shape
    r, c = -(-rows // block_rows), -(-cols // GROUP)
    out = np.empty((r, c))
    for i in range(r):
        for j in range(c):
            out[i, j] = np.abs(y[i * block_rows:(i + 1) * block_rows, j * GROUP:(j + 1) * GROUP]).max()
    return np.maximum(out / E4M3_MAX, MIN_SCALE)


def spread(scale: np.ndarray, shape, block_rows: int) -> np.ndarray:
    return np.repeat(np.repeat(scale, block_rows, 0)[: shape[0]], GROUP, 1)[:, : shape[1]]


# ---------------------------------------------------------------- norm, product
def add_rmsnorm(x, weight, eps, residual=None):
    """(r, y)"""
    r = x if residual is None else x + residual
    return r, r / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps) * weight


def fp8_linear(a_codes, a_scale, b_codes, b_scale):
    """(y, the sum of the terms' magnitudes)"""
    a = e4m3_decode(a_codes) * spread(a_scale, a_codes.shape, 1)
    b = e4m3_decode(b_codes) * spread(b_scale, b_codes.shape, GROUP)
    return a @ b.T, np.abs(a) @ np.abs(b).T


# ---------------------------------------------------------------- rotary positions
def frequencies(d, base, kind="plain", scale=1.0, original=0.0, fast=0.0, slow=0.0):
    """(radians per position of each pair, factor)"""
    i = np.arange(d // 2)
    if kind == "ntk":
        base = base * scale ** (d / (d - 2))
    f = base ** (-2.0 * i / d)
    if kind == "linear":
        return f / scale, 1.0
    if kind == "yarn":
        pair = lambda n: d * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), d - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        return f / scale * ramp + f * (1 - ramp), 0.1 * math.log(scale) + 1
    if kind == "bands":
        turns = original * f / (2 * math.pi)
        keep = np.clip((turns - slow) / (fast - slow), 0, 1)
        return f / scale * (1 - keep) + f * keep, 1.0
    return f, 1.0


def rotate(x, pos, freq, factor, interleaved):
    """x [tokens][heads][d]; pos [tokens] (python ints are exact in 64 bits for
    the angles tested)."""
    rd = 2 * len(freq)
    i = np.arange(len(freq))
    u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + len(freq))
    angle = pos[:, None].astype(np.float64) * freq[None, :]
    c, s = np.cos(angle)[:, None] * factor, np.sin(angle)[:, None] * factor
    y = x.copy()
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., u] * s + x[..., v] * c
    assert rd <= x.shape[-1]
    return y


# ---------------------------------------------------------------- paged cache
def token_positions(q_offsets, kv_lens):
    """[(sequence, position)] of every new token."""
    return [(b, int(kv_lens[b]) - int(q_offsets[b + 1] - q_offsets[b]) + i)
            for b in range(len(kv_lens)) for i in range(int(q_offsets[b + 1] - q_offsets[b]))]


def attention(q, k_cache, v_cache, page_table, q_offsets, kv_lens, scale, causal=True, window=0):
    """(out, lse, sum p|v|, largest sum |q||k| scale of a row): the last two
    are what error bounds are made of."""
    T, H, D = q.shape
    ps, hk = k_cache.shape[1], k_cache.shape[2]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, dots = np.full((T, H), -np.inf), np.zeros((T, H))
    for b in range(len(kv_lens)):
        n, t0 = int(kv_lens[b]), int(q_offsets[b])
        m = int(q_offsets[b + 1]) - t0
        for i in range(m):
            pos = n - m + i
            hi = min(n, pos + 1) if causal else n
            lo = max(0, pos - window + 1) if causal and window else 0
            keys = range(lo, hi)
            if len(keys) == 0:
                continue
            at = np.array([int(page_table[b][j // ps]) * ps + j % ps for j in keys])
            k = k_cache.reshape(-1, hk, D)[at]
            v = v_cache.reshape(-1, hk, D)[at]
            for h in range(H):
                kh, vh = k[:, h // (H // hk)], v[:, h // (H // hk)]
                s = kh @ q[t0 + i, h] * scale
                top = s.max()
                e = np.exp(s - top)
                out[t0 + i, h] = e @ vh / e.sum()
                mag[t0 + i, h] = e @ np.abs(vh) / e.sum()
                lse[t0 + i, h] = top + math.log(e.sum())
                dots[t0 + i, h] = (np.abs(kh) @ np.abs(q[t0 + i, h])).max() * abs(scale)
    return out, lse, mag, dots
