"""Single-token steps beside the rounds, in float64 -- oracle side.

TEST INFRASTRUCTURE ONLY (see the package docstring).

A token that arrives while its unit is being written runs the same block as a
round's chunks: a dense layer, the rotary embedding at the token's own position,
its K and V into the cache, attention over its node's key list as far as the list
is written. Tokens one by one are a reading of this library's own (the Wan-Streamer v0.2
page's smallest block is a streaming unit of many tokens), and the pages give
no formulas; each is the plain one.
"""
from __future__ import annotations

import math

import numpy as np

from . import quant
from .cache import key_entries

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activation(x, act):
    x = np.asarray(x, dtype=np.float64)
    if act == "none":
        return x
    # Each in the form that loses nothing where its factor of x is small.
    if act == "gelu_tanh":  # 0.5 (1 + tanh u) = 1 / (1 + e^(-2u))
        with np.errstate(over="ignore"):
            return x / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
    if act == "gelu_erf":
        return 0.5 * x * _erfc(-x / math.sqrt(2.0))
    if act == "silu":
        # x / (1 + e^-x), without overflow on either side
        e = np.exp(-np.abs(x))
        return np.where(x >= 0, x / (1.0 + e), x * e / (1.0 + e))
    raise ValueError(f"unknown activation {act!r}")


def linear_bias(a, w, bias=None, residual=None, act="none"):
    """act(a w^T + bias) + residual."""
    y = a @ w.T
    if bias is not None:
        y = y + bias
    y = activation(y, act)
    return y if residual is None else y + residual


def frequencies(head_dim, pairs, base, ladder):
    """(axis, radians per position step) of each of the d/2 pairs; axis -1:
    the pair is copied."""
    axis = np.full(head_dim // 2, -1)
    freq = np.zeros(head_dim // 2)
    p = 0
    for a, n in enumerate(pairs):
        for i in range(n):
            axis[p] = a
            freq[p] = base ** (-p / (head_dim // 2) if ladder == "ladder" else -i / n)
            p += 1
    return axis, freq


def rotary(x, positions, pairs, base=10000.0, layout="interleaved", ladder="axis", inverse=False):
    """x [rows][heads][d] turned by positions [rows][3]."""
    rows, _, d = x.shape
    axis, freq = frequencies(d, pairs, base, ladder)
    pos = np.asarray(positions, dtype=np.float64)
    t = np.where(axis >= 0, pos[:, np.maximum(axis, 0)] * freq, 0.0)
    c, s = np.cos(t)[:, None, :], np.sin(t)[:, None, :]
    if inverse:
        s = -s
    turn = (axis >= 0)[None, None, :]
    first = np.arange(d // 2) * 2 if layout == "interleaved" else np.arange(d // 2)
    second = first + 1 if layout == "interleaved" else first + d // 2
    a, b = x[..., first], x[..., second]
    out = np.empty_like(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        out[..., first] = np.where(turn, a * c - b * s, a)
        out[..., second] = np.where(turn, a * s + b * c, b)
    return out


class Fp8Entry:
    """An entry's K (or V) in an FP8 pool, written a few tokens at a time:
    codes [pages][H][128][d], scales [pages][H]."""

    def __init__(self, tokens, heads, d):
        n = -(-tokens // 128)
        self.codes = np.zeros((n, heads, 128, d), dtype=np.uint8)
        self.scales = np.ones((n, heads), dtype=np.float32)
        self.written = 0

    def write(self, first, x):
        """x [n][H][d], bf16 values as float64, at tokens first ..."""
        end = first + x.shape[0]
        for p in range(first // 128, -(-end // 128)):
            lo, hi = max(first, 128 * p), min(end, 128 * (p + 1))
            r0, r1 = lo - 128 * p, hi - 128 * p
            held = min(max(self.written - 128 * p, 0), 128)
            for h in range(x.shape[1]):
                codes, old = self.codes[p, h], self.scales[p, h]
                if held == 0:
                    codes[:] = 0
                keep = np.arange(128) < held
                keep[r0:r1] = False
                new = x[lo - first:hi - first, h].astype(np.float32)
                amax = np.float32(np.abs(new).max())
                want = np.float32(amax / np.float32(448.0))
                if (codes[keep] & 0x7F).any():
                    s = max(old, want)
                else:
                    s = want if amax > 0 else np.float32(1.0)
                if s != old:
                    back = (quant.e4m3_decode(codes[keep]).astype(np.float32) * old).astype(np.float32)
                    codes[keep] = quant.e4m3_encode((back / s).astype(np.float32))
                codes[r0:r1] = quant.e4m3_encode((new / s).astype(np.float32))
                self.scales[p, h] = s
        self.written = max(self.written, end)

    def values(self, tokens):
        """[tokens][H][d] float64: code * scale, not rounded again."""
        v = quant.e4m3_decode(self.codes) * self.scales[:, :, None, None].astype(np.float64)
        n, h, _, d = v.shape
        return v.transpose(0, 2, 1, 3).reshape(n * 128, h, d)[:tokens]


def token_attention(q, keys, values):
    """O [Hq][d], lse [Hq] and A [Hq][d] = the weighted mean of |V| (the scale of
    rounding errors in the weights) of one query token q [Hq][d] over keys,
    values [N][H][d]; Hq a multiple of H. No token: O = 0, lse = -inf."""
    hq, d = q.shape
    g = hq // keys.shape[1]
    o, a, lse = np.zeros((hq, d)), np.zeros((hq, d)), np.full(hq, -np.inf)
    if keys.shape[0] == 0:
        return o, lse, a
    for x in range(hq):
        s = keys[:, x // g] @ q[x] / math.sqrt(d)
        m = s.max()
        e = np.exp(s - m)
        o[x] = e @ values[:, x // g] / e.sum()
        a[x] = e @ np.abs(values[:, x // g]) / e.sum()
        lse[x] = m + math.log(e.sum())
    return o, lse, a


def node_tokens(node, policy, window, entries, prefix, own):
    """K and V [N][H][d] that a token of `node` sees: its key list, the own entry
    up to `own` tokens. ``entries`` maps (c, l) to (K, V)."""
    ks, vs = [], []
    lst = key_entries(node, policy, window, prefix is not None)
    for i, e in enumerate(lst):
        if i + 1 == len(lst) and own == 0:
            continue
        k, v = prefix if e == (-1, 0) else entries[e]
        n = own if i + 1 == len(lst) and own is not None else k.shape[0]
        ks.append(k[:n])
        vs.append(v[:n])
    if not ks:
        shape = (0,) + (next(iter(entries.values()))[0].shape[1:] if entries else (1, 1))
        return np.zeros(shape), np.zeros(shape)
    return np.concatenate(ks), np.concatenate(vs)
