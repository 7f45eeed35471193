"""Float64 restatement of what a serving step does around the packed linears, from its formulas: rotary
positions, low-rank adapters of many requests, and the logits' penalties, biases and grammar masks.  NumPy and
whole numbers only; shares nothing with the library.

The rotary and adapter functions also return the magnitudes from which the tests derive their tolerances.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

# 2 pi to 60 decimals, so that whole turns of positions up to 2^31 leave an angle of more than 53 bits
TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


def rotary_freqs(R, base, scaling="none", factor=1.0, original=0.0, beta_fast=32.0, beta_slow=1.0):
    """(radians a token of each pair, amplitude)."""
    i = np.arange(R // 2, dtype=np.float64)
    if scaling == "base":
        base = base * factor ** (R / (R - 2))
    f = base ** (-2 * i / R)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling != "parts":
        return f, 1.0
    number = [R * math.log(original / (2 * math.pi * beta)) / (2 * math.log(base)) for beta in (beta_fast, beta_slow)]
    low, high = max(math.floor(number[0]), 0), min(math.ceil(number[1]), R - 1)
    out = np.empty_like(f)
    for n in range(R // 2):
        ramp = min(max((n - low) / max(high - low, 1e-3), 0.0), 1.0)
        out[n] = ramp * f[n] / factor + (1 - ramp) * f[n]
    return out, 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def angle(pos, f):
    """pos * f without its whole turns, in (-pi, pi]: exact but for the last rounding."""
    a = Fraction(int(pos)) * Fraction(float(f))
    a -= TWO_PI * round(a / TWO_PI)
    return float(a)


def rotary(x, pos, freqs, amplitude, R, pairs, inverse=False):
    """x [T, H, D] turned; and amplitude * (|a| + |b|) of each element's pair (0 where it is copied)."""
    x = np.asarray(x, dtype=np.float64)
    y, size = x.copy(), np.zeros_like(x)
    n = R // 2
    at = [(2 * i, 2 * i + 1) if pairs else (i, i + n) for i in range(n)]
    for t in range(x.shape[0]):
        for i, (lo, hi) in enumerate(at):
            w = angle(pos[t], freqs[i]) * (-1 if inverse else 1)
            c, s = amplitude * math.cos(w), amplitude * math.sin(w)
            a, b = x[t, :, lo], x[t, :, hi]
            y[t, :, lo], y[t, :, hi] = a * c - b * s, a * s + b * c
            size[t, :, lo] = size[t, :, hi] = amplitude * (np.abs(a) + np.abs(b))
    return y, size


def adapter_linear(x, a, b, scale, rank, row_start, adapter, y):
    """(out, S, H): out [T, N]; S = |scale| |B| sum |A x| in absolute terms, H = |scale| |B| |A x|."""
    x, a, b = (np.asarray(m, dtype=np.float64) for m in (x, a, b))
    out = np.asarray(y, dtype=np.float64).copy()
    S, H = np.zeros_like(out), np.zeros_like(out)
    for r, g in enumerate(adapter):
        if g < 0:
            continue
        n = a.shape[1] if rank is None else int(rank[g])
        rows = slice(row_start[r], row_start[r + 1])
        h = x[rows] @ a[g, :n].T
        out[rows] += float(scale[g]) * (h @ b[g, :, :n].T)
        w = abs(float(scale[g])) * np.abs(b[g, :, :n]).T
        S[rows] = (np.abs(x[rows]) @ np.abs(a[g, :n]).T) @ w
        H[rows] = np.abs(h) @ w
    return out, S, H


def logits_adjust(logits, row_start, history, hist_len, prompt_len=None, slot=None, fresh=None, tree=None, repetition=None,
                  presence=None, frequency=None, biases=None, mask=None, mask_row=None, dtype=np.float64):
    """Row by row in ``dtype``, one step after the other; biases: per request a list of (token, value)."""
    logits = np.asarray(logits)
    out = logits.astype(dtype)
    V = logits.shape[1]
    for b in range(len(row_start) - 1):
        row = b if slot is None else int(slot[b])
        past = [int(i) for i in history[row][: hist_len[b]]] if row >= 0 else []
        prompt = 0 if prompt_len is None else int(prompt_len[b])
        n = row_start[b + 1] - row_start[b]
        for i in range(n):
            t = row_start[b] + i
            path = []
            if fresh is not None:
                path = [int(fresh[row_start[b] + j]) for j in range(n) if (j <= i if tree is None else int(tree[t]) >> j & 1)]
            known = {v for v in past + path if 0 <= v < V}
            made = {}
            for v in past[prompt:] + path:
                if 0 <= v < V:
                    made[v] = made.get(v, 0) + 1
            with np.errstate(all="ignore"):
                for v in known:
                    if repetition is not None:
                        r = dtype(repetition[b])
                        out[t, v] = out[t, v] / r if out[t, v] > 0 else out[t, v] * r
                for v, c in made.items():
                    f = dtype(0 if frequency is None else frequency[b])
                    out[t, v] = (out[t, v] - f * dtype(c)) - dtype(0 if presence is None else presence[b])
                for v, value in dict(biases[b]).items() if biases is not None else ():
                    if 0 <= v < V:
                        out[t, v] = out[t, v] + dtype(value)
            if mask is not None:
                m = t if mask_row is None else int(mask_row[t])
                if m >= 0:
                    words = np.asarray(mask[m]).view(np.uint32)
                    bits = (words[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1
                    out[t, bits == 0] = -np.inf
    return out
