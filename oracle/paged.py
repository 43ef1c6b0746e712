"""Float64 statement of the paged-cache operators, one sequence at a time on
dense arrays (slot j of a sequence is row j), with bounds for fp32 and bf16
arithmetic.  Test infrastructure only.

Readings: rotary pairs and scalings as in include/vx.h; query t of a chunk sits
at slot old + t and sees slot j < old + n iff j < prefix or i - window < j <= i.
"""
from __future__ import annotations

import math

import numpy as np


def rope_freqs(rot, theta=1e6, scaling="none", factor=1.0, orig_len=0, beta_fast=32.0, beta_slow=1.0, mscale=0.0):
    """(f_m [rot / 2], the factor on cosine and sine)."""
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = np.array([theta ** (-2.0 * m / rot) for m in range(rot // 2)])
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        g = np.clip((orig_len * f / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
        return g * f + (1 - g) * f / factor, (mscale or 0.1 * math.log(factor) + 1.0)
    return f, 1.0


def rope(x, pos, rot=0, interleaved=False, **scaling):
    """x [n, H, D], pos [n] -> rotated, float64."""
    x = np.asarray(x, dtype=np.float64)
    rot = rot or x.shape[-1]
    f, ms = rope_freqs(rot, **scaling)
    ang = np.asarray(pos, dtype=np.float64)[:, None, None] * f
    c, s = np.cos(ang) * ms, np.sin(ang) * ms
    y = x.copy()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def seen(old, n, window=0, prefix=0):
    """[n, old + n] truth values: query t sees slot j."""
    i = old + np.arange(n)[:, None]
    j = np.arange(old + n)[None, :]
    m = j <= i
    if window:
        m &= j > i - window
    return m | (j < prefix)


def attention(q, k, v, old, window=0, prefix=0, cap=0.0, slopes=None, scale=0.0):
    """q [n, Hq, D], k, v [old + n, Hkv, D] -> dict of o [n, Hq, D], lse [n, Hq], weights [Hkv, old + n] (summed over
    queries and the group), absv = softmax-weighted |v| [n, Hq, D], smax = the largest sum |q k| * scale of a row's
    visible keys [n, Hq].  Masked k and v are not read."""
    n, Hq, D = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    scale = scale or D ** -0.5
    m = seen(old, n, window, prefix)[:, :L]
    used = m.any(0)
    k = np.where(used[:, None, None], k, 0.0).astype(np.float64)
    v = np.where(used[:, None, None], v, 0.0).astype(np.float64)
    q = q.astype(np.float64)
    dist = np.abs(old + np.arange(n)[:, None] - np.arange(L)[None, :])
    o, absv = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, smax = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    w = np.zeros((Hkv, L))
    some = m.any(1)
    for h in range(Hq):
        kh = h // G
        s = q[:, h] @ k[:, kh].T * scale
        big = np.where(m, np.abs(q[:, h]) @ np.abs(k[:, kh]).T * scale, 0.0)
        if cap:
            s = cap * np.tanh(s / cap)
        if slopes is not None:
            s = s - slopes[h] * dist
        s = np.where(m, s, -np.inf)
        top = np.where(some, s.max(1, initial=-np.inf), 0.0)
        p = np.exp(s - top[:, None])
        z = p.sum(1)
        p = p / np.where(some, z, 1.0)[:, None]
        o[:, h] = p @ v[:, kh]
        absv[:, h] = p @ np.abs(v[:, kh])
        with np.errstate(divide="ignore"):
            lse[:, h] = np.where(some, top + np.log(z), -np.inf)
        smax[:, h] = big.max(1, initial=0.0)
        w[kh] += p.sum(0)
    return dict(o=o, lse=lse, weights=w, absv=absv, smax=smax)


def evict(acc, keep, recent):
    """acc [L] -> the kept slots in order: the last min(recent, m), and the m - r others of largest acc (ties: the
    lowest slot, NaN lowest), m = min(keep, L)."""
    L = len(acc)
    m = min(keep, L)
    r = min(recent, m)
    old = [(-math.inf if math.isnan(a) else float(a)) for a in acc[:L - r]]
    # NaN ranks below every number, -inf included
    order = sorted(range(L - r), key=lambda j: (not math.isnan(acc[j]), old[j], -j), reverse=True)
    return np.array(sorted(order[:m - r]) + list(range(L - r, L)), dtype=np.int64)
