"""The 4-bit cache and the sampler in float64 NumPy, from their definitions in include/wpk.h
(tests only; shares no code with the kernels)."""
from __future__ import annotations

import numpy as np


def bf16_floor(x):
    """The largest bf16 number <= x."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.floor(m * 256), e - 8)


def bf16_near(x):
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256), e - 8)


def quantise(x):
    """(codes, s, z) of the rows of x (last axis)."""
    x = np.asarray(x, dtype=np.float64)
    z = bf16_floor(x.min(-1))
    s = bf16_near((x.max(-1) - z) / 15.0)
    d = np.where(s > 0, s, 1.0)[..., None]
    c = np.where(s[..., None] > 0, np.clip(np.rint((x - z[..., None]) / d), 0, 15), 0.0)
    return c, s, z


def held(x):
    """What the cache holds for rows x."""
    c, s, z = quantise(x)
    return c * s[..., None] + z[..., None]


def rotate(x, pos, table):
    """Rows x [n, heads, hd] at positions pos, by the fp32 (cos, sin) table."""
    h = x.shape[-1] // 2
    cs = np.asarray(table, dtype=np.float64)[pos]
    co, si = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = x[..., :h], x[..., h:]
    return np.concatenate([a * co - b * si, b * co + a * si], -1)


def attention(q, k, v, pos0, scale):
    """q [n, heads, hd] at positions pos0 .. over keys k, v [len, kv, hd]; (out, sum p (s c + |z|) of the rows'
    parts v = s c + z, sum |q||k| scale).  z is taken as the least value of a row, as it is where a
    row's range is not tiny against its values (code 0 is then in use)."""
    n, heads, hd = q.shape
    group = heads // k.shape[1]
    out, bulk = np.zeros_like(q), np.zeros_like(q)
    reach = np.zeros((n, heads))
    for i in range(n):
        upto = pos0 + i + 1
        for h in range(heads):
            kk, vv = k[:upto, h // group], v[:upto, h // group]
            if len(kk) == 0:
                continue
            a = kk @ q[i, h] * scale
            p = np.exp(a - a.max())
            p /= p.sum()
            out[i, h] = p @ vv
            z = vv.min(-1, keepdims=True)
            bulk[i, h] = p @ (vv - z + np.abs(z))
            reach[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return out, bulk, reach


def sample_row(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log-probability, kept ids) of one row."""
    z = np.asarray(z, dtype=np.float64)
    if np.isnan(z).any() or (z == np.inf).any() or not (z > -np.inf).any():
        return -1, np.nan, np.array([], dtype=int)
    if not temperature > 0:
        return int(np.argmax(z)), 0.0, np.array([int(np.argmax(z))])
    ids = np.flatnonzero(z > -np.inf)
    ids = ids[np.argsort(-z[ids], kind="stable")]
    t = (z[ids] - z.max()) / temperature
    w = np.exp(t)
    if top_k > 0:
        ids, w, t = ids[:top_k], w[:top_k], t[:top_k]
    if top_p < 1:
        n = max(1, int(np.searchsorted(np.cumsum(w), max(top_p, 0.0) * w.sum(), side="left")) + 1)
        ids, w, t = ids[:n], w[:n], t[:n]
    if min_p > 0:
        on = w >= min(min_p, 1.0)
        ids, w, t = ids[on], w[on], t[on]
    o = np.argsort(ids)
    cum = np.cumsum(w[o])
    j = min(int(np.searchsorted(cum, min(max(u, 0.0), 1.0) * cum[-1], side="right")), len(o) - 1)
    return int(ids[o][j]), float(t[o][j] - np.log(cum[-1])), ids[o]
