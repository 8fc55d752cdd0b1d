"""fp64 references of a decode step over a tree of drafted tokens: paths and positions, the 8-bit
index-key quantiser, index scores, selection, attention and the commit of accepted tokens.  Plain
numpy, sharing no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np

from .msa_oracle import _f64 as to_f64


def paths(parents, length, capacity):
    """The tokens' paths (lists, root first; empty for an absent token) of one sequence."""
    out = []
    for i, p in enumerate(parents):
        if p == -1:
            path = [i]
        elif 0 <= p < i and out[p]:
            path = out[p] + [i]
        else:
            path = []
        if path and length + len(path) - 1 >= capacity:
            path = []
        out.append(path)
    return out


def word(path):
    return sum(1 << a for a in path)


def e4m3_values():
    """The 127 finite non-negative values of the 8-bit float, ascending; index = code."""
    v = []
    for code in range(127):
        e, f = code >> 3, code & 7
        v.append(math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10))
    return np.array(v)


_E4M3 = e4m3_values()


def quantise(x):
    """Rows x [..., d] -> (codes uint8, exponent bytes uint8 [...], values fp64)."""
    x = to_f64(x)
    bad = ~np.isfinite(x).all(-1)
    y = np.where(bad[..., None], 0.0, x)
    amax = np.abs(y).max(-1)
    e = np.full(amax.shape, -126)
    for _ in range(300):
        e = np.where(np.ldexp(448.0, e) < amax, e + 1, e)
    t = np.abs(np.ldexp(y, -e[..., None]))
    hi = np.clip(np.searchsorted(_E4M3, t), 0, 126)             # first value >= t
    lo = np.clip(hi - 1, 0, 126)
    dh, dl = _E4M3[hi] - t, t - _E4M3[lo]
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    code = np.where(t == _E4M3[hi], hi, code)
    val = np.copysign(np.ldexp(_E4M3[code], e[..., None]), y)
    code = code + np.where(np.signbit(y), 128, 0)
    code = np.where(bad[..., None], 127, code)
    val = np.where(bad[..., None], np.nan, val)
    return code.astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8), val


def scores(q, keys, draft_keys, path_lists, length, block, n_blocks, scale):
    """q [N, H, d], keys [>= length, d], draft_keys [N, d] -> [H, N, n_blocks]."""
    q, keys, kd = to_f64(q), to_f64(keys)[:length], to_f64(draft_keys)
    n, h, _ = q.shape
    out = np.full((h, n, n_blocks), -np.inf)
    for i, path in enumerate(path_lists):
        if not path:
            continue
        pos = np.concatenate([np.arange(length), length + np.arange(len(path))])
        k = np.concatenate([keys, kd[path]]) if length else kd[path]
        z = scale * (q[i] @ k.T)
        for blk in np.unique(pos // block):
            out[:, i, blk] = z[:, pos // block == blk].max(1)
    return out


def select(score_row, position, block, top_k):
    """One token's selection from its scores [n_blocks]: (list of blocks, -1 padded)."""
    if position < 0:
        return [-1] * top_k
    cur = position // block
    order = sorted(range(cur), key=lambda j: (-(score_row[j] + 0.0), j))
    got = sorted(order[:top_k - 1] + [cur])
    return got + [-1] * (top_k - len(got))


def attend(q, k, v, kd, vd, path, length, sel, block, scale):
    """One token and KV head: q [G, d]; k, v [>= length, d]; kd, vd [N, d] -> out [G, d], lse [G]."""
    q = to_f64(q)
    pos = np.concatenate([np.arange(length), length + np.arange(len(path))]).astype(np.int64)
    chosen = [s for s in sel if s >= 0]
    take = np.isin(pos // block, chosen)
    if not path or not take.any():
        return np.zeros_like(q), np.full(q.shape[0], -np.inf)
    kk = np.concatenate([to_f64(k)[:length], to_f64(kd)[path]])[take]
    vv = np.concatenate([to_f64(v)[:length], to_f64(vd)[path]])[take]
    z = scale * (q @ kk.T)
    top = z.max(1, keepdims=True)
    e = np.exp(z - top)
    s = e.sum(1, keepdims=True)
    return (e / s) @ vv, (top + np.log(s))[:, 0]
