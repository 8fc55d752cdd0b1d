"""fp64 references of the operators around the decode cache: rotary positions, the 4-bit KV
cache's quantiser, decode attention with the attention weight of every block, and eviction by
that weight.  Plain numpy, sharing no code with the CUDA path."""
from __future__ import annotations

import numpy as np

from .msa_oracle import _f64 as to_f64

GROUP = 32


def rope(x, positions, freqs, scale=1.0, interleaved=False, inverse=False, head_major=False):
    """x [B, S, H, d] (or [B, H, S, d] with head_major); positions int [B, S]; freqs: turns per
    position in units of 2^-64 turns, one per pair."""
    x = to_f64(x)
    f = np.array([int(v) % (1 << 64) for v in np.asarray(freqs).reshape(-1).tolist()], dtype=object)
    p = np.asarray(positions).astype(object)[..., None]
    phase = ((p * f) % (1 << 64)).astype(object)                   # exact, one turn = 2^64
    turns = (phase / float(1 << 64)).astype(np.float64)
    angle = 2 * np.pi * turns * (-1 if inverse else 1)
    w = scale * (np.cos(angle) + 1j * np.sin(angle))               # [B, S, n]
    w = w[:, None] if head_major else w[:, :, None]
    n = f.shape[0]
    y = x.copy()
    if interleaved:
        z = (x[..., 0:2 * n:2] + 1j * x[..., 1:2 * n:2]) * w
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
    else:
        z = (x[..., :n] + 1j * x[..., n:2 * n]) * w
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y


def round_bf16(x):
    """fp32 array rounded to bf16 (nearest even), as fp32."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    nan = np.isnan(np.asarray(x, dtype=np.float32))
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(nan, np.float32(np.nan), r)


def pack_values(x):
    """What the 4-bit cache holds for rows x [..., d]: (values fp64, step, mid), each group of
    32 dims by the definition's single-precision operations."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], np.float32(0), g)
    hi, lo = g.max(-1), g.min(-1)
    f = np.float32(1 / 15)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        step = round_bf16(np.float32(hi * f) - np.float32(lo * f))
        step = np.where(step < np.float32(2.0 ** -100), np.float32(0), step)
        mid = round_bf16(lo + np.float32(8) * step)
        inv = np.where(step > 0, np.float32(1) / step, np.float32(0)).astype(np.float32)
        t = (g - mid[..., None]).astype(np.float32) * inv[..., None]
        code = np.clip(np.rint(t.astype(np.float32)) + np.float32(8), 0, 15)
        code = np.where(step[..., None] > 0, code, 8)
    mid = np.where(bad, np.nan, mid.astype(np.float64))
    step = np.where(bad, 0.0, step.astype(np.float64))
    value = mid[..., None] + (code.astype(np.float64) - 8) * step[..., None]
    return value.reshape(x.shape), step, mid


def record_offsets(d, is_v):
    """Byte offset and half (0 low, 1 high) of the code of (key, dim), each [128, d]."""
    key, dim = np.arange(128)[:, None], np.arange(d)[None, :]
    ng, g, i = d // GROUP, dim // GROUP, dim % GROUP
    if is_v:
        r, i = i // 4, i % 4
        pair = (key // 2) ^ (4 * (r % (2 if d == 128 else 4)))
        byte = (r * 128 + 2 * pair + key % 2) * 2 * ng + g * 2 + i // 2
    else:
        c, i = i // 8, i % 8
        byte = key * (d // 2) + c * 4 * ng + g * 4 + i // 2
    return byte, np.broadcast_to(i % 2, byte.shape)


def record_values(rec, d, is_v):
    """Values [128, d] of the bytes of one block's K or V record."""
    rec = np.asarray(rec, dtype=np.uint8)
    byte, half = record_offsets(d, is_v)
    code = (rec[byte] >> (4 * half)) & 15
    planes = (rec[64 * d:].view(np.uint16).astype(np.uint32) << 16).view(np.float32)
    at = np.arange(d)[None, :] // GROUP * 128 + np.arange(128)[:, None]
    return planes[4 * d + at].astype(np.float64) + (code.astype(np.float64) - 8) * planes[at]


def decode_mass(q, k, v, sel, lens, block_size=128, sm_scale=None):
    """Decode attention of q [B, 1, Hq, d] over per-sequence caches k, v (lists of [Hkv, >= L, d])
    and the attention weight of every selected block: out, lse [B, Hq, 1], and weight
    [B, Hkv, nB] with nB blocks for the longest cache."""
    q = to_f64(q)
    B, _, Hq, d = q.shape
    Hkv = sel.shape[1]
    G = Hq // Hkv
    scale = d ** -0.5 if not sm_scale else sm_scale
    nB = max(1, max(-(-int(x) // block_size) for x in lens))
    out, lse = np.zeros((B, 1, Hq, d)), np.full((B, Hq, 1), -np.inf)
    mass = np.zeros((B, Hkv, nB))
    for b in range(B):
        L = int(lens[b])
        for g in range(Hkv):
            blocks = [int(x) for x in np.asarray(sel)[b, g].reshape(-1) if 0 <= x < -(-L // block_size)]
            keys = [j for x in blocks for j in range(x * block_size, min(L, (x + 1) * block_size))]
            if not keys:
                continue
            kk, vv = to_f64(k[b][g])[keys], to_f64(v[b][g])[keys]
            for h in range(g * G, (g + 1) * G):
                z = scale * (kk @ q[b, 0, h])
                top = z.max()
                e = np.exp(z - top)
                lse[b, h, 0] = top + np.log(e.sum())
                p = e / e.sum()
                out[b, 0, h] = p @ vv
                np.add.at(mass[b, g], np.array(keys) // block_size, p)
    return out, lse, mass


def evict(mass, lens, keep, n_first, n_recent, block_size=128, table=None):
    """kept [B, keep], new lengths, mass and (if given) table after eviction."""
    mass = np.asarray(mass, dtype=np.float32)
    B, H, nB = mass.shape
    kept = np.full((B, keep), -1, dtype=np.int32)
    new_lens = np.zeros(B, dtype=np.int32)
    moved = np.zeros_like(mass)
    rows = None if table is None else np.array(table, dtype=np.int32)
    for b in range(B):
        L = min(max(int(lens[b]), 0), nB * block_size)
        n = -(-L // block_size)
        with np.errstate(invalid="ignore", over="ignore"):
            score = mass[b, 0].copy()
            for h in range(1, H):
                score = (score + mass[b, h]).astype(np.float32)
        must = [i for i in range(n) if i < n_first or i >= n - n_recent]
        rest = [i for i in range(n) if n_first <= i < n - n_recent]
        rest.sort(key=lambda i: (np.isnan(score[i]), 0.0 if np.isnan(score[i]) else -float(score[i]), i))
        stay = list(range(n)) if n <= keep else sorted(must + rest[:keep - len(must)])
        gone = [i for i in range(n) if i not in set(stay)]
        kept[b, :len(stay)] = stay
        new_lens[b] = L - block_size * len(gone)
        moved[b, :, :len(stay)] = mass[b][:, stay]
        if rows is not None:
            rows[b, :n] = np.asarray(table)[b][stay + gone]
    return kept, new_lens, moved, rows
