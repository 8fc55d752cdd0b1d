"""Inputs of the tree tests: seeded caches whose rows past the lengths, unused blocks and absent
tokens hold garbage (NaN, or any byte), and the same data as the oracle sees it."""
from __future__ import annotations

import numpy as np
import torch

from block_sparse_gqa_02_gb300 import _lib
from oracle import tree_ops

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def random_parents(rng, batch, n, kind):
    p = np.empty((batch, n), dtype=np.int64)
    for b in range(batch):
        for i in range(n):
            if kind == "chain":
                p[b, i] = i - 1
            elif kind == "star":
                p[b, i] = -1
            elif kind == "bad":                 # absent tokens in between, parents out of range
                p[b, i] = rng.choice([-1, i - 1, rng.integers(-1, i + 1), -2, i, 99, -2 ** 31], p=[.2, .4, .2, .05, .05, .05, .05])
            else:
                p[b, i] = max(-1, i - 1 - rng.integers(0, 4))
    return p


class Tree:
    """One tree step's inputs on the GPU; rows as the oracle sees them in keys / k / v."""

    def __init__(self, lens, n, cap, hkv=4, group=16, dim=128, idim=128, block=128, topk=4, dtype="bf16",
                 paged=False, packed=True, kind="tree", seed=0, sel_frac=None, key_scale=1.0):
        rng = self.rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        dt = self.dt = DTYPES[dtype]
        B = len(lens)
        self.lens, self.n, self.cap, self.packed, self.paged = list(lens), n, cap, packed, paged
        self.shape = _lib.make_shape(B, n, cap, hkv * group, hkv, dim, idim, block, topk, 1, dtype)
        nB = self.nB = self.shape.n_blocks
        self.parents = random_parents(rng, B, n, kind)
        self.paths = [tree_ops.paths(self.parents[b], lens[b], cap) for b in range(B)]
        words = [[tree_ops.word(p) for p in row] for row in self.paths]
        self.mask = torch.tensor([[w - (1 << 64) if w >> 63 else w for w in row] for row in words]).cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.n_phys = B * nB + (3 if paged else 0)
        perm = rng.permutation(self.n_phys)[:B * nB].reshape(B, nB)
        self.phys = perm if paged else np.arange(B * nB).reshape(B, nB)
        self.table = torch.tensor(perm, dtype=torch.int32).cuda() if paged else None
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        nan = float("nan")
        there = torch.tensor([[bool(p) for p in row] for row in self.paths])
        # rows [B, H, cap, d] as the sequences have them
        self.k = (rand(B, hkv, cap, dim) * key_scale).to(dt)
        self.v = rand(B, hkv, cap, dim).to(dt)
        self.ik = (rand(B, cap, idim) * rand(B, cap, 1).exp()).to(dt)
        self.q = rand(B, n, hkv * group, dim).to(dt)
        self.iq = rand(B, n, hkv, idim).to(dt)
        self.kd = (rand(B, hkv, n, dim) * key_scale).to(dt)
        self.vd = rand(B, hkv, n, dim).to(dt)
        self.ikd = (rand(B, n, idim) * rand(B, n, 1).exp()).to(dt)
        q, iq, kd, vd, ikd = (x.clone() for x in (self.q, self.iq, self.kd, self.vd, self.ikd))
        q[~there], iq[~there], ikd[~there] = nan, nan, nan
        kd.transpose(1, 2)[~there] = nan
        vd.transpose(1, 2)[~there] = nan
        self.dev = dict(q=q.cuda(), iq=iq.cuda(), kd=kd.cuda(), vd=vd.cuda())
        full = lambda x: self._store(x, block, nan).cuda()  # noqa: E731
        self.dev["k"], self.dev["v"] = full(self.k), full(self.v)
        if packed:
            self.dev["ik"] = self._pack(self.ik, block).cuda()
            rec = torch.randint(0, 256, (B, 128 * (idim + 1)), generator=g, dtype=torch.uint8)
            codes, exps, val = tree_ops.quantise(self.ikd.float().numpy())
            rec[:, :n * idim] = torch.tensor(codes).reshape(B, -1)
            rec[:, 128 * idim:128 * idim + n] = torch.tensor(exps)
            self.dev["ikd"] = rec.cuda()
            self.ikd64 = val
            self.ik64 = tree_ops.quantise(self.ik.float().numpy())[2]
        else:
            self.dev["ik"], self.dev["ikd"] = full(self.ik), ikd.cuda()
            self.ikd64, self.ik64 = self.ikd.double().numpy(), self.ik.double().numpy()
        self.sel = self._selection(topk, sel_frac)
        self.dev["sel"] = torch.tensor(self.sel, dtype=torch.int32).cuda()

    def _store(self, x, block, fill):
        """Rows [B, (H,) cap, d] as a contiguous cache or pools, garbage past the lengths."""
        y = x.clone()
        for b, length in enumerate(self.lens):
            y[b, ..., length:, :] = fill
        if not self.paged:
            return y
        one = y.dim() == 3
        y = y.unsqueeze(1) if one else y
        B, H, cap, d = y.shape
        pad = torch.full((B, H, self.nB * block - cap, d), fill, dtype=y.dtype)
        y = torch.cat([y, pad], 2).view(B, H, self.nB, block, d).transpose(1, 2)
        pool = torch.full((self.n_phys, H, block, d), fill, dtype=y.dtype)
        pool[torch.tensor(self.phys).flatten()] = y.reshape(-1, H, block, d)
        return pool[:, 0].contiguous() if one else pool

    def _pack(self, x, block):
        B, cap, d = x.shape
        rec = torch.tensor(self.rng.integers(0, 256, (self.n_phys, 128 * (d + 1)), dtype=np.uint8))
        codes, exps, _ = tree_ops.quantise(x.float().numpy())
        for b, length in enumerate(self.lens):
            for j in range(-(-length // 128)):
                m = min(128, length - j * 128)
                at = rec[int(self.phys[b, j])]
                at[:m * d] = torch.tensor(codes[b, j * 128:j * 128 + m]).flatten()
                at[128 * d:128 * d + m] = torch.tensor(exps[b, j * 128:j * 128 + m])
        return rec

    def _selection(self, topk, frac):
        """A current block and earlier ones a token, ascending and -1 padded; from a common pool."""
        s, rng = self.shape, self.rng
        out = np.full((s.batch, s.n_heads_kv, self.n, topk), -1)
        for b, length in enumerate(self.lens):
            for h in range(s.n_heads_kv):
                top = length // s.block_size + 1
                pool = rng.permutation(top)[:max(1, int(top * (frac or 1.0)))]
                for i, path in enumerate(self.paths[b]):
                    if not path:
                        continue
                    cur = (length + len(path) - 1) // s.block_size
                    can = [x for x in rng.permutation(pool) if x < cur][:topk - 1]
                    got = sorted(can + [cur])
                    out[b, h, i, :len(got)] = got
        return out

    # ------------------------------------------------------------------ oracle
    def scores(self):
        s = self.shape
        return np.stack([tree_ops.scores(self.iq[b].double().numpy(), self.ik64[b], self.ikd64[b],
                                         self.paths[b], self.lens[b], s.block_size, self.nB,
                                         s.index_dim ** -0.5) for b in range(s.batch)])

    def score_bound(self):
        """Per (b, h, token): fp32 accumulation of index_dim products (twice the rounding bound, for
        an accumulator that truncates), the 2^-18 of the query's largest that its two 8-bit parts may
        miss, and the scaling's rounding."""
        s = self.shape
        d = s.index_dim
        out = np.zeros((s.batch, s.n_heads_kv, self.n, 1))
        for b, length in enumerate(self.lens):
            k = np.abs(np.concatenate([self.ik64[b][:length], self.ikd64[b]]))
            q = np.abs(self.iq[b].double().numpy())                       # [N, H, d]
            dots = (q @ k.T).max(-1)                                      # [N, H]
            lost = q.max(-1) * k.sum(-1).max() * (2.0 ** -18 if self.dt == torch.bfloat16 and self.packed else 0)
            e = (2 * (d + 2) * 2.0 ** -24 * dots + lost) * d ** -0.5 * 1.001
            out[b, :, :, 0] = e.T
        return out

    def attend(self):
        """out, lse, and the bound of each output: with e the error of a score (fp32 sums of d
        products, twice over, and 2^-22 of the exponential), P and the result rounded to the
        type."""
        s = self.shape
        G, d, N = s.n_heads_q // s.n_heads_kv, s.head_dim, self.n
        out = np.zeros((s.batch, N, s.n_heads_q, d))
        lse = np.full((s.batch, s.n_heads_q, N), -np.inf)
        tol, tol_lse = np.zeros_like(out), np.zeros_like(lse)
        half = 2.0 ** -8 if self.dt == torch.bfloat16 else 2.0 ** -24
        for b, length in enumerate(self.lens):
            for h in range(s.n_heads_kv):
                k, v, kd, vd = (x[b, h].double().numpy() for x in (self.k, self.v, self.kd, self.vd))
                for i, path in enumerate(self.paths[b]):
                    heads = slice(h * G, (h + 1) * G)
                    q = self.q[b, i, heads].double().numpy()
                    args = path, length, self.sel[b, h, i], s.block_size, d ** -0.5
                    o, l = tree_ops.attend(q, k, v, kd, vd, *args)
                    out[b, i, heads], lse[b, heads, i] = o, l
                    if not path:
                        continue
                    mag, _ = tree_ops.attend(q, k, np.abs(v), kd, np.abs(vd), *args)
                    big = (np.abs(q) @ np.abs(np.concatenate([k[:length], kd])).T).max(1)
                    e = 2 * (d + 4) * 2.0 ** -24 * big * d ** -0.5 + 2.0 ** -20   # [G]
                    # weights off by e, each (bf16) by its rounding; sums of up to 2^13 terms
                    tol[b, i, heads] = mag * (2 * e[:, None] + half + 2.0 ** -12 * half + 2.0 ** -18) + half * np.abs(o)
                    tol_lse[b, heads, i] = e + 2.0 ** -18 + 2.0 ** -22 * np.abs(l)
        return out, lse, tol, tol_lse
