"""Measured cases of a decode step over a tree of drafted tokens: index keys held in 8 bits
(packing and reading back), index scores of the drafted tokens, their block selection,
attention of the tree over the selected blocks and its own tokens, and the commit of the
accepted tokens to the caches.

`run` computes an operator in plain torch operations (32 bits) or, with `own`, through the
package's calls on the same state; `exact` computes it in 64 bits from its definition.

A drafted token i of a sequence with L cached tokens has a mask of 64 bits: the tokens of its
path from the root, itself among them (0: the tree has no token i).  Its position is L + depth.
It sees the L cached keys and those of its path, each key in the block of its position, so it
gets what a decode step would give it after its path.

Sizes: those of the package's decode workloads (64 query heads on 4 KV heads of 128 dims, blocks
of 128 keys, 64 selected blocks, 8 sequences of up to 2^20 tokens; 32 query heads and 16 blocks
for the smaller one), with trees of 1 to 64 tokens.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # the index keys of one step's drafts into the 8-bit cache, and read back; latency counts
        dict(name="index pack 8 drafts x 8", op="pack", batch=8, new=8, cap=8192, idim=128, dtype="bf16",
             paged=True),
        # the index keys of four prompts of unequal length, packed and read back
        dict(name="index pack prompts 128K", op="pack", batch=4, new=131072, cap=131072, idim=128,
             dtype="bf16", paged=True),
        # scores of a short chain of drafts over one short sequence
        dict(name="tree scores 1 x 8K, 5", op="scores", batch=1, nodes=5, cap=8195, ragged=False, hkv=4,
             idim=128, dtype="bf16", packed=True, paged=False, chain=True),
        # a ragged batch over 16-bit paged index keys
        dict(name="tree scores 16-bit ragged 128K, 12", op="scores", batch=8, nodes=12, cap=131072, ragged=True,
             hkv=4, idim=128, dtype="bf16", packed=False, paged=True, chain=False),
        # 8 sequences of 1M tokens, 16 drafts each, index keys in 8 bits
        dict(name="tree scores 8 x 1M, 16", op="scores", batch=8, nodes=16, cap=1 << 20, ragged=False, hkv=4,
             idim=128, dtype="bf16", packed=True, paged=False, chain=False),
        # the tree's masks and positions and its selections: a short cache
        dict(name="tree selection 2 x 20011, 7", op="select", batch=2, nodes=7, cap=20011, ragged=False, hkv=4,
             topk=16, chain=True),
        # ... and long ones: 8192 candidates for each of 512 rows
        dict(name="tree selection 8 x 1M, 16", op="select", batch=8, nodes=16, cap=1 << 20, ragged=True, hkv=4,
             topk=64, chain=False),
        # attention of a few drafts of one sequence: latency counts
        dict(name="tree attention 1 x 4100, 4", op="attend", batch=1, nodes=4, cap=4100, ragged=False, hq=32,
             hkv=4, dim=128, topk=16, pool=20, dtype="bf16", paged=False, chain=True),
        # the serving form: a ragged batch through block tables, 16 drafts a sequence
        dict(name="tree attention ragged 128K, 16", op="attend", batch=8, nodes=16, cap=131072, ragged=True,
             hq=64, hkv=4, dim=128, topk=64, pool=96, dtype="bf16", paged=True, chain=False),
        # wide trees: 64 drafts on 2 sequences
        dict(name="tree attention 2 x 64K, 64", op="attend", batch=2, nodes=64, cap=65536, ragged=False, hq=64,
             hkv=4, dim=128, topk=64, pool=128, dtype="bf16", paged=False, chain=False),
        # the accepted tokens' K, V and 8-bit index keys into the caches after a step
        dict(name="commit 8 x up to 5", op="commit", batch=8, nodes=16, accept=5, cap=2048, hkv=4, dim=128,
             dtype="bf16", paged=True),
        # ... of a large batch with long chains accepted
        dict(name="commit 64 x up to 48", op="commit", batch=64, nodes=64, accept=48, cap=1000, hkv=4, dim=128,
             dtype="bf16", paged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pack", "scores", "scores", "select", "attend", "attend", "commit"])
    hkv = rng.choice([1, 2, 4, 4, 8])
    dim = rng.choice([64, 128, 128])
    batch = rng.randint(1, 9)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    nodes = _log(rng, 1, 64)
    paged = rng.random() < 0.5
    chain = rng.random() < 0.3
    if op == "pack":
        new = _log(rng, 1, 50000)
        return dict(op=op, batch=batch, new=new, cap=new + rng.randint(0, 5000), idim=dim, dtype=dtype, paged=paged)
    cap = nodes + _log(rng, 1, 100000)
    c = dict(op=op, batch=batch, nodes=nodes, cap=cap, ragged=rng.random() < 0.5, hkv=hkv, chain=chain)
    if op == "scores":
        return dict(c, idim=dim, dtype=dtype, packed=rng.random() < 0.7, paged=paged)
    topk = _log(rng, 1, 64)
    if op == "select":                  # caches of more blocks than are selected
        topk += 1
        return dict(c, topk=topk, cap=nodes + max(cap, 2 * topk * BLOCK))
    if op == "attend":
        c["batch"] = max(1, min(rng.randint(1, 4), 256 // (nodes * hkv)))
        return dict(c, hq=hkv * rng.choice([1, 2, 5, 8, 64 // hkv]), dim=dim, topk=topk, pool=int(topk * rng.uniform(1, 2)),
                    dtype=dtype, paged=paged)
    return dict(op=op, batch=batch, nodes=nodes, accept=rng.randint(1, nodes), cap=nodes + _log(rng, 1, 4000), hkv=hkv,
                dim=dim, dtype=dtype, paged=paged)


# -------------------------------------------------------------------- sizes of a case

def _blocks(c):
    return -(-c["cap"] // BLOCK)


def _lens(c):
    """Cached tokens of each sequence, with room for its drafts: all full, or from full down to
    about an eighth."""
    b, full = c["batch"], c["cap"] - c["nodes"]
    if not c["ragged"]:
        return [full] * b
    return [max(0, full - (full * 7 * i) // (8 * b) - 37 * i) for i in range(b)]


def _counts(c):
    """New tokens of each sequence: all of `new`, and fewer for the later sequences."""
    return [max(1, c["new"] - (c["new"] * i) // (2 * c["batch"])) for i in range(c["batch"])]


def _accepts(c):
    return [1 + (c["accept"] - 1) * (i + 1) // c["batch"] for i in range(c["batch"])]


def work(c):
    e = 2 if c.get("dtype") == "bf16" else 4
    if c["op"] == "pack":
        n = sum(_counts(c))
        return {"bytes": 2 * n * (c["idim"] * e + c["idim"] + 1), "flops": 3 * n * c["idim"]}
    b, n = c["batch"], c["nodes"]
    if c["op"] == "commit":
        per = 2 * c["hkv"] * c["dim"] * e + 129
        return {"bytes": 2 * per * sum(_accepts(c)), "flops": 0}
    rows = b * c["hkv"] * n
    if c["op"] == "scores":
        keys = sum(_lens(c)) + b * n
        per = c["idim"] + 1 if c["packed"] else c["idim"] * e
        return {"bytes": keys * per + rows * (c["idim"] * e + 4 * _blocks(c)), "flops": 2 * c["idim"] * c["hkv"] * n * keys}
    if c["op"] == "select":
        cand = sum(-(-x // BLOCK) for x in _lens(c)) * c["hkv"] * n
        return {"bytes": 4 * cand + 4 * rows * c["topk"], "flops": cand}
    # the blocks that at least one token of a tree selected, each read once for a KV head
    keys = pairs = 0
    for length in _lens(c):
        have = -(-length // BLOCK)
        k, pool = min(c["topk"], have), min(c["pool"], have)
        keys += min(length, BLOCK * pool * (1 - (1 - k / max(1, pool)) ** n)) + n
        pairs += n * min(length + n, k * BLOCK)
    d = c["dim"]
    return {"bytes": int(c["hkv"] * keys * 2 * d * e) + 2 * b * n * c["hq"] * d * e, "flops": 4 * d * c["hq"] * pairs}


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _table(g, batch, blocks):
    """A shuffled block table over pools with a few spare blocks."""
    n_phys = batch * blocks + 5
    perm = torch.randperm(n_phys, generator=g, device=DEV)[: batch * blocks]
    return perm.view(batch, blocks).to(torch.int32).contiguous(), n_phys


def _rows(g, shape, dt):
    """K or V rows as a model makes them: unit normal with an offset of each channel."""
    off = torch.randn(shape[-1], generator=g, device=DEV)
    return torch.randn(shape, generator=g, device=DEV).add_(off).to(dt)


def _index_rows(g, shape, dt):
    """Index keys: unit normal, of magnitudes that differ from token to token."""
    size = torch.randn((*shape[:-1], 1), generator=g, device=DEV).mul_(0.5).exp_()
    return torch.randn(shape, generator=g, device=DEV).mul_(size).to(dt)


def _parents(g, c):
    """Parent of every drafted token (-1: the last cached token).  Chains, or trees whose tokens
    hang on one of the few before them; the later sequences' trees are smaller (-2: no token)."""
    b, n = c["batch"], c["nodes"]
    i = torch.arange(n, device=DEV).expand(b, n)
    back = torch.randint(0, 5, (b, n), generator=g, device=DEV) if not c["chain"] else torch.zeros_like(i)
    parents = (i - 1 - back).clamp(min=-1)
    have = n - (torch.arange(b, device=DEV) * n) // (4 * b)
    return parents.masked_fill(i >= have[:, None], -2).to(torch.int32).contiguous()


def _masks(parents):
    """mask [b, n] (int64, bit a: token a is on the path) of trees on the host."""
    out = []
    for row in parents.tolist():
        m = []
        for i, p in enumerate(row):
            m.append((1 << i) if p == -1 else (m[p] | 1 << i) if 0 <= p < i and m[p] else 0)
        out.append([x - (1 << 64) if x >= 1 << 63 else x for x in m])
    return torch.tensor(out, dtype=torch.int64, device=DEV)


def _select(g, c, lens, depth):
    """Selections [b, hkv, n, topk] as the tokens of one tree make them: each takes its own
    topk - 1 of a pool of earlier blocks that its KV head finds relevant, and its current block;
    ascending, -1 where there are fewer (and for tokens that are not there)."""
    n, hkv, k, rows = c["nodes"], c["hkv"], c["topk"], []
    for length, dep in zip(lens, depth):
        cur = (length + dep.clamp(min=0)) // BLOCK                       # [n]
        tail = length // BLOCK
        pool = torch.rand(hkv, tail + 1, generator=g, device=DEV)
        pool = pool.topk(min(c["pool"], tail + 1), dim=1).indices        # [hkv, pool]
        r = torch.rand(hkv, n, pool.shape[1], generator=g, device=DEV)
        # a token's current block is taken in any case, and is no earlier block
        late = pool[:, None, :] >= cur[None, :, None]
        r = r.masked_fill(late, -1.0)
        m = min(k - 1, pool.shape[1])
        best = r.topk(m, dim=2)
        pick = pool[:, None, :].expand(r.shape).gather(2, best.indices)
        big = 1 << 30
        pick = pick.masked_fill(best.values < 0, big)
        pick = torch.cat([pick, cur[None, :, None].expand(hkv, n, 1)], dim=2).sort(dim=2).values
        pick = torch.nn.functional.pad(pick, (0, k - m - 1), value=big)
        rows.append(torch.where((pick == big) | (dep < 0)[None, :, None], -1, pick))
    return torch.stack(rows).to(torch.int32).contiguous()


def prepare(c, seed):
    g = _gen(seed)
    s = {"case": c}
    dt = TYPES[c.get("dtype", "bf16")]
    b, blocks = c["batch"], _blocks(c)
    if c["op"] == "pack":
        n, d = c["new"], c["idim"]
        s["x"] = _index_rows(g, (b, n, d), dt)
        s["starts"] = torch.randint(0, c["cap"] - n + 1, (b,), generator=g, device=DEV).to(torch.int32)
        s["lens"] = (s["starts"] + torch.tensor(_counts(c), device=DEV)).to(torch.int32)
        s["table"], s["n_phys"] = _table(g, b, blocks) if c["paged"] else (None, b * blocks)
        s["cache"] = torch.zeros((s["n_phys"], BLOCK * (d + 1)), dtype=torch.uint8, device=DEV)
        s["out"] = torch.zeros_like(s["x"])
        return s
    n = c["nodes"]
    if c["op"] == "commit":
        s["table"], s["n_phys"] = _table(g, b, blocks) if c["paged"] else (None, b * blocks)
        d, hkv = c["dim"], c["hkv"]
        lens = torch.randint(0, c["cap"] - n + 1, (b,), generator=g, device=DEV)
        s["lens"] = lens.to(torch.int32)
        shape = (s["n_phys"], hkv, BLOCK, d) if c["paged"] else (b, hkv, c["cap"], d)
        s["k"], s["v"] = _rows(g, shape, dt), _rows(g, shape, dt)
        s["cache"] = torch.zeros((s["n_phys"], BLOCK * 129), dtype=torch.uint8, device=DEV)
        s["kd"], s["vd"] = _rows(g, (b, hkv, n, d), dt), _rows(g, (b, hkv, n, d), dt)
        s["drafts"] = torch.zeros((b, BLOCK * 129), dtype=torch.uint8, device=DEV)
        s["drafts"].copy_(_records(_index_rows(g, (b, BLOCK, 128), torch.bfloat16)))
        # a path of the tree: ascending tokens
        path = torch.rand(b, n, generator=g, device=DEV).topk(c["accept"], dim=1).indices.sort(dim=1).values
        held = torch.arange(c["accept"], device=DEV) < torch.tensor(_accepts(c), device=DEV)[:, None]
        s["accepted"] = torch.where(held, path, -1).to(torch.int32).contiguous()
        s["new_lens"] = torch.zeros_like(s["lens"])
        s["out"] = torch.zeros((b, c["accept"], 128), dtype=torch.bfloat16, device=DEV)
        return s
    lens = _lens(c)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["parents"] = _parents(g, c)
    s["mask"] = _masks(s["parents"])
    depth = _count_bits(s["mask"]) - 1
    if c["op"] == "select":
        s["scores"] = torch.randn((b, c["hkv"], n, blocks), generator=g, device=DEV)
        s["sel"] = torch.empty((b, c["hkv"], n, c["topk"]), dtype=torch.int32, device=DEV)
        s["mask_out"] = torch.empty_like(s["mask"])
        s["positions"] = torch.empty((b, n), dtype=torch.int32, device=DEV)
        return s
    paged = c["paged"]
    s["table"], s["n_phys"] = _table(g, b, blocks) if paged else (None, b * blocks)
    if c["op"] == "scores":
        d = c["idim"]
        s["iq"] = torch.randn((b, n, c["hkv"], d), generator=g, device=DEV).to(dt)
        if c["packed"]:
            s["cache"] = torch.empty((s["n_phys"], BLOCK * (d + 1)), dtype=torch.uint8, device=DEV)
            for p in range(0, s["n_phys"], 16384):
                m = min(16384, s["n_phys"] - p)
                s["cache"][p:p + m] = _records(_index_rows(g, (m, BLOCK, d), dt))
            s["drafts"] = torch.zeros((b, BLOCK * (d + 1)), dtype=torch.uint8, device=DEV)
            s["drafts"].copy_(_records(_index_rows(g, (b, BLOCK, d), dt)))
        else:
            s["cache"] = _index_rows(g, (s["n_phys"], BLOCK, d) if paged else (b, c["cap"], d), dt)
            s["drafts"] = _index_rows(g, (b, n, d), dt)
        s["scores"] = torch.empty((b, c["hkv"], n, blocks), device=DEV)
        return s
    d = c["dim"]
    s["q"] = torch.randn((b, n, c["hq"], d), generator=g, device=DEV).to(dt)
    s["k"], s["v"] = (_rows(g, (s["n_phys"], c["hkv"], BLOCK, d) if paged else (b, c["hkv"], c["cap"], d), dt)
                      for _ in range(2))
    s["kd"], s["vd"] = (_rows(g, (b, c["hkv"], n, d), dt) for _ in range(2))
    s["sel"] = _select(g, c, lens, depth)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((b, c["hq"], n), device=DEV)
    return s


# ------------------------------------------------------------------------ plain forms

def _bits(mask):
    """[..., 64] truth values of the bits of int64 words."""
    return (mask.unsqueeze(-1) >> torch.arange(64, device=DEV)) & 1 == 1


def _count_bits(mask):
    return _bits(mask).sum(-1)


def _pow2(byte):
    """2^(byte - 127) in fp32, for bytes of 1 to 254."""
    return (byte.int() << 23).view(torch.float32)


def _quantise(x):
    """8-bit codes of the rows of x, and each row's exponent byte: the least power of two that
    brings the row's largest magnitude to 448 or less."""
    x = x.float()
    bits = x.abs().amax(-1).contiguous().view(torch.int32)
    byte = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000)).clamp(min=1)
    codes = (x * _pow2(254 - byte).unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, byte.to(torch.uint8)


def _records(x):
    """The bytes that hold the rows x [..., 128, d] of one block."""
    codes, byte = _quantise(x)
    return torch.cat([codes.flatten(-2), byte], dim=-1)


def _values(rec, d):
    """The rows [..., 128, d] that the bytes of a block hold, in fp32."""
    codes, byte = rec.split([BLOCK * d, BLOCK], dim=-1)
    x = codes.contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (BLOCK, d))
    return x * _pow2(byte).unsqueeze(-1)


def _physical(s, blocks):
    """Physical block of every (sequence, logical block)."""
    if s["table"] is not None:
        return s["table"].long()
    b = s["case"]["batch"]
    return torch.arange(b * blocks, device=DEV).view(b, blocks)


def _pack_plain(s):
    c = s["case"]
    d, blocks = c["idim"], _blocks(c)
    pos = s["starts"].long()[:, None] + torch.arange(c["new"], device=DEV)
    there = pos < s["lens"].long()[:, None]
    at = pos.clamp(max=blocks * BLOCK - 1)
    phys, row = _physical(s, blocks).gather(1, at // BLOCK), at % BLOCK
    codes, byte = _quantise(s["x"])
    p = there.nonzero(as_tuple=True)
    table = s["cache"][:, :BLOCK * d].unflatten(-1, (BLOCK, d))
    table[phys[p], row[p]] = codes[p]
    s["cache"][:, BLOCK * d:][phys[p], row[p]] = byte[p]
    held = table[phys, row].view(torch.float8_e4m3fn).float()
    held = held * _pow2(s["cache"][:, BLOCK * d:][phys, row]).unsqueeze(-1)
    s["out"].copy_(torch.where(there.unsqueeze(-1), held.to(s["out"].dtype), s["out"]))
    return s["out"]


def _tree_blocks(s):
    """The masks' bits [b, n, n], each token's position and whether it is there."""
    n = s["case"]["nodes"]
    bits = _bits(s["mask"])[..., :n]
    depth = bits.sum(-1) - 1
    return bits, s["lens"].long()[:, None] + depth, depth >= 0


def _scores_plain(s):
    c = s["case"]
    b, n, h, d, blocks = c["batch"], c["nodes"], c["hkv"], c["idim"], _blocks(c)
    q = s["iq"].float().flatten(1, 2)                                        # [b, n h, d]
    if c["packed"]:
        k = _values(s["cache"][_physical(s, blocks)] if s["table"] is not None else
                    s["cache"].view(b, blocks, -1), d).flatten(1, 2)
        kd = _values(s["drafts"], d)[:, :n]
    else:
        k = (s["cache"][_physical(s, blocks)].flatten(1, 2) if s["table"] is not None else s["cache"]).float()
        k = torch.nn.functional.pad(k, (0, 0, 0, blocks * BLOCK - k.shape[1]))
        kd = s["drafts"].float()
    scale = d ** -0.5
    z = (q @ k.transpose(1, 2)) * scale                                      # [b, n h, keys]
    seen = torch.arange(blocks * BLOCK, device=DEV) < s["lens"][:, None]
    z = z.masked_fill_(~seen[:, None], -math.inf)
    best = z.unflatten(-1, (blocks, BLOCK)).amax(-1).unflatten(1, (n, h)).transpose(1, 2)   # [b, h, n, blocks]
    bits, pos, there = _tree_blocks(s)
    zd = ((q @ kd.transpose(1, 2)) * scale).unflatten(1, (n, h)).transpose(1, 2)            # [b, h, n, n]
    zd = zd.masked_fill(~bits.unsqueeze(1), -math.inf)
    at = (pos // BLOCK)[:, None, None].expand_as(zd).clamp(0, blocks - 1)
    best = best.scatter_reduce(3, at, zd, "amax")
    s["scores"].copy_(best.masked_fill(~there[:, None, :, None], -math.inf))
    return s["scores"]


def _select_plain(s):
    c = s["case"]
    n, k, blocks = c["nodes"], c["topk"], _blocks(c)
    # paths: a token's bits are its own and those of its parent's path, after as many steps as
    # doubling the distance takes
    par = s["parents"].long()
    i = torch.arange(n, device=DEV)
    ok = (par >= -1) & (par < i)
    one = torch.eye(n, dtype=torch.float32, device=DEV).expand(*par.shape, n)
    root = par == -1
    step = (one.gather(1, par.clamp(min=0).unsqueeze(-1).expand_as(one)) * (ok & ~root).unsqueeze(-1))
    reach = one + step
    reach = reach @ reach                          # each product doubles the distance: 64 tokens need 6
    reach = (reach @ reach).clamp(max=1)
    reach = (reach @ reach).clamp(max=1)
    reach = (reach @ reach).clamp(max=1)
    reach = (reach @ reach).clamp(max=1)
    reach = ((reach @ reach) > 0)
    there = ~(reach & ~ok.unsqueeze(1)).any(-1)
    bits = reach & there.unsqueeze(-1)
    s["mask_out"].copy_((bits.long() << i).sum(-1))
    depth = bits.sum(-1) - 1
    pos = s["lens"].long()[:, None] + depth
    s["positions"].copy_(torch.where(there, pos, -1))
    cur = (pos // BLOCK)[:, None, :, None]
    j = torch.arange(blocks, device=DEV)
    x = s["scores"].masked_fill(j == cur, math.inf)
    x = x.masked_fill((j > cur) | ~there[:, None, :, None], -math.inf)
    order = x.sort(dim=-1, descending=True, stable=True)
    m = min(k, blocks)
    take = order.indices[..., :m].masked_fill(order.values[..., :m] == -math.inf, 1 << 30).sort(dim=-1).values
    take = torch.nn.functional.pad(take, (0, k - m), value=1 << 30)
    s["sel"].copy_(take.masked_fill(take == 1 << 30, -1))
    return [s["mask_out"], s["positions"], s["sel"]]


def _attend_plain(s):
    c = s["case"]
    b, n, h, d, k, blocks = c["batch"], c["nodes"], c["hkv"], c["dim"], c["topk"], _blocks(c)
    group = c["hq"] // h
    sel = s["sel"].long()                                                    # [b, h, n, k]
    safe = sel.clamp(min=0)
    j = torch.arange(h, device=DEV).view(1, h, 1, 1)
    if c["paged"]:
        phys = _physical(s, blocks)[:, None, None].expand(b, h, n, blocks).gather(3, safe)
        kk, vv = s["k"][phys, j], s["v"][phys, j]                            # [b, h, n, k, 128, d]
    else:
        rows = (safe.unsqueeze(-1) * BLOCK + torch.arange(BLOCK, device=DEV)).clamp(max=c["cap"] - 1)
        i = torch.arange(b, device=DEV).view(b, 1, 1, 1, 1)
        kk, vv = s["k"][i, j.unsqueeze(-1), rows], s["v"][i, j.unsqueeze(-1), rows]
    kk, vv = kk.flatten(3, 4).float(), vv.flatten(3, 4).float()
    at = (sel.unsqueeze(-1) * BLOCK + torch.arange(BLOCK, device=DEV)).flatten(3)
    seen = (sel >= 0).repeat_interleave(BLOCK, dim=3) & (at < s["lens"].view(b, 1, 1, 1))
    q = s["q"].float().unflatten(2, (h, group)).transpose(1, 2)              # [b, h, n, group, d]
    z = (q @ kk.transpose(-1, -2)).masked_fill(~seen.unsqueeze(3), -math.inf)
    bits, pos, _ = _tree_blocks(s)
    mine = bits[:, None] & (sel.unsqueeze(-1) == (pos // BLOCK)[:, None, None, None]).any(3)  # [b, h, n, n]
    zd = (q @ s["kd"].float()[:, :, None].transpose(-1, -2)).masked_fill(~mine.unsqueeze(3), -math.inf)
    z = torch.cat([z, zd], dim=-1) / math.sqrt(d)
    top = z.amax(-1, keepdim=True)
    e = (z - top.masked_fill(top == -math.inf, 0)).exp()
    total = e.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    p = e / total.clamp(min=1e-38)
    vv = vv.masked_fill_(~seen.unsqueeze(-1), 0)
    m = vv.shape[3]
    out = p[..., :m] @ vv + p[..., m:] @ s["vd"].float()[:, :, None]
    s["out"].copy_(out.transpose(1, 2).flatten(2, 3))
    s["lse"].copy_(lse.permute(0, 1, 3, 2).flatten(1, 2))
    return [s["out"], s["lse"]]


def _commit_plain(s):
    c = s["case"]
    b, blocks = c["batch"], _blocks(c)
    node = s["accepted"].long()
    held = node >= 0
    pos = s["lens"].long()[:, None] + torch.arange(c["accept"], device=DEV)
    seq, i = held.nonzero(as_tuple=True)
    node, to = node[seq, i], pos[seq, i]
    phys = _physical(s, blocks)[seq, to // BLOCK]
    for name in ("k", "v"):
        rows = s[name + "d"][seq, :, node]
        if c["paged"]:
            s[name][phys, :, to % BLOCK] = rows
        else:
            s[name][seq, :, to] = rows
    at = s["cache"][:, :BLOCK * 128].unflatten(-1, (BLOCK, 128))
    at[phys, to % BLOCK] = s["drafts"][:, :BLOCK * 128].unflatten(-1, (BLOCK, 128))[seq, node]
    s["cache"][phys, BLOCK * 128 + to % BLOCK] = s["drafts"][seq, BLOCK * 128 + node]
    s["new_lens"].copy_(s["lens"] + held.sum(1))
    x = at[phys, to % BLOCK].view(torch.float8_e4m3fn).float()
    x = x * _pow2(s["cache"][phys, BLOCK * 128 + to % BLOCK]).unsqueeze(-1)
    s["out"][seq, i] = x.to(s["out"].dtype)
    return [s["k"], s["v"], s["new_lens"], s["out"]]


def run(s):
    if own:
        return _run_own(s)
    return {"pack": _pack_plain, "scores": _scores_plain, "select": _select_plain, "attend": _attend_plain,
            "commit": _commit_plain}[s["case"]["op"]](s)


# ---------------------------------------------------------------- the package's calls

def _plan(s):
    """What a user's program keeps between steps: the shape, the workspace, the list of caches."""
    from block_sparse_gqa_02_gb300 import _lib
    c = s["case"]
    hkv = c.get("hkv", 1)
    shape = _lib.make_shape(c["batch"], c.get("nodes", 1), c["cap"], c.get("hq", hkv), hkv, c.get("dim", 128),
                            c.get("idim", 128), BLOCK, c.get("topk", 1), 1, c.get("dtype", "bf16"))
    more = None
    if c["op"] == "attend":
        more = torch.empty(_lib.msa_workspace_bytes(shape, 5) // 4 + 4, device=DEV)
    if c["op"] == "commit":
        more = (_lib.make_commit_tensors([(s["kd"], s["k"]), (s["vd"], s["v"])], [(s["drafts"], s["cache"])]),
                # the index keys are bf16 whatever K and V are
                _lib.make_shape(c["batch"], 1, c["cap"], hkv, hkv, c["dim"], 128, BLOCK, 1, 1, "bf16"))
    if c["op"] == "pack":
        shape.seq_q = 1
    return _lib, shape, more


def _run_own(s):
    c = s["case"]
    if "plan" not in s:
        s["plan"] = _plan(s)
    lib, shape, more = s["plan"]
    if c["op"] == "pack":
        lib.msa_index_pack(shape, c["new"], s["starts"], s["lens"], s["table"], s["n_phys"], s["x"], s["cache"])
        lib.msa_index_unpack(shape, c["new"], s["starts"], s["lens"], s["table"], s["n_phys"], s["cache"], s["out"])
        return s["out"]
    if c["op"] == "scores":
        lib.msa_index_scores_tree(shape, s["lens"], s["table"], s["n_phys"], s["mask"], s["iq"], s["cache"],
                                  s["drafts"], s["scores"], packed=c["packed"])
        return s["scores"]
    if c["op"] == "select":
        lib.msa_tree_mask(shape, s["lens"], s["parents"], s["mask_out"], s["positions"])
        lib.msa_block_topk_tree(shape, s["lens"], s["mask_out"], s["scores"], s["sel"])
        return [s["mask_out"], s["positions"], s["sel"]]
    if c["op"] == "attend":
        lib.msa_sparse_decode_tree(shape, s["lens"], s["table"], s["n_phys"], s["mask"], s["q"], s["k"], s["v"],
                                   s["kd"], s["vd"], s["sel"], s["out"], s["lse"], more)
        return [s["out"], s["lse"]]
    tensors, index = more
    lib.msa_tree_commit(shape, s["lens"], s["table"], s["n_phys"], s["accepted"], tensors, s["new_lens"])
    # the committed tokens' index keys as the cache now holds them
    lib.msa_index_unpack(index, c["accept"], s["lens"], s["new_lens"], s["table"], s["n_phys"], s["cache"], s["out"])
    return [s["k"], s["v"], s["new_lens"], s["out"]]


# ------------------------------------------------------- the definitions, in 64 bits

def _two(n):
    """2^n in 64 bits, exactly, for whole n from -1022 to 1023."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _decode_e4m3(codes):
    """Values of the 8-bit codes: sign, 4 bits of exponent (bias 7), 3 bits of fraction."""
    v = codes.long()
    e, f = (v // 8) % 16, (v % 8).double()
    mag = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * _two(e - 7))
    return torch.where(v >= 128, -mag, mag)


def _exact_held(x):
    """The values that the cache holds for rows x: to four significant bits, in steps that stop
    falling 2^-6 * 2^e below, e the least with every magnitude within 448 * 2^e."""
    y = x.double()
    amax = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -200) / 448))
    e = torch.where(448 * _two(e - 1) >= amax, e - 1, e)
    e = torch.where(448 * _two(e) < amax, e + 1, e).clamp(min=-126)
    mag = y.abs()
    top = torch.floor(torch.log2(mag.clamp(min=2.0 ** -300)))
    top = torch.where(_two(top) > mag, top - 1, top)
    top = torch.where(_two(top + 1) <= mag, top + 1, top)
    step = _two(torch.maximum(top, e - 6) - 3)
    return torch.round(y / step) * step                       # ties to even


def _exact_scores(s):
    c = s["case"]
    b, n, h, d, blocks = c["batch"], c["nodes"], c["hkv"], c["idim"], _blocks(c)
    out = torch.full((b, h, n, blocks), -math.inf, dtype=torch.float64, device=DEV)
    masks = s["mask"].tolist()
    lens = s["lens"].tolist()
    for i in range(b):
        q = s["iq"][i].double().reshape(n * h, d) / math.sqrt(d)
        for j0 in range(0, -(-lens[i] // BLOCK), 1024):
            j1 = min(blocks, j0 + 1024)
            at = s["table"][i, j0:j1].long() if s["table"] is not None else torch.arange(i * blocks + j0, i * blocks + j1, device=DEV)
            if c["packed"]:
                rec = s["cache"][at]
                key = _decode_e4m3(rec[:, :BLOCK * d]).view(-1, BLOCK, d)
                key = (key * _two(rec[:, BLOCK * d:].long() - 127)[..., None]).reshape(-1, d)
            elif s["table"] is not None:
                key = s["cache"][at].double().reshape(-1, d)
            else:
                key = s["cache"][i, j0 * BLOCK:j1 * BLOCK].double()
            key = key[:max(0, lens[i] - j0 * BLOCK)]
            z = key @ q.T
            whole = z.shape[0] // BLOCK
            out[i, :, :, j0:j0 + whole] = z[:whole * BLOCK].view(whole, BLOCK, n, h).amax(1).permute(2, 1, 0)
            if z.shape[0] % BLOCK:
                out[i, :, :, j0 + whole] = z[whole * BLOCK:].amax(0).view(n, h).T
        if c["packed"]:
            rec = s["drafts"][i]
            kd = _decode_e4m3(rec[:BLOCK * d]).view(BLOCK, d) * _two(rec[BLOCK * d:].long() - 127)[:, None]
        else:
            kd = s["drafts"][i].double()
        z = (kd[:n] @ q.T).view(n, n, h).cpu()                                # [key, token, head]
        best = out[i].cpu()
        for t in range(n):
            path = [a for a in range(n) if masks[i][t] >> a & 1]
            if not path:
                best[:, t] = -math.inf
            for a in path:
                blk = (lens[i] + bin(masks[i][a] % (1 << 64)).count("1") - 1) // BLOCK
                best[:, t, blk] = torch.maximum(best[:, t, blk], z[a, t])
        out[i] = best.to(DEV)
    return out


def _exact_attend(s):
    c = s["case"]
    b, n, h, d, blocks = c["batch"], c["nodes"], c["hkv"], c["dim"], _blocks(c)
    group = c["hq"] // h
    out = torch.zeros((b, n, c["hq"], d), dtype=torch.float64, device=DEV)
    lse = torch.full((b, c["hq"], n), -math.inf, dtype=torch.float64, device=DEV)
    masks, lens, sel = s["mask"].tolist(), s["lens"].tolist(), s["sel"].tolist()
    for i in range(b):
        place = [(lens[i] + bin(m % (1 << 64)).count("1") - 1) // BLOCK for m in masks[i]]
        for j in range(h):
            kd, vd = s["kd"][i, j].double(), s["vd"][i, j].double()
            for t in range(n):
                chosen = [x for x in sel[i][j][t] if x >= 0]
                path = [a for a in range(n) if masks[i][t] >> a & 1 and place[a] in chosen]
                at = torch.tensor(chosen, dtype=torch.long, device=DEV)
                pos = (at[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten()
                pos = pos[pos < lens[i]]
                if c["paged"]:
                    phys = s["table"][i].long()[pos // BLOCK]
                    k, v = s["k"][phys, j, pos % BLOCK], s["v"][phys, j, pos % BLOCK]
                else:
                    k, v = s["k"][i, j, pos], s["v"][i, j, pos]
                k, v = torch.cat([k.double(), kd[path]]), torch.cat([v.double(), vd[path]])
                if not k.shape[0]:
                    continue
                heads = slice(j * group, (j + 1) * group)
                z = s["q"][i, t, heads].double() @ k.T * d ** -0.5
                norm = torch.logsumexp(z, dim=1)
                out[i, t, heads] = torch.exp(z - norm[:, None]) @ v
                lse[i, heads, t] = norm
    return [out, lse]


def exact(c, seed):
    if c["op"] == "select":
        return None
    s = prepare(c, seed)
    if c["op"] == "pack":
        there = torch.arange(c["new"], device=DEV) < (s["lens"] - s["starts"])[:, None]
        return _exact_held(s["x"]) * there[..., None]
    if c["op"] == "scores":
        return _exact_scores(s)
    if c["op"] == "attend":
        return _exact_attend(s)
    blocks, lens, table = _blocks(c), s["lens"].tolist(), s["table"]
    rec = s["drafts"]
    key = _decode_e4m3(rec[:, :BLOCK * 128]).view(-1, BLOCK, 128) * _two(rec[:, BLOCK * 128:].long() - 127)[..., None]
    got = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    k, v = s["k"].double(), s["v"].double()
    for i, row in enumerate(s["accepted"].tolist()):
        for m, node in enumerate(x for x in row if x >= 0):
            to = lens[i] + m
            where = (int(table[i, to // BLOCK]), slice(None), to % BLOCK) if c["paged"] else (i, slice(None), to)
            k[where], v[where] = s["kd"][i, :, node].double(), s["vd"][i, :, node].double()
            got[i, m] = key[i, node]
    return [k, v, None, got]
