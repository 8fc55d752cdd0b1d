"""Measured cases of the operators around the decode cache: rotary positions, the 4-bit
cache (packing, and decode attention over it), decode attention that accumulates the
attention weight of every block, and eviction of blocks by that weight.

`run` computes an operator in plain torch operations (32 bits, 64 for angles) or, with
`own`, through the package's calls on the same state; `exact` computes it in 64 bits from
its definition.

Sizes: the decode shapes are those of the package's workloads (64 query heads on 4 KV heads
of 128 dims, blocks of 128 keys, 64 selected blocks, 8 sequences of up to 2^20 tokens; 32
query heads and 16 blocks for the smaller one), and ragged relatives of them.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
GROUP = 32
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 8 sequences: the new token's q, k, index q and index k, each
        # sequence at its own far position; latency counts
        dict(name="rope decode 8 seqs", op="rope", batch=8, seq=1, hq=64, hkv=4, dim=128, rot=128,
             dtype="bf16", interleaved=False, scaling="yarn", factor=8.0, inverse=False,
             positions="lens", max_pos=1 << 20),
        # the gradients of a training batch rotated back: fp32, half of each head, interleaved
        dict(name="rope backward f32", op="rope", batch=2, seq=5003, hq=32, hkv=4, dim=128, rot=64,
             dtype="f32", interleaved=True, scaling="none", factor=1.0, inverse=True,
             positions="given", max_pos=5003),
        # the whole 128K prefill's tensors before its index branch
        dict(name="rope prefill 128K", op="rope", batch=1, seq=131072, hq=64, hkv=4, dim=128, rot=128,
             dtype="bf16", interleaved=False, scaling="ntk", factor=4.0, inverse=False,
             positions="range", max_pos=131072),
        # a decode step's new K and V rows into the 4-bit pools, and read back
        dict(name="pack 1 token x 8", op="pack", batch=8, new=1, cap=8192, hkv=4, dim=128,
             dtype="bf16", paged=True),
        # two prompts of unequal length into the 4-bit pools, and read back
        dict(name="pack prompts 32K", op="pack", batch=2, new=32768, cap=32768, hkv=4, dim=128,
             dtype="bf16", paged=True),
        # decode attention over the 4-bit cache: one short sequence
        dict(name="packed decode 1 x 4097", op="packed", batch=1, cap=4097, ragged=False, hq=32, hkv=4,
             dim=128, topk=16, dtype="bf16", paged=False, mass=False),
        # a ragged batch of the serving form, with the blocks' weights accumulated
        dict(name="packed decode ragged 128K", op="packed", batch=8, cap=131072, ragged=True, hq=64,
             hkv=4, dim=128, topk=64, dtype="bf16", paged=True, mass=True),
        # the 8 x 1M decode over a 4-bit cache
        dict(name="packed decode 8 x 1M", op="packed", batch=8, cap=1 << 20, ragged=False, hq=64, hkv=4,
             dim=128, topk=64, dtype="bf16", paged=False, mass=False),
        # decode over the 16-bit cache with the blocks' weights accumulated: a small one
        dict(name="mass decode 2 x 20011", op="mass", batch=2, cap=20011, ragged=False, hq=32, hkv=4,
             dim=128, topk=16, dtype="bf16", paged=False),
        # ... and the serving form's batch
        dict(name="mass decode ragged 256K", op="mass", batch=8, cap=262144, ragged=True, hq=64, hkv=4,
             dim=128, topk=64, dtype="bf16", paged=True),
        # 8 paged sequences of 1M tokens cut to a quarter: block tables and weights only
        dict(name="evict paged 8 x 1M", op="evict", batch=8, cap=1 << 20, ragged=True, hkv=4, dim=128,
             keep=2048, first=4, recent=16, dtype="bf16", paged=True),
        # contiguous caches of 128K tokens cut to a quarter: K, V and index keys move
        dict(name="evict contiguous 2 x 128K", op="evict", batch=2, cap=131000, ragged=False, hkv=4,
             dim=128, keep=256, first=1, recent=8, dtype="bf16", paged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "pack", "packed", "packed", "mass", "evict"])
    hkv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128, 128])
    batch = rng.randint(1, 9)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        seq = _log(rng, 1, 12000)
        return dict(op=op, batch=batch, seq=seq, hq=hkv * rng.randint(1, 8), hkv=hkv, dim=dim,
                    rot=16 * rng.randint(1, dim // 16), dtype=dtype, interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), inverse=rng.random() < 0.4,
                    positions=rng.choice(["range", "given"]), max_pos=seq + rng.randint(0, 1 << 20))
    if op == "pack":
        new = _log(rng, 1, 12000)
        return dict(op=op, batch=batch, new=new, cap=new + rng.randint(0, 5000), hkv=hkv, dim=dim,
                    dtype=dtype, paged=rng.random() < 0.5)
    if op in ("packed", "mass"):
        cap = _log(rng, 1, 100000)
        topk = _log(rng, 1, 64)
        c = dict(op=op, batch=batch, cap=cap, ragged=rng.random() < 0.5, hkv=hkv, dim=dim, topk=topk,
                 hq=hkv * rng.choice([1, 2, 5, 8, 16]), dtype=dtype)
        if op == "packed":
            return dict(c, paged=rng.random() < 0.5, mass=rng.random() < 0.5)
        if rng.random() < 0.5:          # the paged 16-bit pools: 4 KV heads of 128 dims
            return dict(c, paged=True, hkv=4, dim=128, dtype="bf16", hq=4 * rng.choice([1, 4, 16]))
        return dict(c, paged=False, ragged=False)
    cap = _log(rng, 1, 130000)
    blocks = -(-cap // BLOCK)
    paged = rng.random() < 0.5
    recent = rng.randint(1, 8)
    first = rng.randint(0, 4)
    keep = max(first + recent, _log(rng, 1, max(2, blocks)))
    return dict(op=op, batch=rng.randint(1, 4), cap=cap, ragged=paged and rng.random() < 0.7, hkv=hkv, dim=dim,
                keep=keep, first=first, recent=recent, dtype=dtype, paged=paged)


# -------------------------------------------------------------------- sizes of a case

def _lens(c):
    """Cache lengths of the batch: all full, or from full down to about an eighth."""
    b = c["batch"]
    if not c["ragged"]:
        return [c["cap"]] * b
    return [max(1, c["cap"] - (c["cap"] * 7 * i) // (8 * b) - 37 * i) for i in range(b)]


def _keys(c):
    """Keys each sequence attends: the current block and top_k - 1 full ones before it."""
    n = []
    for length in _lens(c):
        blocks = -(-length // BLOCK)
        tail = length - (blocks - 1) * BLOCK
        n.append((min(c["topk"], blocks) - 1) * BLOCK + tail)
    return n


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    d = c["dim"]
    if c["op"] == "rope":
        rows = c["batch"] * c["seq"] * (c["hq"] + 2 * c["hkv"] + 1)
        return {"bytes": 2 * rows * d * e, "flops": 3 * rows * c["rot"]}
    if c["op"] == "pack":
        # values in, packed out, packed in, values out
        values = 2 * sum(_pack_counts(c)) * c["hkv"] * d
        return {"bytes": 2 * values * e + 2 * values * 5 // 8, "flops": 8 * values}
    if c["op"] in ("packed", "mass"):
        keys = sum(_keys(c)) * c["hkv"]
        per_key = d * 5 // 4 if c["op"] == "packed" else 2 * d * e
        other = 2 * c["batch"] * c["hq"] * d * e + c["batch"] * c["hkv"] * c["topk"] * 12
        return {"bytes": keys * per_key + other, "flops": 4 * d * keys * (c["hq"] // c["hkv"])}
    blocks = -(-c["cap"] // BLOCK)
    n = c["batch"] * blocks * (4 * c["hkv"] * 2 + (8 if c["paged"] else 0))
    if not c["paged"]:
        kept = sum(_kept_len(c, x) for x in _lens(c))
        n += 2 * kept * d * e * (2 * c["hkv"] + 1)
    return {"bytes": n, "flops": c["batch"] * blocks * c["hkv"]}


def _kept_len(c, length):
    blocks = -(-length // BLOCK)
    return length - (blocks - min(blocks, c["keep"])) * BLOCK


def _pack_counts(c):
    """New tokens of each sequence: all of `new`, and fewer for the later sequences."""
    return [max(1, c["new"] - (c["new"] * i) // (2 * c["batch"])) for i in range(c["batch"])]


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _inv_freq(c):
    """Radians per position of each pair (base 10000), scaled for a context `factor` times
    the original one: positions divided (linear), the base raised (ntk), or low frequencies
    divided and high ones kept with a ramp between (yarn: original length 32768, ramp from
    32 turns down to 1, and the attention factor 0.1 ln(factor) + 1 on the rotated part)."""
    rot, f = c["rot"], c["factor"]
    base = 10000.0
    if c["scaling"] == "ntk":
        base = base * f ** (rot / max(1, rot - 2))
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    inv = base ** (-i / rot)
    scale = 1.0
    if c["scaling"] == "linear":
        inv = inv / f
    if c["scaling"] == "yarn":
        turns = 32768 * inv / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        inv = inv * keep + inv / f * (1 - keep)
        scale = 0.1 * math.log(f) + 1
    return inv, scale


def _table(g, batch, blocks):
    """A shuffled block table over pools with a few spare blocks."""
    n_phys = batch * blocks + 5
    perm = torch.randperm(n_phys, generator=g, device=DEV)[: batch * blocks]
    return perm.view(batch, blocks).to(torch.int32).contiguous(), n_phys


def _select(g, lens, hkv, topk):
    """For each sequence and KV head the current block and top_k - 1 earlier ones, ascending,
    -1 where there are fewer."""
    rows = []
    for length in lens:
        cur = -(-length // BLOCK) - 1
        r = torch.rand(hkv, cur + 1, generator=g, device=DEV)
        r[:, cur] = 2.0
        n = min(topk, cur + 1)
        pick = r.topk(n, dim=1).indices.sort(dim=1).values
        pad = torch.full((hkv, topk - n), -1, device=DEV, dtype=pick.dtype)
        rows.append(torch.cat([pick, pad], dim=1))
    return torch.stack(rows).unsqueeze(2).to(torch.int32).contiguous()


def _kv_rows(g, shape, dt):
    """K or V rows as a model makes them: unit normal with an offset of each channel."""
    off = torch.randn(shape[-1], generator=g, device=DEV)
    x = torch.randn(shape, generator=g, device=DEV)
    return x.add_(off).to(dt)


def prepare(c, seed):
    g = _gen(seed)
    dt = TYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "rope":
        b, t, d = c["batch"], c["seq"], c["dim"]
        s["x"] = [torch.randn(n, generator=g, device=DEV, dtype=dt) for n in
                  ((b, t, c["hq"], d), (b, c["hkv"], t, d), (b, t, c["hkv"], d), (b, t, d))]
        s["y"] = [torch.empty_like(x) for x in s["x"]]
        inv, s["scale"] = _inv_freq(c)
        s["inv_freq"] = inv.to(DEV)
        # turns per position, in units of 2^-64 turns
        s["freqs"] = (inv / (2 * math.pi) * 2.0 ** 64).to(torch.int64).to(DEV)
        s["positions"], s["pos0"] = None, 0
        if c["positions"] == "lens":         # the new token is the last of its sequence
            s["positions"] = torch.randint(1, c["max_pos"] + 1, (b, t), generator=g, device=DEV,
                                           dtype=torch.int32)
            s["pos0"] = -1
        elif c["positions"] == "given":      # two documents packed into each row
            first = torch.randint(0, max(1, c["max_pos"] - t) + 1, (b, 1), generator=g, device=DEV)
            i = torch.arange(t, device=DEV)
            s["positions"] = torch.where(i < t // 3, i, i - t // 3 + first).to(torch.int32)
        return s
    blocks = -(-c["cap"] // BLOCK)
    if c["op"] == "pack":
        b, n = c["batch"], c["new"]
        s["k"] = _kv_rows(g, (b, c["hkv"], n, c["dim"]), dt)
        s["v"] = _kv_rows(g, (b, c["hkv"], n, c["dim"]), dt)
        counts = torch.tensor(_pack_counts(c), device=DEV)
        room = c["cap"] - n
        s["starts"] = torch.randint(0, room + 1, (b,), generator=g, device=DEV).to(torch.int32)
        s["lens"] = (s["starts"] + counts).to(torch.int32)
        s["table"], s["n_phys"] = _table(g, b, blocks) if c["paged"] else (None, b * blocks)
        s["cache"] = torch.zeros((s["n_phys"], c["hkv"], 160 * c["dim"]), dtype=torch.uint8, device=DEV)
        s["k_out"] = torch.zeros_like(s["k"])
        s["v_out"] = torch.zeros_like(s["v"])
        return s
    lens = _lens(c)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if c["op"] in ("packed", "mass"):
        b, d = c["batch"], c["dim"]
        s["q"] = torch.randn((b, 1, c["hq"], d), generator=g, device=DEV).to(dt)
        s["sel"] = _select(g, lens, c["hkv"], c["topk"])
        s["table"], s["n_phys"] = _table(g, b, blocks) if c["paged"] else (None, b * blocks)
        if c["op"] == "packed":
            cache = torch.empty((s["n_phys"], c["hkv"], 160 * d), dtype=torch.uint8, device=DEV)
            step = max(1, (1 << 28) // (c["hkv"] * BLOCK * d))
            for p in range(0, s["n_phys"], step):
                n = min(step, s["n_phys"] - p)
                k, v = (_kv_rows(g, (n, c["hkv"], BLOCK, d), dt) for _ in range(2))
                cache[p:p + n] = torch.cat([_records(k, False), _records(v, True)], dim=-1)
            s["cache"] = cache
        elif c["paged"]:
            s["k"], s["v"] = (_kv_rows(g, (s["n_phys"], c["hkv"], BLOCK, d), dt) for _ in range(2))
        else:
            s["k"], s["v"] = (_kv_rows(g, (b, c["hkv"], c["cap"], d), dt) for _ in range(2))
        s["mass"] = torch.zeros((b, c["hkv"], blocks), device=DEV)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((b, c["hq"], 1), device=DEV)
        return s
    # weights of a cache that has been decoded from for a while: a few blocks hold most
    b = c["batch"]
    s["mass"] = torch.randn((b, c["hkv"], blocks), generator=g, device=DEV).mul_(2).exp_()
    s["mass"].mul_((torch.arange(blocks, device=DEV) * BLOCK < s["lens"][:, None])[:, None])
    s["table"] = None
    s["kept"] = torch.empty((b, c["keep"]), dtype=torch.int32, device=DEV)
    s["new_lens"] = torch.empty((b,), dtype=torch.int32, device=DEV)
    s["mass_out"] = torch.empty_like(s["mass"])
    if c["paged"]:
        s["table"], _ = _table(g, b, blocks)
        s["table_out"] = torch.empty_like(s["table"])
        return s
    d, rows = c["dim"], _kept_len(c, c["cap"])
    s["src"] = [_kv_rows(g, n, dt) for n in ((b, c["hkv"], c["cap"], d), (b, c["hkv"], c["cap"], d),
                                             (b, c["cap"], d))]
    s["dst"] = [torch.empty((*x.shape[:-2], rows, d), dtype=dt, device=DEV) for x in s["src"]]
    return s


# ------------------------------------------------------------------------ plain forms

def _rope_plain(x, cos, sin, rot, interleaved):
    """Rotates the first `rot` dims of x [..., d]; cos, sin [..., rot / 2]."""
    xf = x.float()
    y = xf.clone()
    if interleaved:
        a, b = xf[..., 0:rot:2], xf[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = a * sin + b * cos
    else:
        h = rot // 2
        a, b = xf[..., :h], xf[..., h:rot]
        y[..., :h] = a * cos - b * sin
        y[..., h:rot] = a * sin + b * cos
    return y.to(x.dtype)


def _quantise(x):
    """4-bit codes of the groups of 32 dims, and each group's step and middle (bf16):
    step = (max - min) / 15, middle = min + 8 step, code = round((x - middle) / step) + 8."""
    xg = x.float().unflatten(-1, (-1, GROUP))
    hi, lo = xg.amax(-1), xg.amin(-1)
    fifteenth = torch.tensor(1 / 15, dtype=torch.float32, device=x.device)
    step = (hi * fifteenth - lo * fifteenth).bfloat16().float()
    step = torch.where(step < 2.0 ** -100, torch.zeros_like(step), step)
    mid = (lo + 8 * step).bfloat16().float()
    inv = torch.where(step > 0, 1 / step, torch.zeros_like(step))
    codes = (((xg - mid.unsqueeze(-1)) * inv.unsqueeze(-1)).round() + 8).clamp(0, 15)
    return codes.to(torch.uint8), step, mid


def _records(x, is_v):
    """The bytes that hold rows x [..., 128, d] of one block: 4-bit codes, then the planes
    [group][key] of the steps and of the middles (bf16)."""
    codes, step, mid = _quantise(x)                                # [..., 128, g, 32]
    lead = codes.shape[:-3]
    groups = codes.shape[-2]
    if is_v:
        # [r][key][group][4 dims 32 group + 4 r + i]; key pairs exchanged by fours of pairs
        # within the rows r that are odd (two groups: by r mod 4)
        n = codes.unflatten(-1, (8, 4)).movedim(-2, -4)            # [..., r, key, g, 4]
        n = n.unflatten(-3, (64, 2))                               # [..., r, pair, 2, g, 4]
        n = torch.gather(n, -4, _swizzle(groups, n.device).view(8, 64, 1, 1, 1).expand_as(n))
    else:
        # [key][c][group][8 dims 32 group + 8 c + i]
        n = codes.unflatten(-1, (4, 8)).movedim(-2, -3)            # [..., key, c, g, 8]
    n = n.reshape(*lead, -1, 2)
    packed = n[..., 0] | (n[..., 1] << 4)
    planes = [p.movedim(-1, -2).bfloat16().contiguous().view(torch.uint8).reshape(*lead, -1)
              for p in (step, mid)]
    return torch.cat([packed, *planes], dim=-1)


def _swizzle(groups, device):
    """Pair held at place p of row r of a V record: p with bit 2 (and 3) flipped by r."""
    r = torch.arange(8, device=device).unsqueeze(1)
    return torch.arange(64, device=device) ^ (4 * (r & (1 if groups == 4 else 3)))


def _values(rec, d, is_v):
    """The rows [..., 128, d] that the bytes of a block's K or V hold, in fp32."""
    groups = d // GROUP
    lead = rec.shape[:-1]
    codes, step, mid = rec.split([64 * d, 8 * d, 8 * d], dim=-1)
    nib = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(*lead, -1)
    if is_v:
        n = nib.reshape(*lead, 8, 64, 2, groups, 4)
        n = torch.gather(n, -4, _swizzle(groups, n.device).view(8, 64, 1, 1, 1).expand_as(n))
        n = n.reshape(*lead, 8, BLOCK, groups, 4).movedim(-4, -2)
    else:
        n = nib.reshape(*lead, BLOCK, 4, groups, 8).movedim(-3, -2)
    n = n.reshape(*lead, BLOCK, groups, GROUP).float()
    step, mid = (p.contiguous().view(torch.bfloat16).float().reshape(*lead, groups, BLOCK).movedim(-1, -2)
                 for p in (step, mid))
    return ((n - 8) * step.unsqueeze(-1) + mid.unsqueeze(-1)).reshape(*lead, BLOCK, d)


def _physical(s, blocks):
    """Physical block of every (sequence, logical block)."""
    if s["table"] is not None:
        return s["table"].long()
    b = s["case"]["batch"]
    return torch.arange(b * blocks, device=DEV).view(b, blocks)


def _token_rows(s, blocks):
    """Position of every new token, whether it is stored, and its block's place and its row."""
    c = s["case"]
    pos = s["starts"].long()[:, None] + torch.arange(c["new"], device=DEV)
    there = pos < s["lens"].long()[:, None]
    at = pos.clamp(max=blocks * BLOCK - 1)
    return there, _physical(s, blocks).gather(1, at // BLOCK), at % BLOCK


def _pack_plain(s):
    c = s["case"]
    blocks = -(-c["cap"] // BLOCK)
    there, phys, row = _token_rows(s, blocks)
    d, cache = c["dim"], s["cache"]
    for name, is_v in (("k", False), ("v", True)):
        half = cache[..., 80 * d * is_v:80 * d * (1 + is_v)]
        codes, step, mid = _quantise(s[name])                     # [b, h, n, g, 32]
        groups = codes.shape[-2]
        w = half[..., :64 * d]
        at = torch.arange(64 * d // BLOCK, device=DEV)            # the row's bytes, in order
        if is_v:
            per = 2 * groups                                      # bytes of one r
            n = codes.unflatten(-1, (8, 4)).movedim(-2, -3)       # [b, h, n, r, g, 4]
            r = at // per
            place = (row[..., None] // 2) ^ (4 * (r & (1 if groups == 4 else 3)))
            at = (r * BLOCK + place * 2 + row[..., None] % 2) * per + at % per
        else:
            n = codes.unflatten(-1, (4, 8)).movedim(-2, -3)       # [b, h, n, c, g, 8]
            at = row[..., None] * (d // 2) + at
        n = n.reshape(*codes.shape[:3], -1, 2)
        packed = n[..., 0] | (n[..., 1] << 4)
        p = there.nonzero(as_tuple=True)
        w.movedim(1, -1)[phys[p][:, None], at[p]] = packed.movedim(1, -1)[p]
        for k, plane in enumerate((step, mid)):
            rows = half[..., (64 + 8 * k) * d:(72 + 8 * k) * d].view(torch.bfloat16).unflatten(-1, (groups, BLOCK))
            rows.permute(0, 3, 1, 2)[phys[p], row[p]] = plane.movedim(1, 2).bfloat16()[p]
    # ... and the values that the cache now holds for these tokens, from the blocks they are in
    first = s["starts"].long()[:, None] // BLOCK
    near = (first + torch.arange(-(-c["new"] // BLOCK) + 1, device=DEV)).clamp(max=blocks - 1)
    rec = cache[_physical(s, blocks).gather(1, near)]                        # [b, blocks, h, bytes]
    row = s["starts"].long()[:, None] % BLOCK + torch.arange(c["new"], device=DEV)
    got = []
    for name, is_v in (("k", False), ("v", True)):
        held = _values(rec[..., 80 * d * is_v:80 * d * (1 + is_v)], d, is_v)  # [b, blocks, h, 128, d]
        held = held.transpose(1, 2).flatten(2, 3)
        x = held.gather(2, row[:, None, :, None].expand(*s[name].shape))
        out = s[name + "_out"]
        out.copy_(torch.where(there[:, None, :, None], x.to(out.dtype), out))
        got.append(out)
    return got


def _attend_plain(s, k, v):
    """Decode attention over the selected blocks' rows k, v [b, h, topk, 128, d] (fp32)."""
    c = s["case"]
    b, h, kk = c["batch"], c["hkv"], c["topk"]
    sel = s["sel"].view(b, h, kk).long()
    q = s["q"].float().view(b, h, c["hq"] // h, c["dim"])
    pos = sel.unsqueeze(-1) * BLOCK + torch.arange(BLOCK, device=DEV)
    seen = (sel.unsqueeze(-1) >= 0) & (pos < s["lens"].view(b, 1, 1, 1))
    z = (q @ k.flatten(2, 3).transpose(-1, -2)) / math.sqrt(c["dim"])
    z = z.masked_fill(~seen.flatten(2).unsqueeze(2), -math.inf)
    top = z.amax(-1, keepdim=True)
    e = (z - top.masked_fill(top == -math.inf, 0)).exp()
    total = e.sum(-1, keepdim=True)
    lse = (top + total.log()).view(b, c["hq"], 1)
    p = e / total
    v = v.masked_fill(~seen.unsqueeze(-1), 0)
    out = (p @ v.flatten(2, 3)).view(b, 1, c["hq"], c["dim"]).to(s["q"].dtype)
    weight = p.sum(2).unflatten(-1, (kk, BLOCK)).sum(-1)           # [b, h, topk]
    s["mass"].scatter_add_(2, sel.clamp(min=0), weight)
    return out, lse


def _evict_plain(s):
    c = s["case"]
    mass, lens = s["mass"], s["lens"].long()
    b, h, blocks = mass.shape
    score = mass[:, 0]
    for g in range(1, h):                                          # head order: it fixes the fp32 sum
        score = score + mass[:, g]
    n = (lens + BLOCK - 1) // BLOCK
    i = torch.arange(blocks, device=DEV).expand(b, blocks)
    inside = i < n[:, None]
    forced = inside & ((i < c["first"]) | (i >= n[:, None] - c["recent"]))
    score = score.masked_fill(forced, math.inf).masked_fill(~inside, -math.inf)
    order = score.sort(dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, i)
    n_kept = n.clamp(max=c["keep"])
    keeps = inside & (rank < n_kept[:, None])
    kind = torch.where(keeps, 0, torch.where(inside, 1, 2))
    place = kind.sort(dim=1, stable=True).indices                  # kept, evicted, the rest
    held = i < n_kept[:, None]
    pad = max(0, c["keep"] - blocks)
    kept = torch.nn.functional.pad(place.masked_fill(~held, -1), (0, pad), value=-1)[:, :c["keep"]].to(torch.int32)
    new_lens = (lens - (n - n_kept) * BLOCK).to(torch.int32)
    moved = mass.gather(2, place.unsqueeze(1).expand(b, h, blocks)).masked_fill(~held.unsqueeze(1), 0)
    if c["paged"]:
        return kept, new_lens, moved, s["table"].gather(1, place)
    rows = (place[:, :, None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten(1)
    rows = rows[:, :s["dst"][0].shape[-2]]
    j = torch.arange(b, device=DEV)[:, None]
    return (kept, new_lens, moved, s["src"][0].transpose(1, 2)[j, rows].transpose(1, 2).contiguous(),
            s["src"][1].transpose(1, 2)[j, rows].transpose(1, 2).contiguous(), s["src"][2][j, rows])


def run(s):
    c = s["case"]
    if own:
        return _run_own(s)
    if c["op"] == "rope":
        i = torch.arange(c["seq"], device=DEV).expand(c["batch"], c["seq"]) if s["positions"] is None else s["positions"]
        angle = (i.double() + s["pos0"]).unsqueeze(-1) * s["inv_freq"]
        cos = (angle.cos() * s["scale"]).float()
        sin = (angle.sin() * (-s["scale"] if c["inverse"] else s["scale"])).float()
        q, k, iq, ik = s["x"]
        by_token, by_head = (cos.unsqueeze(2), sin.unsqueeze(2)), (cos.unsqueeze(1), sin.unsqueeze(1))
        return [_rope_plain(q, *by_token, c["rot"], c["interleaved"]),
                _rope_plain(k, *by_head, c["rot"], c["interleaved"]),
                _rope_plain(iq, *by_token, c["rot"], c["interleaved"]),
                _rope_plain(ik, cos, sin, c["rot"], c["interleaved"])]
    if c["op"] == "pack":
        return _pack_plain(s)
    if c["op"] == "evict":
        return _evict_plain(s)
    b, h, d = c["batch"], c["hkv"], c["dim"]
    blocks = -(-c["cap"] // BLOCK)
    sel = s["sel"].view(b, h, -1).long().clamp(min=0)
    j = torch.arange(h, device=DEV).view(1, h, 1)
    if c["op"] == "packed":
        phys = _physical(s, blocks).unsqueeze(1).expand(b, h, blocks).gather(2, sel)
        rec = s["cache"][phys, j]
        k, v = _values(rec[..., :80 * d], d, False), _values(rec[..., 80 * d:], d, True)
    elif c["paged"]:
        phys = _physical(s, blocks).unsqueeze(1).expand(b, h, blocks).gather(2, sel)
        k, v = s["k"][phys, j].float(), s["v"][phys, j].float()
    else:
        rows = (sel.unsqueeze(-1) * BLOCK + torch.arange(BLOCK, device=DEV)).clamp(max=c["cap"] - 1)
        i = torch.arange(b, device=DEV).view(b, 1, 1, 1)
        k, v = (s[n][i, j.unsqueeze(-1), rows].float() for n in ("k", "v"))
    out, lse = _attend_plain(s, k, v)
    return [out, lse, s["mass"]] if c.get("mass", True) else [out, lse]


# ---------------------------------------------------------------- the package's calls

def _plan(s):
    """What a user's program keeps between steps: the shape and the workspace."""
    from block_sparse_gqa_02_gb300 import _lib
    c = s["case"]
    if c["op"] == "rope":
        q, k, iq, ik = zip(s["x"], s["y"])
        desc = _lib.make_rope(c["batch"], c["seq"], c["dtype"], pos_offset=s["pos0"], scale=s["scale"],
                              interleaved=c["interleaved"], inverse=c["inverse"])
        rows = [(*q, s["freqs"], False), (*k, s["freqs"], True), (*iq, s["freqs"], False), (*ik, s["freqs"], True)]
        return _lib, desc, _lib.make_rope_tensors(rows)
    hq = c.get("hq", c["hkv"])
    shape = _lib.make_shape(c["batch"], 1, c["cap"], hq, c["hkv"], c["dim"], 128, BLOCK, c.get("topk", 1), 1,
                            c["dtype"])
    more = None
    if c["op"] == "mass":
        more = torch.empty(_lib.msa_workspace_bytes(shape, 4) // 4 + 4, device=DEV)
    if c["op"] == "evict" and not c["paged"]:
        more = _lib.make_gather_tensors(list(zip(s["src"], s["dst"])))
    return _lib, shape, more


def _run_own(s):
    c = s["case"]
    if "plan" not in s:
        s["plan"] = _plan(s)
    lib, shape, more = s["plan"]
    if c["op"] == "rope":
        lib.msa_rope(shape, more, s["positions"])
        return s["y"]
    if c["op"] == "pack":
        lib.msa_cache_pack(shape, c["new"], s["starts"], s["lens"], s["table"], s["n_phys"], s["k"], s["v"], s["cache"])
        lib.msa_cache_unpack(shape, c["new"], s["starts"], s["lens"], s["table"], s["n_phys"], s["cache"], s["k_out"],
                             s["v_out"])
        return [s["k_out"], s["v_out"]]
    if c["op"] == "packed":
        lib.msa_sparse_decode_packed(shape, s["lens"], s["table"], s["n_phys"], s["q"], s["cache"], s["sel"], s["out"],
                                     s["lse"], s["mass"] if c["mass"] else None)
        return [s["out"], s["lse"], s["mass"]] if c["mass"] else [s["out"], s["lse"]]
    if c["op"] == "mass":
        paged = (s["lens"], s["table"], s["n_phys"]) if c["paged"] else (None, None, 0)
        lib.msa_sparse_decode_mass(shape, *paged, s["q"], s["k"], s["v"], s["sel"], s["out"], s["lse"], s["mass"], more)
        return [s["out"], s["lse"], s["mass"]]
    lib.msa_cache_evict(shape, c["keep"], c["first"], c["recent"], s["lens"], s["mass"], s["table"], s["kept"],
                        s["new_lens"], s["mass_out"], s.get("table_out"))
    if c["paged"]:
        return s["kept"], s["new_lens"], s["mass_out"], s["table_out"]
    lib.msa_cache_gather(c["batch"], more, s["kept"], BLOCK)
    return s["kept"], s["new_lens"], s["mass_out"], *s["dst"]


# ------------------------------------------------------- the definitions, in 64 bits

def _exact_rope(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    pos = (torch.arange(c["seq"], device=DEV).repeat(c["batch"], 1) if s["positions"] is None
           else s["positions"].long() + s["pos0"]).double()
    # the rotation is a product with exp(i angle) of the pair taken as a complex number
    turn = torch.polar(torch.full((), s["scale"], dtype=torch.float64, device=DEV),
                       pos[:, :, None] * s["inv_freq"] * (-1 if c["inverse"] else 1))
    got = []
    for x, at in zip(s["x"], ((slice(None), slice(None), None), (slice(None), None), (slice(None), slice(None), None), ())):
        y = x.double()
        w = turn[at] if at else turn
        head = y[..., :rot]
        pairs = head.unflatten(-1, (half, 2)) if c["interleaved"] else head.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
        y[..., :rot] = (z if c["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        got.append(y)
    return got


def _exact_codes(x):
    """Values after the round trip. The definition fixes the step and the middle as single
    precision results rounded to bf16, so those two are formed in single precision."""
    g = x.to(torch.float32).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    top, low = g.max(-1, keepdim=True).values, g.min(-1, keepdim=True).values
    f = torch.full_like(top, 1 / 15)
    step = torch.sub(torch.mul(top, f), torch.mul(low, f)).to(torch.bfloat16).float()
    step[step < 2.0 ** -100] = 0
    mid = torch.add(low, step, alpha=8).to(torch.bfloat16)
    inv = torch.nan_to_num(step.reciprocal(), posinf=0.0)
    n = torch.round((g - mid.float()) * inv).clamp_(-8, 7).double()
    return (n * step.double() + mid.double()).reshape(x.shape)


def _exact_block(rec, d, is_v):
    """One block's rows [128, d] from its record, dim by dim as the format says."""
    groups = d // GROUP
    dim = torch.arange(d, device=DEV)[None, :]
    key = torch.arange(BLOCK, device=DEV)[:, None]
    g, i = dim // GROUP, dim % GROUP
    if is_v:
        r = i // 4
        pair = (key // 2) ^ (4 * (r % (2 if groups == 4 else 4)))
        byte = (r * BLOCK + pair * 2 + key % 2) * 2 * groups + g * 2 + (i % 4) // 2
    else:
        byte = key * (d // 2) + (i // 8) * 4 * groups + g * 4 + (i % 8) // 2
    nibble = (rec[..., byte].long() // torch.where(i % 2 == 1, 16, 1)) % 16
    planes = rec[..., 64 * d:].contiguous().view(torch.bfloat16).double()
    at = g * BLOCK + key
    return (nibble.double() - 8) * planes[..., at] + planes[..., 4 * d + at]


def _exact_attention(s):
    c = s["case"]
    b, h, d, group = c["batch"], c["hkv"], c["dim"], c["hq"] // c["hkv"]
    blocks = -(-c["cap"] // BLOCK)
    out = torch.zeros((b, 1, c["hq"], d), dtype=torch.float64, device=DEV)
    lse = torch.full((b, c["hq"], 1), -math.inf, dtype=torch.float64, device=DEV)
    mass = torch.zeros((b, h, blocks), dtype=torch.float64, device=DEV)
    lens, sel = s["lens"].tolist(), s["sel"].tolist()
    for i in range(b):
        for j in range(h):
            chosen = [x for x in sel[i][j][0] if x >= 0]
            at = torch.tensor(chosen, device=DEV)
            if c["op"] == "packed" or c["paged"]:
                phys = s["table"][i].long()[at] if s["table"] is not None else i * blocks + at
            if c["op"] == "packed":
                rec = s["cache"][phys, j]
                k, v = _exact_block(rec[:, :80 * d], d, False), _exact_block(rec[:, 80 * d:], d, True)
            elif c["paged"]:
                k, v = s["k"][phys, j].double(), s["v"][phys, j].double()
            else:
                rows = (at[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)).clamp(max=c["cap"] - 1)
                k, v = s["k"][i, j, rows].double(), s["v"][i, j, rows].double()
            here = (at[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten() < lens[i]
            k, v = k.reshape(-1, d)[here], v.reshape(-1, d)[here]
            z = s["q"][i, 0, j * group:(j + 1) * group].double() @ k.T * d ** -0.5
            norm = torch.logsumexp(z, dim=1)
            w = torch.exp(z - norm[:, None])
            out[i, 0, j * group:(j + 1) * group] = w @ v
            lse[i, j * group:(j + 1) * group, 0] = norm
            owner = at.repeat_interleave(BLOCK)[here]
            mass[i, j].index_add_(0, owner, w.sum(0))
    return [out, lse, mass] if c.get("mass", True) else [out, lse]


def _exact_evict(s):
    import numpy as np
    c = s["case"]
    mass, lens = s["mass"].cpu().numpy(), s["lens"].tolist()
    b, h, blocks = mass.shape
    moved = np.zeros_like(mass, dtype=np.float64)
    rows = []
    for i in range(b):
        score = mass[i, 0].copy()
        for g in range(1, h):
            score = np.add(score, mass[i, g], dtype=np.float32)
        n = -(-lens[i] // BLOCK)
        must = [x for x in range(n) if x < c["first"] or x >= n - c["recent"]]
        rest = sorted(set(range(n)) - set(must), key=lambda x: (-score[x], x))
        keep = sorted((must + rest)[:min(n, c["keep"])])
        moved[i, :, :len(keep)] = mass[i][:, keep]
        rows.append([x * BLOCK + r for x in keep for r in range(BLOCK) if x * BLOCK + r < lens[i]])
    if c["paged"]:
        return [None, None, torch.from_numpy(moved), None]
    got = [None, None, torch.from_numpy(moved)]
    for x in s["src"]:
        got.append(torch.stack([x[i][..., torch.tensor(rows[i], device=DEV), :] for i in range(b)]).double())
    return got


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _exact_rope(s)
    if c["op"] == "pack":
        there = torch.arange(c["new"], device=DEV) < (s["lens"] - s["starts"])[:, None]
        return [_exact_codes(s[n]) * there[:, None, :, None] for n in ("k", "v")]
    if c["op"] == "evict":
        return _exact_evict(s)
    return _exact_attention(s)
