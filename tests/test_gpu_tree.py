"""Decode over a tree of drafted tokens: every call against the fp64 oracle."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib
from oracle import tree_ops
from tests.canary import guarded_like
from tests.tree_cases import DTYPES, Tree, random_parents

pytestmark = pytest.mark.gpu


def _ok():
    _lib.msa_get_device_status()


# -------------------------------------------------------------------------- paths

@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("kind", ["chain", "tree", "bad", "star"])
def test_mask(n, kind):
    rng = np.random.default_rng(n)
    lens, cap = [0, 5, 970, 1000, 999], 1000
    parents = random_parents(rng, 5, n, kind)
    shape = _lib.make_shape(5, n, cap, 4, 4, 128, 128, 128, 1, 1)
    mask, pos = guarded_like((5, n), torch.int64), guarded_like((5, n), torch.int32)
    lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
    _lib.msa_tree_mask(shape, lens_t, torch.tensor(parents, dtype=torch.int32).cuda(), mask.tensor,
                       pos.tensor)
    _ok()
    for b in range(5):
        want = tree_ops.paths(parents[b], lens[b], cap)
        got = [x % (1 << 64) for x in mask.tensor[b].tolist()]
        assert got == [tree_ops.word(p) for p in want]
        assert pos.tensor[b].tolist() == [lens[b] + len(p) - 1 if p else -1 for p in want]
    mask.check("mask")
    pos.check("positions")
    _lib.msa_tree_mask(shape, lens_t, torch.tensor(parents, dtype=torch.int32).cuda(), mask.tensor)


# ------------------------------------------------------------- 8-bit index keys

def _special(x):
    """Rows of zeros, one large value, tiny ones, the ends of the range, not finite ones."""
    x = x.clone()
    flat = x.view(-1, x.shape[-1])
    for r, fill in enumerate([0.0, 2.0 ** -130, 3e38, 448.0, 450.0]):
        if r < flat.shape[0]:
            flat[r] = flat[r] * 0 + fill
    if flat.shape[0] > 8:
        flat[5, 3] = float("inf")
        flat[6, 0] = float("nan")
        flat[7] *= 2.0 ** -120
        flat[8, 1] = 1e30
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("idim", [64, 128])
@pytest.mark.parametrize("n,cap,paged,starts", [
    (1, 1, False, None), (1, 700, True, None), (130, 1000, True, [0, 127, 869, 500]),
    (333, 333, False, [0, 0, 0, 0]), (700, 640, True, [-100, 3, 600, 639]), (64, 64, False, None)])
def test_index_pack(dtype, idim, n, cap, paged, starts):
    B, nB = 4, -(-cap // 128)
    g = torch.Generator().manual_seed(n)
    dt = DTYPES[dtype]
    lens = [cap, max(0, cap - 1), cap // 2, 0]
    x = _special((torch.randn(B, n, idim, generator=g) * torch.randn(B, n, 1, generator=g).exp()).to(dt))
    shape = _lib.make_shape(B, 1, cap, 4, 4, 128, idim, 128, 1, 1, dtype)
    n_phys = B * nB + 2 * paged
    perm = torch.randperm(n_phys, generator=g)[:B * nB].view(B, nB)
    table = perm.to(torch.int32).cuda() if paged else None
    where = perm if paged else torch.arange(B * nB).view(B, nB)
    rec = 128 * (idim + 1)
    before = torch.randint(0, 256, (n_phys, rec), generator=g, dtype=torch.uint8)
    cache = guarded_like((n_phys, rec), torch.uint8)
    cache.tensor.copy_(before)
    lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
    starts_t = torch.tensor(starts, dtype=torch.int32).cuda() if starts else None
    args = starts_t, lens_t, table, n_phys
    _lib.msa_index_pack(shape, n, *args, x.cuda(), cache.tensor)
    out = guarded_like((B, n, idim), dt, fill=7.0)
    _lib.msa_index_unpack(shape, n, *args, cache.tensor, out.tensor)
    _ok()
    codes, exps, val = tree_ops.quantise(x.float().numpy())
    want, want_out = before.clone(), torch.full((B, n, idim), 7.0, dtype=torch.float64)
    for b in range(B):
        first = starts[b] if starts else lens[b] - n
        for i in range(n):
            pos = first + i
            if not 0 <= pos < lens[b]:
                continue
            r = want[int(where[b, pos // 128])]
            j = pos % 128
            r[j * idim:(j + 1) * idim] = torch.tensor(codes[b, i])
            r[128 * idim + j] = int(exps[b, i])
            want_out[b, i] = torch.tensor(val[b, i])
    got = cache.tensor.cpu()
    # a zero's sign is kept too, so the bytes are equal; NaN rows hold NaN codes of either sign
    assert torch.equal(got, want)
    y = out.tensor.cpu().double()
    assert torch.equal(torch.isnan(y), torch.isnan(want_out))
    want_out = want_out.to(dt).double()            # 2^128 and above, and below the type's range
    fine = ~torch.isnan(want_out)
    assert torch.equal(y[fine], want_out[fine])
    cache.check("cache")
    out.check("rows")


def test_index_pack_skips_bad_table_entries():
    B, cap, idim = 2, 256, 128
    shape = _lib.make_shape(B, 1, cap, 4, 4, 128, idim, 128, 1, 1)
    table = torch.tensor([[0, 5], [-1, 2 ** 31 - 1]], dtype=torch.int32).cuda()
    cache = guarded_like((3, 129 * 128), torch.uint8, fill=9)
    x = torch.randn(B, cap, idim, device="cuda").bfloat16()
    _lib.msa_index_pack(shape, cap, None, None, table, 3, x, cache.tensor)
    y = torch.full_like(x, 5.0)
    _lib.msa_index_unpack(shape, cap, None, None, table, 3, cache.tensor, y)
    torch.cuda.synchronize()
    assert (cache.tensor[1:] == 9).all() and not (cache.tensor[0] == 9).all()
    assert (y[0, 128:] == 5).all() and (y[1] == 5).all() and not (y[0, :128] == 5).all()
    cache.check()


# ------------------------------------------------------------------ index scores

SCORES = [
    # the tensor-core form's shapes: lengths inside, at and past block ends; one token to 64
    dict(lens=[0, 1, 127, 128], n=5, cap=300),
    dict(lens=[1000, 129, 1023, 1024], n=16, cap=1100, paged=True),
    dict(lens=[5000], n=1, cap=5001),
    dict(lens=[3000, 17], n=64, cap=3100, kind="chain"),
    dict(lens=[700, 250], n=64, cap=800, kind="bad", paged=True),
    dict(lens=[100, 2000, 120], n=33, cap=2100, hkv=8, kind="chain", paged=True),
    dict(lens=[600, 120], n=64, cap=700, hkv=8),
    dict(lens=[600], n=7, cap=700, hkv=1),
    dict(lens=[640, 640], n=9, cap=645, hkv=2, kind="chain"),           # the drafts fill the cache
    dict(lens=[200] * 33, n=3, cap=260, hkv=3),
    # 16-bit keys
    dict(lens=[0, 1, 127, 128], n=5, cap=300, packed=False),
    dict(lens=[1000, 129, 1023, 1024], n=16, cap=1100, packed=False, paged=True),
    dict(lens=[2000, 20], n=64, cap=2100, kind="chain", packed=False),
    dict(lens=[600, 100], n=64, cap=700, hkv=8, packed=False, kind="bad"),
    # caches shorter than a tile, odd head counts, more sequences than SMs
    dict(lens=[0, 1, 2], n=1, cap=3),
    dict(lens=[0, 1, 2], n=2, cap=3, packed=False, kind="chain"),
    dict(lens=[300, 260], n=5, cap=310, hkv=33, group=1, packed=False),
    dict(lens=[i % 140 for i in range(170)], n=3, cap=150, hkv=2, paged=True),
    dict(lens=[0] * 160, n=2, cap=129),
    # other dims, types and blocks
    dict(lens=[700, 0, 130], n=6, cap=800, idim=64),
    dict(lens=[700, 0, 130], n=6, cap=800, dtype="f32", paged=True),
    dict(lens=[300, 64], n=40, cap=400, idim=64, packed=False, block=32, kind="chain"),
    dict(lens=[300, 64], n=9, cap=400, dtype="f32", packed=False, block=200, paged=True),
    dict(lens=[30, 4], n=20, cap=60, dtype="bf16", packed=False, block=1, kind="chain", paged=True),
]


@pytest.mark.parametrize("c", SCORES, ids=lambda c: "-".join(f"{k}{v if k != 'lens' else len(v)}" for k, v in c.items()))
def test_scores(c):
    t = Tree(seed=len(c["lens"]) * 100 + c["n"], **c)
    s = t.shape
    out = guarded_like((s.batch, s.n_heads_kv, t.n, t.nB), torch.float32)
    d = t.dev
    _lib.msa_index_scores_tree(s, t.seq_lens, t.table, t.n_phys, t.mask, d["iq"], d["ik"], d["ikd"],
                               out.tensor, packed=t.packed)
    _ok()
    got, want = out.tensor.cpu().double().numpy(), t.scores()
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    assert not np.isnan(got).any()
    fine = np.isfinite(want)
    err = np.abs(np.where(fine, got, 0) - np.where(fine, want, 0))
    assert (err <= t.score_bound() + 2.0 ** -23 * np.abs(np.where(fine, want, 0))).all(), err.max()
    out.check("scores")


# --------------------------------------------------------------------- selection

@pytest.mark.parametrize("c,topk", [
    (dict(lens=[1000, 129, 0, 1023], n=16, cap=1100), 3), (dict(lens=[900], n=64, cap=1000, kind="chain"), 1),
    (dict(lens=[900, 5], n=20, cap=1000, kind="bad", hkv=2), 20), (dict(lens=[20], n=9, cap=40, block=2, packed=False, kind="chain"), 5),
    (dict(lens=[300000], n=2, cap=300100, hkv=1, group=1, dim=64, idim=64), 64)])
def test_selection(c, topk):
    t = Tree(seed=3, topk=topk, **c)
    s = t.shape
    rng = np.random.default_rng(1)
    x = rng.integers(-4, 4, (s.batch, s.n_heads_kv, t.n, t.nB)).astype(np.float32)   # many ties
    x[rng.random(x.shape) < 0.1] = -np.inf
    x[rng.random(x.shape) < 0.1] = -0.0
    sel = guarded_like((s.batch, s.n_heads_kv, t.n, topk), torch.int32)
    _lib.msa_block_topk_tree(s, t.seq_lens, t.mask, torch.tensor(x).cuda(), sel.tensor)
    _ok()
    for b in range(s.batch):
        for h in range(s.n_heads_kv):
            for i, path in enumerate(t.paths[b]):
                pos = t.lens[b] + len(path) - 1 if path else -1
                assert sel.tensor[b, h, i].tolist() == tree_ops.select(x[b, h, i], pos, s.block_size, topk)
    sel.check("sel")


@pytest.mark.parametrize("lens,n,topk", [([1_199_000, 700_000], 2, 64), ([1_199_000], 1, 700), ([140_000, 90_000], 3, 300),
                                         ([1_040_000], 3, 64), ([127_000], 5, 129)])
def test_selection_of_many_blocks(lens, n, topk):
    """Distinct scores (ranked candidates), and scores with few values (ties over the whole row)."""
    cap = max(lens) + 64
    shape = _lib.make_shape(len(lens), n, cap, 2, 2, 64, 64, 128, topk, 1)
    paths, mask = _random_tree(len(lens), n, lens, cap, 1)
    lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
    rng = np.random.default_rng(2)
    shp = (len(lens), 2, n, shape.n_blocks)
    for x in (rng.standard_normal(shp), rng.integers(0, 5, shp), np.full(shp, -np.inf),
              np.where(rng.random(shp) < 0.01, rng.standard_normal(shp), -1.0)):
        x = x.astype(np.float32)
        sel = guarded_like((*shp[:3], topk), torch.int32)
        _lib.msa_block_topk_tree(shape, lens_t, mask, torch.tensor(x).cuda(), sel.tensor)
        _ok()
        for b, length in enumerate(lens):
            for h in range(2):
                for i, path in enumerate(paths[b]):
                    want = tree_ops.select(x[b, h, i], length + len(path) - 1, 128, topk)
                    assert sel.tensor[b, h, i].tolist() == want
        sel.check("sel")


# --------------------------------------------------------------------- attention

ATTEND = [
    dict(lens=[0, 1, 127, 128], n=5, cap=300),
    dict(lens=[1000, 129, 1023, 1024], n=16, cap=1100, paged=True, topk=6),
    dict(lens=[3000], n=1, cap=3001, topk=24),
    dict(lens=[1500, 17], n=64, cap=1600, kind="chain", topk=5, sel_frac=0.6),
    dict(lens=[700, 250], n=64, cap=800, kind="bad", paged=True, hkv=2),
    dict(lens=[1990, 100], n=8, cap=2000, kind="star", topk=9, sel_frac=0.7),
    dict(lens=[600], n=7, cap=700, hkv=1, group=1),
    dict(lens=[600, 90], n=40, cap=700, hkv=2, group=5, kind="chain"),
    dict(lens=[600], n=33, cap=700, hkv=2, group=33, paged=True),
    dict(lens=[500], n=3, cap=600, hkv=1, group=64),
    dict(lens=[640, 640], n=9, cap=645, hkv=2, kind="chain", topk=2),
    dict(lens=[200] * 20, n=3, cap=260, hkv=8, group=2, topk=1),
    dict(lens=[1200, 0], n=24, cap=1300, hkv=4, group=8, topk=300),
    dict(lens=[900], n=12, cap=1000, topk=4, key_scale=12.0),            # peaked rows, rescaled often
    dict(lens=[0, 1, 2], n=2, cap=3, kind="chain"),
    dict(lens=[i % 140 for i in range(90)], n=3, cap=150, hkv=2, paged=True),
    dict(lens=[900, 140], n=20, cap=1000, dim=64, group=8, kind="chain"),
    dict(lens=[900, 140], n=6, cap=1000, dtype="f32", group=16, paged=True),
    dict(lens=[300, 64], n=40, cap=400, dtype="f32", dim=64, group=3, packed=False, block=32, kind="chain"),
    dict(lens=[300, 64], n=9, cap=400, packed=False, block=200, paged=True, group=4),
    dict(lens=[30, 4], n=20, cap=60, packed=False, block=1, kind="chain", paged=True, topk=30, group=2),
]


@pytest.mark.parametrize("c", ATTEND, ids=lambda c: "-".join(f"{k}{v if k != 'lens' else len(v)}" for k, v in c.items()))
def test_attention(c):
    t = Tree(seed=len(c["lens"]) * 100 + c["n"], **c)
    s, d = t.shape, t.dev
    out = guarded_like((s.batch, t.n, s.n_heads_q, s.head_dim), t.dt)
    lse = guarded_like((s.batch, s.n_heads_q, t.n), torch.float32)
    ws = guarded_like((_lib.msa_workspace_bytes(s, 5) // 4,), torch.float32)
    args = (s, t.seq_lens, t.table, t.n_phys, t.mask, d["q"], d["k"], d["v"], d["kd"], d["vd"], d["sel"])
    _lib.msa_sparse_decode_tree(*args, out.tensor, lse.tensor, ws.tensor)
    _ok()
    want, want_lse, tol, tol_lse = t.attend()
    got, got_lse = out.tensor.cpu().double().numpy(), lse.tensor.cpu().double().numpy()
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(want_lse))
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), (err.max(), (err / np.maximum(tol, 1e-30)).max())
    fine = np.isfinite(want_lse)
    err = np.abs(np.where(fine, got_lse, 0) - np.where(fine, want_lse, 0))
    assert (err <= tol_lse).all(), err.max()
    for x in (out, lse, ws):
        x.check()
    # without lse, and again: the same bits
    again = torch.empty_like(out.tensor)
    _lib.msa_sparse_decode_tree(*args, again, None, ws.tensor)
    torch.cuda.synchronize()
    assert torch.equal(again, out.tensor)


# ------------------------------------------------------------------------ commit

@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_commit(paged, in_place, dtype):
    t = Tree(lens=[0, 126, 290, 300, 255], n=11, cap=300, paged=paged, kind="star", hkv=3, group=1, dim=64, dtype=dtype)
    s, d = t.shape, t.dev
    accepted = [[3, 4, 10, -1, 2], [0, 0, 7, 7, 1], [5, 4, 3, 2, 1], [1, 2, 3, 4, 5], [-1, 3, 4, 5, 6]]
    counts = [3, 5, 5, 0, 0]
    acc = torch.tensor(accepted, dtype=torch.int32).cuda()
    names = [("kd", "k"), ("vd", "v"), ("ikd", "ik")]
    before = {n: d[n].clone() for _, n in names}
    guards = {}
    for _, n in names:
        guards[n] = guarded_like(d[n].shape, d[n].dtype)
        guards[n].tensor.copy_(d[n])
    lens = t.seq_lens.clone()
    new = lens if in_place else torch.full_like(lens, -5)
    rows = [(d[a], guards[b].tensor) for a, b in names[:2]]
    tensors = _lib.make_commit_tensors(rows, [(d["ikd"], guards["ik"].tensor)])
    _lib.msa_tree_commit(s, lens, t.table, t.n_phys, acc, tensors, new)
    _ok()
    assert new.tolist() == [t.lens[b] + counts[b] for b in range(5)]
    want = {n: x.clone() for n, x in before.items()}
    for b in range(5):
        for i in range(counts[b]):
            pos, a = t.lens[b] + i, accepted[b][i]
            phys = int(t.phys[b, pos // 128])
            for src, dst in names[:2]:
                if paged:
                    want[dst][phys, :, pos % 128] = d[src][b, :, a]
                else:
                    want[dst][b, :, pos] = d[src][b, :, a]
            r, q = want["ik"][phys], d["ikd"][b]
            j = pos % 128
            r[j * 128:(j + 1) * 128] = q[a * 128:(a + 1) * 128]
            r[128 * 128 + j] = q[128 * 128 + a]
    for _, n in names:
        assert torch.equal(guards[n].tensor.view(torch.uint8), want[n].view(torch.uint8)), n
        guards[n].check(n)


def test_commit_bad_table_entry_and_long_lists():
    n = 64
    shape = _lib.make_shape(2, n, 512, 4, 4, 64, 128, 128, 1, 1)
    src = torch.randn(2, 4, n, 64, device="cuda").bfloat16()
    pool = guarded_like((5, 4, 128, 64), torch.bfloat16, fill=2.0)
    table = torch.tensor([[3, 9, -1, 2 ** 30], [0, 1, 2, 4]], dtype=torch.int32).cuda()
    acc = torch.arange(n, dtype=torch.int32).repeat(2, 1).cuda()
    lens = torch.tensor([100, 470], dtype=torch.int32).cuda()
    new = torch.zeros_like(lens)
    _lib.msa_tree_commit(shape, lens, table, 5, acc, _lib.make_commit_tensors([(src, pool.tensor)]), new)
    torch.cuda.synchronize()
    assert new.tolist() == [164, 512]
    want = torch.full_like(pool.tensor, 2.0)
    want[3, :, 100:] = src[0, :, :28]
    want[4, :, 86:] = src[1, :, :42]
    assert torch.equal(pool.tensor, want)
    pool.check()


# ------------------------------------------- long ranges: many blocks for every CTA

def _random_tree(batch, n, lens, cap, seed):
    rng = np.random.default_rng(seed)
    parents = random_parents(rng, batch, n, "tree")
    paths = [tree_ops.paths(parents[b], lens[b], cap) for b in range(batch)]
    words = [[tree_ops.word(p) for p in row] for row in paths]
    return paths, torch.tensor([[w - (1 << 64) if w >> 63 else w for w in row] for row in words]).cuda()


@pytest.mark.parametrize("n", [1, 5, 12, 16, 20, 28, 32, 64])
@pytest.mark.parametrize("packed", [True, False])
def test_scores_long_ranges(n, packed):
    """160 sequences of up to 60 blocks: more sequences than SMs, so that every CTA's ring, its
    accumulators and its result buffers wrap many times.  Cached blocks only; fp64 on the GPU."""
    B, cap, d, h = 160, 7700, 128, 4
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(4000, cap - 64, B)]
    _, mask = _random_tree(B, n, lens, cap, n)
    g = torch.Generator(device="cuda").manual_seed(n)
    nB = -(-cap // 128)
    ik = torch.randn(B, cap, d, generator=g, device="cuda").bfloat16()
    iq = torch.randn(B, n, h, d, generator=g, device="cuda").bfloat16()
    ikd = torch.randn(B, n, d, generator=g, device="cuda").bfloat16()
    lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
    shape = _lib.make_shape(B, n, cap, h, h, d, d, 128, 1, 1)
    cache, drafts, keys = ik, ikd, ik
    if packed:
        cache = torch.zeros(B * nB, 129 * 128, dtype=torch.uint8, device="cuda")
        _lib.msa_index_pack(shape, cap, None, None, None, B * nB, ik, cache)
        keys = torch.empty_like(ik)
        _lib.msa_index_unpack(shape, cap, None, None, None, B * nB, cache, keys)
        drafts = torch.zeros(B, 129 * 128, dtype=torch.uint8, device="cuda")
        one = _lib.make_shape(B, 1, n, h, h, d, d, 128, 1, 1)
        _lib.msa_index_pack(one, n, None, None, None, B, ikd, drafts)
    out = guarded_like((B, h, n, nB), torch.float32)
    _lib.msa_index_scores_tree(shape, lens_t, None, B * nB, mask, iq, cache, drafts, out.tensor, packed=packed)
    _ok()
    for b in range(B):
        whole = lens[b] // 128
        k = keys[b, :whole * 128].double()
        z = (iq[b].double().flatten(0, 1) @ k.T) * d ** -0.5               # [n h, keys]
        want = z.view(n, h, whole, 128).amax(-1).transpose(0, 1)
        # fp32 sums of 128 products, twice over, and what the queries' two parts may miss
        mag = (iq[b].double().abs().flatten(0, 1) @ k.abs().T).amax(-1)
        lost = iq[b].double().abs().amax(-1).flatten() * k.abs().sum(-1).max() * (2.0 ** -18 if packed else 0)
        tol = ((2 * 130 * 2.0 ** -24 * mag + lost) * d ** -0.5).view(n, h).T[..., None] + 2.0 ** -23 * want.abs()
        got = out.tensor[b, :, :, :whole].double()
        assert ((got - want).abs() <= tol).all(), (b, float((got - want).abs().max()))
    out.check("scores")


@pytest.mark.parametrize("c", [dict(n=4, group=16), dict(n=11, group=16, paged=True), dict(n=20, group=4, hkv=4, dim=64)],
                         ids=["one-tile", "two-tiles", "dim64"])
def test_attention_long_ranges(c):
    """48 sequences x 4 KV heads: one CTA for each, so that its ring and buffers wrap many times."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1500, 2900, 48)]
    t = Tree(lens=lens, cap=3000, topk=14, sel_frac=0.9, seed=7, **{"hkv": 4, **c})
    s, d = t.shape, t.dev
    out, lse = torch.empty_like(d["q"]), torch.empty(s.batch, s.n_heads_q, t.n, device="cuda")
    ws = torch.empty(_lib.msa_workspace_bytes(s, 5) // 4, device="cuda")
    _lib.msa_sparse_decode_tree(s, t.seq_lens, t.table, t.n_phys, t.mask, d["q"], d["k"], d["v"], d["kd"], d["vd"],
                                d["sel"], out, lse, ws)
    _ok()
    want, want_lse, tol, tol_lse = t.attend()
    err = np.abs(out.cpu().double().numpy() - want)
    assert (err <= tol).all(), (err.max(), (err / np.maximum(tol, 1e-30)).max())
    assert (np.abs(lse.cpu().double().numpy() - want_lse) <= tol_lse).all()


def test_attention_more_blocks_than_a_list_holds():
    """Selections of 650 of 700 blocks on 160 (sequence, KV head) pairs: one CTA a pair would need a
    longer list of blocks than it has, so the selection is split.  The sequences share the pools'
    blocks.  fp64 on the GPU for some of the pairs."""
    B, h, g, d, n, nB, topk = 40, 4, 4, 128, 2, 700, 650
    cap = nB * 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(cap - 3000, cap - 2, B)]
    paths, mask = _random_tree(B, n, lens, cap, 3)
    k, v = (torch.randn(nB, h, 128, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    kd, vd = (torch.randn(B, h, n, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, n, h * g, d, generator=gen, device="cuda").bfloat16()
    table = torch.stack([torch.randperm(nB, generator=gen, device="cuda") for _ in range(B)]).to(torch.int32)
    sel = np.full((B, h, n, topk), -1, dtype=np.int32)
    for b in range(B):
        for j in range(h):
            for i, path in enumerate(paths[b]):
                cur = (lens[b] + len(path) - 1) // 128
                got = sorted(rng.permutation(cur)[:topk - 1].tolist() + [cur])
                sel[b, j, i, :len(got)] = got
    shape = _lib.make_shape(B, n, cap, h * g, h, d, d, 128, topk, 1)
    lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
    sel_t = torch.tensor(sel).cuda()
    out, lse = torch.empty_like(q), torch.empty(B, h * g, n, device="cuda")
    ws = torch.empty(_lib.msa_workspace_bytes(shape, 5) // 4, device="cuda")
    assert ws.numel() >= 2 * B * n * h * g * (d + 1)                       # two splits or more
    _lib.msa_sparse_decode_tree(shape, lens_t, table, nB, mask, q, k, v, kd, vd, sel_t, out, lse, ws)
    _ok()
    for b, j in ((0, 0), (7, 3), (19, 1), (39, 2)):
        for i, path in enumerate(paths[b]):
            chosen = [x for x in sel[b, j, i].tolist() if x >= 0]
            at = torch.tensor(chosen, device="cuda")
            keep = ((at[:, None] * 128 + torch.arange(128, device="cuda")) < lens[b]).flatten()
            phys = table[b].long()[at]
            mine = [a for a in path if (lens[b] + len(paths[b][a]) - 1) // 128 in chosen]
            kk = torch.cat([k[phys, j].flatten(0, 1)[keep], kd[b, j][mine]]).double()
            vv = torch.cat([v[phys, j].flatten(0, 1)[keep], vd[b, j][mine]]).double()
            heads = slice(j * g, (j + 1) * g)
            qq = q[b, i, heads].double()
            z = qq @ kk.T * d ** -0.5
            norm = torch.logsumexp(z, 1)
            w = torch.exp(z - norm[:, None])
            want, mag = w @ vv, w @ vv.abs()
            # as in tree_cases: scores off by e, weights and result rounded to bf16
            e = 2 * (d + 4) * 2.0 ** -24 * (qq.abs() @ kk.abs().T).amax(1) * d ** -0.5 + 2.0 ** -20
            tol = mag * (2 * e[:, None] + 2.0 ** -8 + 2.0 ** -20 + 2.0 ** -18) + 2.0 ** -8 * want.abs()
            assert ((out[b, i, heads].double() - want).abs() <= tol).all()
            # sums of 83,000 weights in fp32 chains of 64 and 1300: 2^-18 and 2^-22 of the log-sum
            assert ((lse[b, heads, i].double() - norm).abs() <= e + 2.0 ** -16 + 2.0 ** -22 * norm.abs()).all()
