"""Decode with accumulated attention weights, eviction by them, and the calls as they are used
together, against the fp64 reference.  Integers and moved values are compared exactly; weights
with the bound derived in tests/test_gpu_packed.py."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api
from block_sparse_gqa_02_gb300.configs import CONFIGS
from block_sparse_gqa_02_gb300.inputs import make_paged_decode_inputs, random_selection
from oracle import cache_ops as co
from tests.canary import guarded_like
from tests.parity import check_lse, check_out, to_np
from tests.test_gpu_packed import DT, _i32, _rows, _weight_tol

pytestmark = pytest.mark.gpu


def _ws(shape, which):
    return torch.empty(_lib.msa_workspace_bytes(shape, which) // 4 + 4, device="cuda")


MASS = {
    # B, L, Hq, Hkv, d, block, top_k, dtype
    "tc_small": (2, 300, 32, 4, 128, 128, 3, "bf16"),
    "tc_one": (1, 1, 64, 4, 128, 128, 2, "bf16"),
    "tc_long": (2, 9001, 64, 4, 128, 128, 40, "bf16"),
    "tc_group_3": (3, 1290, 24, 8, 128, 128, 5, "bf16"),
    "wide_group": (1, 700, 40, 2, 128, 128, 4, "bf16"),
    "d64": (2, 1000, 16, 2, 64, 128, 6, "bf16"),
    "block_64": (2, 1000, 16, 4, 128, 64, 6, "bf16"),
    "block_200": (1, 1000, 8, 4, 64, 200, 3, "f32"),
    "f32": (2, 1100, 16, 4, 128, 128, 5, "f32"),
    "block_1": (1, 50, 4, 1, 64, 1, 7, "f32"),
    "long_d64": (2, 20011, 32, 4, 64, 128, 64, "bf16"),
    "long_f32": (1, 9001, 16, 2, 128, 128, 40, "f32"),
    "block_1000": (2, 3001, 8, 2, 64, 1000, 3, "bf16"),
    "block_129": (1, 1500, 12, 1, 128, 129, 6, "f32"),
    "block_32": (2, 999, 10, 2, 128, 32, 20, "bf16"),
    "heads_8_of_5": (2, 5200, 10, 2, 128, 128, 40, "f32"),
    "heads_16": (4, 5200, 32, 2, 128, 128, 40, "f32"),
    "heads_16_of_12": (4, 5200, 24, 2, 64, 128, 40, "f32"),
    "heads_16_d64": (4, 5200, 32, 2, 64, 128, 40, "bf16"),
    "heads_16_of_20": (4, 5200, 40, 2, 128, 64, 60, "bf16"),
    "batch_300": (300, 130, 2, 2, 64, 128, 2, "bf16"),
    "k_past_blocks": (2, 300, 8, 4, 64, 128, 70, "f32"),
    "group_1": (2, 500, 4, 4, 128, 128, 3, "f32"),
    "group_9": (1, 400, 18, 2, 64, 128, 4, "f32"),
    "group_64": (1, 300, 64, 1, 64, 128, 3, "bf16"),
}


@pytest.mark.parametrize("name", list(MASS))
def test_decode_mass(name):
    B, L, Hq, Hkv, d, block, topk, dtype = MASS[name]
    shape = _lib.make_shape(B, 1, L, Hq, Hkv, d, 128, block, topk, 1, dtype)
    nB = shape.n_blocks
    q, k, v = (_rows(s, DT[dtype], i) for i, s in enumerate(
        ((B, 1, Hq, d), (B, Hkv, L, d), (B, Hkv, L, d))))
    sel_np = random_selection(np.full((B, Hkv, 1), nB), topk, 4)
    sel = torch.from_numpy(sel_np).cuda()
    out, lse = guarded_like(q.shape, q.dtype), guarded_like((B, Hq, 1), torch.float32)
    mass = guarded_like((B, Hkv, nB), torch.float32, fill=0.25)
    ws = guarded_like((_lib.msa_workspace_bytes(shape, 4) // 4,), torch.float32)
    _lib.msa_sparse_decode_mass(shape, None, None, 0, q, k, v, sel, out.tensor, lse.tensor,
                                mass.tensor, ws.tensor)
    _lib.msa_get_device_status()
    for x in (out, lse, mass, ws):
        x.check(name)
    o, l, m = co.decode_mass(q, k, v, sel_np, [L] * B, block)
    check_out(out.tensor, o, dtype, name)
    check_lse(lse.tensor, l, dtype, name)
    o2, l2 = torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")
    if name.startswith("tc"):      # on the tensor cores bit for bit those of the decode call
        _lib.msa_sparse_decode(shape, q, k, v, sel, o2, l2, _ws(shape, 1))
        assert torch.equal(o2, out.tensor) and torch.equal(l2, lse.tensor)
    tol = _weight_tol(to_np(q), to_np(k), d ** -0.5, d)
    added = to_np(mass.tensor) - 0.25
    assert np.all(np.abs(added - m) <= tol * m + 2.0 ** -24 * (0.25 + m)), name
    # without lse, and again: the same bits
    m2 = torch.full((B, Hkv, nB), 0.25, device="cuda")
    _lib.msa_sparse_decode_mass(shape, None, None, 0, q, k, v, sel, o2, None, m2, _ws(shape, 4))
    assert torch.equal(m2, mass.tensor) and torch.equal(o2, out.tensor)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "bf16"), (128, "f32")])
def test_decode_mass_specials(d, dtype):
    """NaN in a key that nobody selected changes nothing; in a selected one it shows in that KV
    head's rows only; keys whose scores are all -inf, and rows without a selection, add nothing."""
    B, L, Hq, Hkv = 2, 700, 8, 4
    shape = _lib.make_shape(B, 1, L, Hq, Hkv, d, 128, 128, 3, 1, dtype)
    q, k, v = (_rows(s, DT[dtype], i) for i, s in enumerate(
        ((B, 1, Hq, d), (B, Hkv, L, d), (B, Hkv, L, d))))
    sel = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda").repeat(B, Hkv, 1, 1).contiguous()
    sel[0, 1] = -1

    def run():
        out, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")
        mass = torch.zeros((B, Hkv, 6), device="cuda")
        _lib.msa_sparse_decode_mass(shape, None, None, 0, q, k, v, sel, out, lse, mass, _ws(shape, 4))
        return out, lse, mass

    want = run()
    assert not want[0][0, 0, 2:4].any() and torch.isneginf(want[1][0, 2:4]).all()
    assert not want[2][0, 1].any() and not want[2][:, :, [1, 3, 4]].any()
    k[0, 0, 128], v[0, 0, 511] = float("nan"), float("inf")    # blocks 1 and 3
    assert all(torch.equal(x, y) for x, y in zip(run(), want))
    k[1, 3, 300, 0] = float("nan")                             # block 2, selected
    out, lse, mass = run()
    assert torch.isnan(out[1, 0, 6:]).all() and not torch.isnan(out[1, 0, :6]).any()
    assert torch.equal(out[0], want[0][0]) and torch.equal(mass[1, :3], want[2][1, :3])
    # one head pair's q against keys that leave only -inf
    q[1, 0, :2] = 1.0
    k[1, 0] = 0.0
    k[1, 0, :, 0] = float("-inf")
    out, lse, mass = run()
    assert not out[1, 0, :2].any() and torch.isneginf(lse[1, :2]).all() and not mass[1, 0].any()


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "bf16"), (128, "f32")])
def test_decode_mass_graphs_and_streams(d, dtype):
    """Two captured steps, each with a workspace of its own, replayed at once on two streams, and
    two that share one replayed in turn: the bits of the eager calls."""
    B, L, Hq, Hkv = 2, 3000, 16, 4
    shape = _lib.make_shape(B, 1, L, Hq, Hkv, d, 128, 128, 6, 1, dtype)
    nB = shape.n_blocks
    steps = []
    for i in range(2):
        q, k, v = (_rows(s, DT[dtype], 10 * i + j) for j, s in enumerate(
            ((B, 1, Hq, d), (B, Hkv, L, d), (B, Hkv, L, d))))
        sel = torch.from_numpy(random_selection(np.full((B, Hkv, 1), nB), 6, i)).cuda()
        steps.append((q, k, v, sel, torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda"),
                      torch.zeros((B, Hkv, nB), device="cuda")))

    def call(step, ws):
        q, k, v, sel, out, lse, mass = step
        _lib.msa_sparse_decode_mass(shape, None, None, 0, q, k, v, sel, out, lse, mass, ws)

    own = [_ws(shape, 4), _ws(shape, 4)]
    for step in steps:
        call(step, own[0])
    torch.cuda.synchronize()
    want = [[x.clone() for x in step[4:]] for step in steps]

    def graphs(spaces):
        out = []
        for step, ws in zip(steps, spaces):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call(step, ws)
            out.append(g)
        return out

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for captured, at_once in ((graphs(own), True), (graphs([own[0]] * 2), False)):
        for step in steps:
            for x in step[4:]:
                x.zero_()
        torch.cuda.synchronize()
        for g, stream in zip(captured, streams):
            with torch.cuda.stream(stream if at_once else streams[0]):
                g.replay()
        torch.cuda.synchronize()
        for step, w in zip(steps, want):
            assert all(torch.equal(x, y) for x, y in zip(step[4:], w))


@pytest.mark.parametrize("lens", [[1, 127, 129, 4097, 0], [3000, 2999, 64]])
def test_decode_mass_paged(lens):
    cfg = CONFIGS["d1m"].with_(seq=5000, top_k=8, n_plants=0)
    x = make_paged_decode_inputs(cfg, lens, device="cuda", seed=3)
    B = len(lens)
    shape = _lib.shape_from_config(cfg, batch=B)
    sel_np = random_selection(np.array([[[max(1, -(-n // 128))]] * 4 for n in lens]), 8, 2)
    sel = torch.from_numpy(sel_np).cuda()
    out, lse = torch.empty_like(x["q"]), torch.empty((B, 64, 1), device="cuda")
    mass = torch.zeros((B, 4, shape.n_blocks), device="cuda")
    _lib.msa_sparse_decode_mass(shape, x["seq_lens"], x["block_table"], x["n_phys"], x["q"],
                                x["k_pool"], x["v_pool"], sel, out, lse, mass, _ws(shape, 4))
    _lib.msa_get_device_status()
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    _lib.msa_sparse_decode_paged(shape, x["seq_lens"], x["block_table"], x["n_phys"], x["q"],
                                 x["k_pool"], x["v_pool"], sel, o2, l2, _ws(shape, 1))
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    caches = []
    for n in ("k_pool", "v_pool"):
        rows = []
        for b, L in enumerate(lens):
            phys = x["block_table"][b, :-(-L // 128)].long()
            rows.append(to_np(x[n][phys].transpose(0, 1).reshape(4, -1, 128)))
        caches.append(rows)
    _, _, m = co.decode_mass(x["q"], *caches, sel_np, lens)
    big = np.concatenate([c.reshape(-1, 128) for c in caches[0]])
    tol = _weight_tol(to_np(x["q"]), big, 128 ** -0.5, 128)
    got = to_np(mass)
    assert np.all(np.abs(got[:, :, :m.shape[2]] - m) <= (tol + 2.0 ** -24) * m)
    assert not got[:, :, m.shape[2]:].any()


EVICT = {
    # B, cap, Hkv, lens (None: all full), keep, first, recent, block
    "tiny": (1, 100, 1, None, 1, 0, 1, 128),
    "ragged": (6, 5000, 4, [5000, 0, 1, 640, 641, 4999], 5, 1, 2, 128),
    "all_fit": (2, 1000, 2, None, 9, 2, 2, 128),
    "only_forced": (3, 3000, 2, [3000, 100, 1700], 4, 1, 3, 128),
    "no_first": (2, 130000, 8, [130000, 77777], 200, 0, 1, 128),
    "wide": (3, 1 << 20, 4, [1 << 20, 5, 600001], 2048, 4, 16, 128),
    "max_blocks": (1, 32768, 2, None, 20000, 7, 9, 1),
    "keep_past_blocks": (2, 700, 2, [700, 300], 50, 0, 1, 128),
    "one_goes": (1, 1281, 3, None, 10, 1, 1, 128),
    # 3, 5 and 7 CTAs a sequence; rows of lengths that are no multiple of anything
    "three_parts": (2, 2501, 5, [2501, 2048], 777, 3, 5, 1),
    "five_parts": (1, 4999, 1, None, 2500, 0, 1, 1),
    "seven_parts": (2, 7001 * 128, 3, None, 6999, 1, 1, 128),
}


def _weights(B, Hkv, nB, kind, seed):
    rng = np.random.default_rng(seed)
    m = np.exp(2 * rng.standard_normal((B, Hkv, nB))).astype(np.float32)
    if kind == "ties":
        m = rng.integers(0, 3, m.shape).astype(np.float32)
    elif kind == "special":
        m[:, 0, ::3] = np.nan
        m[:, 0, 1::5] = np.inf
        m[:, -1, 2::7] = -1.0
        m[:, :, 3::11] = -0.0
    elif kind == "equal":
        m[:] = 0.5
    return m


@pytest.mark.parametrize("kind", ["plain", "ties", "special", "equal"])
@pytest.mark.parametrize("name", list(EVICT))
def test_evict(name, kind):
    B, cap, Hkv, lens, keep, first, recent, block = EVICT[name]
    shape = _lib.make_shape(B, 1, cap, Hkv, Hkv, 128, 128, block, 1, 1)
    nB = shape.n_blocks
    m = _weights(B, Hkv, nB, kind, 1)
    table = np.random.default_rng(2).permutation(B * nB).astype(np.int32).reshape(B, nB)
    lens_t = None if lens is None else _i32(lens)
    mass, tab = torch.from_numpy(m).cuda(), torch.from_numpy(table).cuda()
    outs = [guarded_like(s, t, fill=99) for s, t in (((B, keep), torch.int32), ((B,), torch.int32),
                                                     (m.shape, torch.float32), (table.shape, torch.int32))]
    kept, new_lens, mass_out, tab_out = (x.tensor for x in outs)
    _lib.msa_cache_evict(shape, keep, first, recent, lens_t, mass, tab, kept, new_lens, mass_out, tab_out)
    _lib.msa_get_device_status()
    for x in outs:
        x.check(name)
    want = co.evict(m, lens or [cap] * B, keep, first, recent, block, table)
    assert np.array_equal(to_np(kept), want[0]), name
    assert np.array_equal(to_np(new_lens), want[1])
    assert np.array_equal(mass_out.cpu().numpy(), want[2], equal_nan=True)
    assert np.array_equal(to_np(tab_out), want[3])
    assert torch.equal(mass.cpu(), torch.from_numpy(m)) or kind == "special"
    # in place, without a table and with one
    lens2 = _i32(lens or [cap] * B)
    _lib.msa_cache_evict(shape, keep, first, recent, lens2, mass, tab, kept, lens2, mass, tab)
    assert np.array_equal(to_np(lens2), want[1]) and np.array_equal(to_np(tab), want[3])
    assert np.array_equal(mass.cpu().numpy(), want[2], equal_nan=True)
    k2 = torch.full_like(kept, 77)
    mass = torch.from_numpy(m).cuda()
    _lib.msa_cache_evict(shape, keep, first, recent, lens_t, mass, None, k2, new_lens, mass_out)
    assert np.array_equal(to_np(k2), want[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gather(dtype):
    """Kept blocks of caches of odd lengths; padding (-1), the cut last block, rows that nothing
    covers, entries past the source."""
    B, Hkv, L, rows = 2, 3, 700, 450
    k, ik = _rows((B, Hkv, L, 64), DT[dtype], 1), _rows((B, L, 128), DT[dtype], 2)
    kept = _i32([[0, 2, 4, 5], [1, 5, 77, -1]])
    dst = [guarded_like((B, Hkv, rows, 64), DT[dtype], fill=5.0),
           guarded_like((B, rows, 128), DT[dtype], fill=5.0)]
    _lib.msa_cache_gather(B, _lib.make_gather_tensors([(k, dst[0].tensor), (ik, dst[1].tensor)]), kept)
    _lib.msa_get_device_status()
    for src, got in ((to_np(k), dst[0]), (to_np(ik)[:, None], dst[1])):
        got.check("gather")
        res = to_np(got.tensor).reshape(src.shape[0], src.shape[1], rows, src.shape[-1])
        for b in range(B):
            want = np.full((src.shape[1], rows, src.shape[-1]), 5.0)
            for i, blk in enumerate(to_np(kept)[b]):
                if 0 <= blk <= 5:
                    part = src[b][:, blk * 128:(blk + 1) * 128]
                    n = min(part.shape[1], rows - i * 128)
                    want[:, i * 128:i * 128 + n] = part[:, :n]
            assert np.array_equal(res[b], want), b


def test_gather_of_the_4_bit_cache():
    """A table-less 4-bit cache cut by whole blocks: the decode over the kept blocks' new places is
    the decode over their old ones, bit for bit."""
    B, Hkv, d, cap, keep = 2, 4, 128, 1100, 5
    shape = _lib.make_shape(B, 1, cap, 16, Hkv, d, 128, 128, keep, 1)
    nB = shape.n_blocks
    cache = api.alloc_packed_cache(B * nB, Hkv, d)
    k, v = _rows((B, Hkv, cap, d), DT["bf16"], 1), _rows((B, Hkv, cap, d), DT["bf16"], 2)
    _lib.msa_cache_pack(shape, cap, None, None, None, B * nB, k, v, cache)
    kept = _i32([[0, 2, 3, 7, 8], [1, 4, 5, 6, 8]])
    small = api.alloc_packed_cache(B * keep, Hkv, d)
    pair = (cache.view(B, 1, nB * 128, -1), small.view(B, 1, keep * 128, -1))
    _lib.msa_cache_gather(B, _lib.make_gather_tensors([pair]), kept)
    q = _rows((B, 1, 16, d), DT["bf16"], 3)
    outs = []
    for c, n, sel in ((cache, cap, kept), (small, cap - (nB - keep) * 128,
                                           torch.arange(keep, device="cuda", dtype=torch.int32).expand(B, keep))):
        s = _lib.make_shape(B, 1, n, 16, Hkv, d, 128, 128, keep, 1)
        out = torch.empty_like(q)
        _lib.msa_sparse_decode_packed(s, None, None, c.shape[0], q, c,
                                      sel[:, None, None].expand(B, Hkv, 1, keep).contiguous(), out)
        outs.append(out)
    assert torch.equal(*outs)


def test_gather_past_32_bit_offsets():
    """Sources and destinations of more than 4 GiB a tensor."""
    rows, d = 9_000_000, 256
    src = torch.zeros((1, 2, rows, d), dtype=torch.bfloat16, device="cuda")
    dst = torch.zeros((1, 2, rows - 128, d), dtype=torch.bfloat16, device="cuda")
    n = -(-rows // 128)
    src[:, :, -200:] = _rows((1, 2, 200, d), torch.bfloat16, 1)
    kept = torch.arange(1, n, dtype=torch.int32, device="cuda").view(1, n - 1)
    _lib.msa_cache_gather(1, _lib.make_gather_tensors([(src, dst)]), kept)
    assert torch.equal(dst[:, :, -200:], src[:, :, -200:]) and not dst[:, :, :-200].any()


def test_evict_graph_and_stream():
    """Captured once and replayed as the cache fills again."""
    B, cap = 2, 4096
    shape = _lib.make_shape(B, 1, cap, 4, 4, 128, 128, 128, 1, 1)
    m = _weights(B, 4, 32, "plain", 5)
    mass, lens = torch.from_numpy(m).cuda(), _i32([4000, 900])
    table = torch.arange(B * 32, dtype=torch.int32, device="cuda").view(B, 32).contiguous()
    t0 = table.cpu().numpy()
    kept = torch.zeros((B, 10), dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.msa_cache_evict(shape, 10, 1, 2, lens, mass, table, kept, lens, mass, table)
    graph.replay()
    torch.cuda.synchronize()
    want = co.evict(m, [4000, 900], 10, 1, 2, table=t0)
    assert np.array_equal(to_np(kept), want[0]) and np.array_equal(to_np(table), want[3])
    lens += 1000                                                     # the caches grow again
    mass += 1.0
    graph.replay()
    torch.cuda.synchronize()
    want2 = co.evict(want[2] + np.float32(1), want[1] + 1000, 10, 1, 2, table=want[3])
    assert np.array_equal(to_np(kept), want2[0]) and np.array_equal(to_np(table), want2[3])
    assert np.array_equal(to_np(lens), want2[1])


# ------------------------------------------------------------------- used together

def test_decode_loop_with_packed_cache_rope_and_eviction():
    """A serving loop over a paged 4-bit cache: every step rotates and packs the new token, scores
    and selects blocks, attends and adds up the blocks' weights; the sequences are cut now and
    then.  Each step's output against the fp64 attention over the values that a plain list of
    tokens, cut the same way, holds."""
    B, Hq, Hkv, d, cap, topk, keep = 2, 16, 4, 128, 1024, 3, 4
    freqs, scale = api.rope_freqs(128, device="cuda")
    rope = api.Rope(freqs, scale=scale)
    P = B * 8
    table = torch.randperm(P, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    table = table.to(torch.int32).view(B, 8).contiguous()
    cache = api.alloc_packed_cache(P, Hkv, d)
    idx_pool = torch.zeros((P, 128, 128), dtype=torch.bfloat16, device="cuda")
    mass = torch.zeros((B, Hkv, 8), device="cuda")
    lens0 = [890, 640]
    lens = _i32(lens0)
    # prompts
    shape = _lib.make_shape(B, 1, cap, Hq, Hkv, d, 128, 128, topk, 1)
    n0 = max(lens0)
    k, v = _rows((B, Hkv, n0, d), torch.bfloat16, 1), _rows((B, Hkv, n0, d), torch.bfloat16, 2)
    ik = _rows((B, n0, 128), torch.bfloat16, 3)
    k, ik = api.rope([(k, freqs, True), (ik, freqs, False)], scale=scale)
    _lib.msa_cache_pack(shape, n0, torch.zeros_like(lens), lens, table, P, k, v, cache)
    for b in range(B):
        for j in range(-(-lens0[b] // 128)):
            part = ik[b, 128 * j:min(lens0[b], 128 * (j + 1))]
            idx_pool[table[b, j].item(), :part.shape[0]] = part
    kv = [list(np.moveaxis(co.pack_values(to_np(k[b, :, :lens0[b]]))[0], 1, 0)) for b in range(B)]
    vv = [list(np.moveaxis(co.pack_values(to_np(v[b, :, :lens0[b]]))[0], 1, 0)) for b in range(B)]
    total = np.zeros((B, Hkv, 8))
    for step in range(6):
        lens += 1
        n = [int(x) for x in lens]
        q = _rows((B, 1, Hq, d), torch.bfloat16, 10 + step)
        k1, v1 = (_rows((B, Hkv, 1, d), torch.bfloat16, 20 + 2 * step + i) for i in range(2))
        iq, ik1 = _rows((B, 1, 4, 128), torch.bfloat16, 40 + step), _rows((B, 1, 128), torch.bfloat16, 50 + step)
        pos = lens.view(B, 1)
        desc = _lib.make_rope(B, 1, pos_offset=-1, scale=scale)
        rot = torch.empty_like(ik1)
        _lib.msa_rope(desc, _lib.make_rope_tensors([(ik1, rot, freqs, False)]), pos)
        for b in range(B):
            idx_pool[table[b, (n[b] - 1) // 128].item(), (n[b] - 1) % 128] = rot[b, 0]
        got = api.decode_packed(q, k1, v1, cache, iq, idx_pool, lens, table, cap, topk, rope=rope,
                                mass=mass)
        _lib.msa_get_device_status()
        qr, kr = api.rope([(q, freqs, False), (k1, freqs, True)], pos, -1, scale)
        for b in range(B):
            kv[b].append(co.pack_values(to_np(kr))[0][b, :, 0])
            vv[b].append(co.pack_values(to_np(v1))[0][b, :, 0])
        sel = to_np(got["sel"])
        o, l, m = co.decode_mass(qr, [np.stack(x, 1) for x in kv], [np.stack(x, 1) for x in vv], sel, n)
        check_out(got["out"], o, "bf16", f"step {step}")
        check_lse(got["lse"], l, "bf16", f"step {step}")
        for b in range(B):
            assert all((n[b] - 1) // 128 in row for row in sel[b, :, 0])
        total[:, :, :m.shape[2]] += m
        assert np.allclose(to_np(mass), total, rtol=2e-3, atol=1e-6)
        if step in (2, 4):
            before = mass.cpu().numpy()
            kept = api.evict_paged(lens, mass, table, cap, keep)
            want = co.evict(before, n, keep, 1, 2)
            assert np.array_equal(to_np(kept), want[0]) and np.array_equal(to_np(lens), want[1])
            for b in range(B):
                stay = [int(x) for x in want[0][b] if x >= 0]
                rows = [j for x in stay for j in range(128 * x, min(n[b], 128 * (x + 1)))]
                kv[b], vv[b] = [kv[b][j] for j in rows], [vv[b][j] for j in rows]
                total[b] = np.pad(total[b][:, stay], ((0, 0), (0, 8 - len(stay))))


def test_contiguous_decode_and_eviction():
    """api.decode with mass, then api.evict: the next step over the shorter caches is the decode
    over the kept blocks of the long ones."""
    B, Hq, Hkv, d, L = 2, 16, 4, 128, 1500
    q, k, v = (_rows(s, torch.bfloat16, i) for i, s in enumerate(
        ((B, 1, Hq, d), (B, Hkv, L, d), (B, Hkv, L, d))))
    iq, ik = _rows((B, 1, 4, 128), torch.bfloat16, 5), _rows((B, L, 128), torch.bfloat16, 6)
    mass = torch.zeros((B, Hkv, 12), device="cuda")
    first = api.decode(q, k, v, iq, ik, top_k=5, mass=mass)
    plain = api.decode(q, k, v, iq, ik, top_k=5)
    for n in ("scores", "sel", "out", "lse"):
        assert torch.equal(first[n], plain[n])
    cut = api.evict(k, v, ik, mass, keep=6, n_first=1, n_recent=2)
    kept = to_np(cut["kept"])
    want = co.evict(mass.cpu().numpy(), [L] * B, 6, 1, 2)
    assert np.array_equal(kept, want[0]) and cut["k"].shape == (B, Hkv, L - 6 * 128, d)
    assert np.array_equal(cut["mass"].cpu().numpy(), want[2][:, :, :6])
    step = api.decode(q, cut["k"], cut["v"], iq, cut["idx_k"], top_k=6)
    # all six kept blocks, in the long cache's numbering
    sel = torch.from_numpy(np.repeat(kept[:, None, None], Hkv, 1).astype(np.int32)).cuda().contiguous()
    shape = _lib.make_shape(B, 1, L, Hq, Hkv, d, 128, 128, 6, 1)
    out, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")
    _lib.msa_sparse_decode(shape, q, k, v, sel, out, lse, _ws(shape, 1))
    check_out(step["out"], to_np(out), "bf16")
    check_lse(step["lse"], to_np(lse), "bf16")
    # kept blocks keep their index scores
    gathered = np.take_along_axis(to_np(plain["scores"])[:, :, 0], np.repeat(kept[:, None], Hkv, 1), 2)
    assert np.array_equal(to_np(step["scores"])[:, :, 0], gathered)
