"""The 4-bit KV cache: packing, unpacking and decode attention over it, against the fp64
reference.

Packed values are compared exactly (the definition fixes every operation).  Attention outputs and
log-sum-exps use the package's attention tolerances (tests/parity.py) on the values that the cache
holds.  Weights: exp(z - lse) is off by the errors of z and lse; z is an fp32 sum of d products
scaled, at most (d + 8) 2^-24 of sum |q k| scale (in log2 units and back: 2 roundings more), lse
no more than the largest such error, exp2 2^-21: relative, on every weight, so on their sums."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api
from block_sparse_gqa_02_gb300.inputs import random_selection
from oracle import cache_ops as co
from tests.canary import guarded_like
from tests.parity import check_lse, check_out, to_np

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _shape(B, cap, Hq, Hkv, d, k=4, dtype="bf16", **kw):
    return _lib.make_shape(B, 1, cap, Hq, Hkv, d, 128, 128, k, 1, dtype, **kw)


def _rows(shape, dt, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    off = torch.randn(shape[-1], generator=g, device="cuda")
    return (torch.randn(shape, generator=g, device="cuda") + off).to(dt)


def _table(B, nB, seed, spare=3):
    p = np.random.default_rng(seed).permutation(B * nB + spare)[:B * nB]
    return torch.from_numpy(p.astype(np.int32).reshape(B, nB)).cuda(), B * nB + spare


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("paged", [False, True])
def test_pack_and_unpack(dtype, d, paged):
    """Ragged appends at odd places: stored tokens' values exactly, every other byte as it was,
    unstored rows of the outputs as they were."""
    B, Hkv, n, cap = 4, 3, 200, 700
    starts, lens = [0, 130, 255, 699], [200, 200, 456, 700]      # 70 and 1 of 200 stored, too
    shape = _shape(B, cap, Hkv, Hkv, d, dtype=dtype)
    table, P = _table(B, 6, 1) if paged else (None, B * 6)
    k, v = _rows((B, Hkv, n, d), DT[dtype], 2), _rows((B, Hkv, n, d), DT[dtype], 3)
    cache = guarded_like((P, Hkv, 160 * d), torch.uint8, fill=0x5C)
    _lib.msa_cache_pack(shape, n, _i32(starts), _i32(lens), table, P, k, v, cache.tensor)
    ko, vo = guarded_like(k.shape, k.dtype, fill=7.0), guarded_like(v.shape, v.dtype, fill=7.0)
    _lib.msa_cache_unpack(shape, n, _i32(starts), _i32(lens), table, P, cache.tensor, ko.tensor,
                          vo.tensor)
    _lib.msa_get_device_status()
    for x in (cache, ko, vo):
        x.check("packed cache")
    raw = cache.tensor.cpu().numpy()
    phys = table.cpu().numpy() if paged else np.arange(B * 6).reshape(B, 6)
    touched = np.zeros(raw.shape, dtype=bool)
    for src, got, is_v in ((k, ko, False), (v, vo, True)):
        want, step, mid = co.pack_values(to_np(src))
        held = torch.from_numpy(want).to(DT[dtype]).double().numpy()   # rounded once
        byte, _ = co.record_offsets(d, is_v)
        for b in range(B):
            stored = [i for i in range(n) if starts[b] + i < lens[b]]
            assert np.array_equal(to_np(got.tensor)[b][:, stored], held[b][:, stored])
            rest = [i for i in range(n) if i not in set(stored)]
            assert np.all(to_np(got.tensor)[b][:, rest] == 7.0)
            for i in stored:
                p, row = starts[b] + i, (starts[b] + i) % 128
                at = touched[phys[b, p // 128]][:, 80 * d * is_v:]
                at[:, byte[row]] = True
                for g in range(d // 32):
                    for base in (64 * d, 72 * d):
                        at[:, base + (g * 128 + row) * 2:base + (g * 128 + row) * 2 + 2] = True
            i = stored[-1]
            p = starts[b] + i
            rec = raw[phys[b, p // 128], 1, 80 * d * is_v:80 * d * (1 + is_v)]
            assert np.array_equal(co.record_values(rec, d, is_v)[p % 128], want[b, 1, i])
    assert np.all(raw[~touched] == 0x5C)


def test_pack_default_positions_and_single_tokens():
    """Without starts the tokens are the last of each sequence; appending them one by one gives
    the bytes of one call."""
    B, Hkv, d, n = 3, 4, 128, 9
    lens = [9, 131, 300]
    shape = _shape(B, 384, Hkv, Hkv, d)
    k, v = _rows((B, Hkv, n, d), DT["bf16"], 4), _rows((B, Hkv, n, d), DT["bf16"], 5)
    one = torch.zeros((9, Hkv, 160 * d), dtype=torch.uint8, device="cuda")
    each = torch.zeros_like(one)
    _lib.msa_cache_pack(shape, n, None, _i32(lens), None, 9, k, v, one)
    for i in range(n):
        _lib.msa_cache_pack(shape, 1, None, _i32([x - n + 1 + i for x in lens]), None, 9,
                            k[:, :, i:i + 1].contiguous(), v[:, :, i:i + 1].contiguous(), each)
    assert torch.equal(one, each) and one.any()
    # whole capacity, no lengths; and lengths shorter than the call: the first tokens fall out
    full = _rows((1, Hkv, 384, d), DT["bf16"], 6)
    s1 = _shape(1, 384, Hkv, Hkv, d)
    c = torch.zeros((3, Hkv, 160 * d), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(full)
    _lib.msa_cache_pack(s1, 384, None, None, None, 3, full, full, c)
    _lib.msa_cache_unpack(s1, 384, None, None, None, 3, c, out, torch.empty_like(out))
    assert np.array_equal(to_np(out), to_np(torch.from_numpy(co.pack_values(to_np(full))[0]).bfloat16()))
    c2 = torch.zeros_like(c)
    _lib.msa_cache_pack(s1, 384, None, _i32([10]), None, 3, full, full, c2)
    _lib.msa_cache_unpack(s1, 10, None, _i32([10]), None, 3, c2, out[:, :, :10].contiguous(),
                          got := torch.empty((1, Hkv, 10, d), dtype=torch.bfloat16, device="cuda"))
    assert np.array_equal(to_np(got), to_np(torch.from_numpy(
        co.pack_values(to_np(full[:, :, -10:]))[0]).bfloat16()))


def test_pack_special_values():
    x = torch.randn((1, 1, 4, 64), device="cuda")
    x[0, 0, 1, 3] = float("nan")
    x[0, 0, 2, 40] = float("inf")
    x[0, 0, 3] = 2.5
    c = torch.zeros((1, 1, 160 * 64), dtype=torch.uint8, device="cuda")
    ko, vo = torch.zeros_like(x), torch.zeros_like(x)
    s = _shape(1, 4, 1, 1, 64, dtype="f32")
    _lib.msa_cache_pack(s, 4, None, None, None, 1, x, x, c)
    _lib.msa_cache_unpack(s, 4, None, None, None, 1, c, ko, vo)
    want = co.pack_values(to_np(x))[0].astype(np.float32).astype(np.float64)
    assert np.array_equal(to_np(ko), want, equal_nan=True)
    assert np.array_equal(to_np(vo), want, equal_nan=True)
    assert torch.isnan(ko[0, 0, 1, :32]).all() and not torch.isnan(ko[0, 0, 1, 32:]).any()
    assert torch.isnan(ko[0, 0, 2, 32:]).all() and torch.all(ko[0, 0, 3] == 2.5)


def _filled(B, cap, Hkv, d, lens, dtype, paged, seed):
    """A cache of random tokens whose bytes past each sequence's end are 0xFF (NaN steps)."""
    nB = -(-cap // 128)
    table, P = _table(B, nB, seed) if paged else (None, B * nB)
    cache = torch.full((P, Hkv, 160 * d), 0xFF, dtype=torch.uint8, device="cuda")
    k, v = _rows((B, Hkv, cap, d), DT[dtype], seed), _rows((B, Hkv, cap, d), DT[dtype], seed + 1)
    shape = _shape(B, cap, Hkv, Hkv, d, dtype=dtype)
    _lib.msa_cache_pack(shape, cap, torch.zeros(B, dtype=torch.int32, device="cuda"), _i32(lens),
                        table, P, k, v, cache)
    return cache, table, P, co.pack_values(to_np(k))[0], co.pack_values(to_np(v))[0]


def _weight_tol(q, kv, scale, d):
    big = max(float((np.abs(q).reshape(-1, d).max(0) * np.abs(kv).reshape(-1, d).max(0)).sum()), 1.0)
    return 2 * ((d + 8) * 2.0 ** -24 * big * scale) + 2.0 ** -20


DECODE = {
    # B, cap, Hq, Hkv, d, lens, top_k, dtype, paged
    "one_token": (1, 1, 4, 4, 128, [1], 1, "bf16", False),
    "short": (2, 300, 32, 4, 128, [300, 129], 3, "bf16", False),
    "ragged_paged": (5, 2000, 64, 4, 128, [2000, 1, 0, 1153, 640], 6, "bf16", True),
    "d64": (3, 1500, 16, 2, 64, [1500, 127, 128], 5, "bf16", True),
    "one_head": (2, 900, 3, 3, 64, [900, 513], 8, "bf16", False),
    "wide_group": (1, 1000, 40, 1, 128, [1000], 7, "bf16", False),
    "group_5": (2, 1000, 40, 8, 128, [1000, 999], 4, "bf16", True),
    "group_64": (1, 700, 64, 1, 64, [700], 4, "bf16", False),
    "many_splits": (1, 9000, 16, 1, 128, [9000], 64, "bf16", True),
    "k_past_blocks": (2, 500, 8, 4, 128, [500, 40], 100, "bf16", False),
    "f32": (3, 1500, 16, 4, 128, [1500, 1, 700], 6, "f32", True),
    "f32_d64_wide": (1, 800, 34, 2, 64, [800], 5, "f32", False),
}


@pytest.mark.parametrize("name", list(DECODE))
def test_packed_decode(name):
    B, cap, Hq, Hkv, d, lens, topk, dtype, paged = DECODE[name]
    cache, table, P, kv, vv = _filled(B, cap, Hkv, d, lens, dtype, paged, seed=len(name))
    shape = _shape(B, cap, Hq, Hkv, d, topk, dtype)
    nB = shape.n_blocks
    blocks = np.array([[[max(1, -(-x // 128))] * Hkv] for x in lens]).reshape(B, Hkv, 1)
    sel_np = random_selection(blocks, topk, 3)
    sel = torch.from_numpy(sel_np).cuda()
    q = _rows((B, 1, Hq, d), DT[dtype], 9)
    out, lse = guarded_like(q.shape, q.dtype), guarded_like((B, Hq, 1), torch.float32)
    mass = guarded_like((B, Hkv, nB), torch.float32, fill=0.5)
    _lib.msa_sparse_decode_packed(shape, _i32(lens), table, P, q, cache, sel, out.tensor, lse.tensor,
                                  mass.tensor)
    _lib.msa_get_device_status()
    for x in (out, lse, mass):
        x.check(name)
    o, l, m = co.decode_mass(q, list(kv), list(vv), sel_np, lens)
    check_out(out.tensor, o, dtype, name)
    check_lse(lse.tensor, l, dtype, name)
    added = to_np(mass.tensor)[:, :, :m.shape[2]] - 0.5
    tol = _weight_tol(to_np(q), kv, d ** -0.5, d)
    # the addition to 0.5 rounds once more
    assert np.all(np.abs(added - m) <= tol * m + 2.0 ** -24 * (0.5 + m)), name
    # without mass and lse: the same output, and again: the same bits
    out2 = torch.empty_like(q)
    _lib.msa_sparse_decode_packed(shape, _i32(lens), table, P, q, cache, sel, out2)
    assert torch.equal(out2, out.tensor)
    m2 = torch.full((B, Hkv, nB), 0.5, device="cuda")
    _lib.msa_sparse_decode_packed(shape, _i32(lens), table, P, q, cache, sel, out2, None, m2)
    assert torch.equal(m2, mass.tensor)
    # a user's scale
    s2 = _shape(B, cap, Hq, Hkv, d, topk, dtype, sm_scale=0.03)
    _lib.msa_sparse_decode_packed(s2, _i32(lens), table, P, q, cache, sel, out2, l2 := torch.empty(
        (B, Hq, 1), device="cuda"))
    o, l, _ = co.decode_mass(q, list(kv), list(vv), sel_np, lens, sm_scale=0.03)
    check_out(out2, o, dtype, name)
    check_lse(l2, l, dtype, name)


def test_packed_decode_thousands_of_entries():
    """More entries than a split lists at once, the blocks anywhere among them; the same with
    weights' limit."""
    B, cap, Hkv, d = 1, 9 * 128, 2, 128
    for dtype, topk in (("bf16", 8300), ("f32", 17000), ("bf16", 1024)):
        cache, table, P, kv, vv = _filled(B, cap, Hkv, d, [cap], dtype, True, 7)
        shape = _shape(B, cap, 8, Hkv, d, topk, dtype)
        rng = np.random.default_rng(topk)
        sel_np = np.full((B, Hkv, 1, topk), -1, dtype=np.int32)
        for g in range(Hkv):
            sel_np[0, g, 0, np.sort(rng.choice(topk, 8, replace=False))] = rng.permutation(9)[:8]
        sel, q = torch.from_numpy(sel_np).cuda(), _rows((B, 1, 8, d), DT[dtype], 1)
        out, lse = torch.empty_like(q), torch.empty((B, 8, 1), device="cuda")
        mass = torch.zeros((B, Hkv, 9), device="cuda") if topk <= 1024 else None
        _lib.msa_sparse_decode_packed(shape, None, table, P, q, cache, sel, out, lse, mass)
        _lib.msa_get_device_status()
        o, l, m = co.decode_mass(q, list(kv), list(vv), sel_np, [cap])
        check_out(out, o, dtype)
        check_lse(lse, l, dtype)
        if mass is not None:
            tol = _weight_tol(to_np(q), kv, d ** -0.5, d) + 2.0 ** -24
            assert np.all(np.abs(to_np(mass) - m) <= tol * m)


def test_packed_decode_bad_entries():
    """Selection entries that are no block of the sequence and table entries that are no physical
    block are skipped: the output of the row without them."""
    B, cap, Hkv, d, lens = 2, 1000, 4, 128, [1000, 300]
    cache, table, P, _, _ = _filled(B, cap, Hkv, d, lens, "bf16", True, 5)
    shape = _shape(B, cap, 32, Hkv, d, 5)
    q = _rows((B, 1, 32, d), DT["bf16"], 1)
    good = _i32([[[[0, 3, 7, -1, -1]]] * 4, [[[0, 2, -1, -1, -1]]] * 4]).reshape(B, 4, 1, 5).contiguous()
    bad = _i32([[[[0, 3, 7, 8, 1 << 30]]] * 4, [[[0, 2, 3, 7, -5]]] * 4]).reshape(B, 4, 1, 5).contiguous()
    def go(sel, tab):
        out = torch.empty_like(q)
        lse, mass = torch.empty((B, 32, 1), device="cuda"), torch.zeros((B, Hkv, 8), device="cuda")
        _lib.msa_sparse_decode_packed(shape, _i32(lens), tab, P, q, cache, sel, out, lse, mass)
        torch.cuda.synchronize()
        return out, lse, mass
    want = go(good, table)
    for x, y in zip(go(bad, table), want):
        assert torch.equal(x, y)
    broken = table.clone()
    broken[0, 3], broken[1, 2] = P, -2
    less = _i32([[[[0, -1, 7, -1, -1]]] * 4, [[[0, -1, -1, -1, -1]]] * 4]).reshape(B, 4, 1, 5).contiguous()
    for x, y in zip(go(good, broken), go(less, table)):
        assert torch.equal(x, y)
    # packing into such an entry writes nothing, reading leaves the rows
    before = cache.clone()
    k = _rows((B, Hkv, 1, d), DT["bf16"], 2)
    gone = torch.full_like(table, P)
    _lib.msa_cache_pack(shape, 1, None, _i32(lens), gone, P, k, k, cache)
    ko = torch.full_like(k, 3.0)
    _lib.msa_cache_unpack(shape, 1, None, _i32(lens), gone, P, cache, ko, torch.empty_like(k))
    assert torch.equal(before, cache) and torch.all(ko == 3.0)
    # lengths outside [0, capacity] count as the nearest
    a, b = torch.empty_like(q), torch.empty_like(q)
    _lib.msa_sparse_decode_packed(shape, _i32([5000, -3]), table, P, q, cache, good, a)
    _lib.msa_sparse_decode_packed(shape, _i32([1000, 0]), table, P, q, cache, good, b)
    assert torch.equal(a, b) and not a[1].any()


def test_packed_decode_large_logits_and_outlier_scales():
    """Logits of hundreds (one key takes all the weight) and V steps that differ by 2^60 between
    groups: no overflow, no loss."""
    B, cap, Hkv, d = 1, 600, 2, 128
    shape = _shape(B, cap, 8, Hkv, d, 5)
    k, v = _rows((B, Hkv, cap, d), DT["bf16"], 1) * 40, _rows((B, Hkv, cap, d), DT["bf16"], 2)
    v[..., 32:64] *= 2.0 ** 40
    v[..., 64:96] *= 2.0 ** -20
    cache = torch.zeros((5, Hkv, 160 * d), dtype=torch.uint8, device="cuda")
    _lib.msa_cache_pack(shape, cap, None, None, None, 5, k, v, cache)
    q = _rows((B, 1, 8, d), DT["bf16"], 3) * 10
    sel = _i32([0, 1, 2, 3, 4]).expand(B, Hkv, 1, 5).contiguous()
    out, lse = torch.empty_like(q), torch.empty((B, 8, 1), device="cuda")
    _lib.msa_sparse_decode_packed(shape, None, None, 5, q, cache, sel, out, lse)
    o, l, _ = co.decode_mass(q, co.pack_values(to_np(k))[0], co.pack_values(to_np(v))[0],
                             sel.cpu().numpy(), [cap])
    for g in range(4):                                             # each group at its own scale
        a, b = to_np(out)[..., 32 * g:32 * g + 32], o[..., 32 * g:32 * g + 32]
        assert np.linalg.norm(a - b) <= 5e-3 * np.linalg.norm(b), g
    # fp32 logits of magnitude |z|: their sums' rounding scales with it
    assert np.all(np.abs(to_np(lse) - l) <= 2e-3 + (d + 8) * 2.0 ** -24 * np.abs(l) * 8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_decode_small_value_under_all_the_weight(dtype):
    """One key of values 2^-20 of the others' takes (almost) all the weight: its digits stay."""
    B, cap, Hkv, d = 1, 400, 1, 64
    shape = _shape(B, cap, 4, Hkv, d, 4, dtype)
    k, v = _rows((B, Hkv, cap, d), DT[dtype], 1) * 0.1, _rows((B, Hkv, cap, d), DT[dtype], 2)
    q = torch.ones((B, 1, 4, d), device="cuda").to(DT[dtype])
    k[0, 0, 7] = 10.0                                       # a logit of 80, the others' about 0
    v[0, 0, 7] *= 2.0 ** -20
    cache = torch.zeros((4, Hkv, 160 * d), dtype=torch.uint8, device="cuda")
    _lib.msa_cache_pack(shape, cap, None, None, None, 4, k, v, cache)
    sel = _i32([3, 2, 1, 0]).expand(B, Hkv, 1, 4).contiguous()   # the key comes last
    out = torch.empty_like(q)
    _lib.msa_sparse_decode_packed(shape, None, None, 4, q, cache, sel, out)
    o, _, _ = co.decode_mass(q, co.pack_values(to_np(k))[0], co.pack_values(to_np(v))[0],
                             sel.cpu().numpy(), [cap])
    # the key's p * step is 2^-10 of fp16's unit here: normal, so 2^-11 of it (fp32: its rest too)
    assert np.abs(o).max() < 1e-5
    check_out(out.double() * 2.0 ** 20, o * 2.0 ** 20, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_decode_extreme_magnitudes(dtype):
    """Queries, keys and values far from one, the logits in the ordinary range; a query row of
    zeros; fp32 and bf16."""
    B, cap, Hkv, d = 1, 500, 2, 128
    shape = _shape(B, cap, 8, Hkv, d, 4, dtype)
    sel = _i32([0, 1, 2, 3]).expand(B, Hkv, 1, 4).contiguous()
    for qs, vs in ((2.0 ** 80, 2.0 ** 100), (2.0 ** -80, 2.0 ** -80), (2.0 ** 40, 1.0)):
        k, v = _rows((B, Hkv, cap, d), DT[dtype], 1) / qs, _rows((B, Hkv, cap, d), DT[dtype], 2) * vs
        q = _rows((B, 1, 8, d), DT[dtype], 3) * qs
        q[0, 0, 3] = 0
        cache = torch.zeros((4, Hkv, 160 * d), dtype=torch.uint8, device="cuda")
        _lib.msa_cache_pack(shape, cap, None, None, None, 4, k, v, cache)
        out, lse = torch.empty_like(q), torch.empty((B, 8, 1), device="cuda")
        _lib.msa_sparse_decode_packed(shape, None, None, 4, q, cache, sel, out, lse)
        o, l, _ = co.decode_mass(q, co.pack_values(to_np(k))[0], co.pack_values(to_np(v))[0],
                                 sel.cpu().numpy(), [cap])
        check_out(out.double() / vs, o / vs, dtype)
        check_lse(lse, l, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_decode_not_a_number(dtype):
    """A NaN in a key that is seen shows in every output of its head, alone or among others; one in
    a value in its group's dims; none of another sequence's or head's."""
    B, cap, Hkv, d = 2, 300, 2, 64
    shape = _shape(B, cap, 4, Hkv, d, 3, dtype)
    for where, lens in (("alone", [1, 300]), ("among", [290, 300])):
        k, v = _rows((B, Hkv, cap, d), DT[dtype], 1), _rows((B, Hkv, cap, d), DT[dtype], 2)
        k[0, 0, 0, 5] = float("nan")
        v[1, 1, 200, 40] = float("nan")
        cache = torch.full((6, Hkv, 160 * d), 0xFF, dtype=torch.uint8, device="cuda")
        _lib.msa_cache_pack(shape, cap, _i32([0, 0]), _i32(lens), None, 6, k, v, cache)
        sel = _i32([0, 1, 2]).expand(B, Hkv, 1, 3).contiguous()
        q = _rows((B, 1, 4, d), DT[dtype], 3)
        out, lse = torch.empty_like(q), torch.empty((B, 4, 1), device="cuda")
        _lib.msa_sparse_decode_packed(shape, _i32(lens), None, 6, q, cache, sel, out, lse)
        bad = torch.isnan(out)
        want = torch.zeros_like(bad)
        want[0, 0, :2] = True
        want[1, 0, 2:, 32:] = True
        assert torch.equal(bad, want), where
        assert torch.equal(torch.isnan(lse[..., 0]), want[:, 0, :, 0]), where


def test_packed_decode_many_sequences():
    """More (sequence, KV head) pairs than SMs: one CTA each, several waves."""
    B, cap, Hkv, d = 90, 260, 4, 64
    lens = [1 + (37 * i) % cap for i in range(B)]
    cache, table, P, kv, vv = _filled(B, cap, Hkv, d, lens, "bf16", True, 3)
    shape = _shape(B, cap, 8, Hkv, d, 3)
    sel = _i32([0, 1, 2]).expand(B, Hkv, 1, 3).contiguous()
    q = _rows((B, 1, 8, d), DT["bf16"], 1)
    out, lse, mass = torch.empty_like(q), torch.empty((B, 8, 1), device="cuda"), \
        torch.zeros((B, Hkv, 3), device="cuda")
    _lib.msa_sparse_decode_packed(shape, _i32(lens), table, P, q, cache, sel, out, lse, mass)
    o, l, m = co.decode_mass(q, list(kv), list(vv), sel.cpu().numpy(), lens)
    check_out(out, o, "bf16")
    check_lse(lse, l, "bf16")
    tol = _weight_tol(to_np(q), kv, d ** -0.5, d) + 2.0 ** -24
    assert np.all(np.abs(to_np(mass) - m) <= tol * m)


def test_packed_cache_past_32_bit_offsets():
    """A pool of more than 4 GiB: the last physical blocks hold the sequence."""
    Hkv, d = 8, 128
    P = (1 << 32) // (Hkv * 160 * d) + 40
    cache = torch.zeros((P, Hkv, 160 * d), dtype=torch.uint8, device="cuda")
    lens, cap = [1000], 1024
    table = torch.arange(P - 8, P, dtype=torch.int32, device="cuda").view(1, 8)
    shape = _shape(1, cap, 16, Hkv, d, 8)
    k, v = _rows((1, Hkv, 1000, d), DT["bf16"], 1), _rows((1, Hkv, 1000, d), DT["bf16"], 2)
    _lib.msa_cache_pack(shape, 1000, None, _i32(lens), table, P, k, v, cache)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    _lib.msa_cache_unpack(shape, 1000, None, _i32(lens), table, P, cache, ko, vo)
    kv, vv = co.pack_values(to_np(k))[0], co.pack_values(to_np(v))[0]
    assert np.array_equal(to_np(vo), to_np(torch.from_numpy(vv).bfloat16()))
    q = _rows((1, 1, 16, d), DT["bf16"], 3)
    sel = torch.arange(8, dtype=torch.int32, device="cuda").expand(1, Hkv, 1, 8).contiguous()
    out = torch.empty_like(q)
    _lib.msa_sparse_decode_packed(shape, _i32(lens), table, P, q, cache, sel, out)
    o, _, _ = co.decode_mass(q, list(kv), list(vv), sel.cpu().numpy(), lens)
    check_out(out, o, "bf16")


def test_packed_decode_concurrent_and_graph():
    """Two calls at once on two streams, and a captured step replayed on new inputs."""
    lens, cap = [1500, 900], 1500
    cache, table, P, kv, vv = _filled(2, cap, 4, 128, lens, "bf16", True, 8)
    shape = _shape(2, cap, 64, 4, 128, 6)
    sel_np = random_selection(np.array([[[12]] * 4, [[8]] * 4]), 6, 1)
    sel = torch.from_numpy(sel_np).cuda()
    n = _i32(lens)
    qs = [_rows((2, 1, 64, 128), DT["bf16"], s) for s in range(2)]
    want = []
    for q in qs:
        out = torch.empty_like(q)
        _lib.msa_sparse_decode_packed(shape, n, table, P, q, cache, sel, out)
        want.append(out)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in qs], [torch.empty_like(q) for q in qs]
    for _ in range(20):
        for st, q, out in zip(streams, qs, outs):
            _lib.msa_sparse_decode_packed(shape, n, table, P, q, cache, sel, out, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    q, out, mass = qs[0].clone(), torch.zeros_like(qs[0]), torch.zeros((2, 4, 12), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.msa_sparse_decode_packed(shape, n, table, P, q, cache, sel, out, None, mass)
    q.copy_(qs[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[1])
    once = mass.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(mass, 2 * once) and once.any()


def test_packed_binding_refuses():
    cache, table, P, _, _ = _filled(1, 200, 4, 128, [200], "bf16", True, 2)
    shape = _shape(1, 200, 16, 4, 128, 2)
    q = _rows((1, 1, 16, 128), DT["bf16"], 1)
    sel, out = _i32([[[[0, 1]]] * 4]), torch.empty_like(q)
    ok = (shape, _i32([200]), table, P, q, cache, sel, out)
    _lib.msa_sparse_decode_packed(*ok)
    for i, bad in ((1, _i32([200]).long()), (1, _i32([])), (2, table[:, :1].contiguous()),
                   (4, q.float()), (4, q[..., ::2]), (5, cache[:-1]), (5, cache.view(torch.int8)),
                   (6, sel[:, :2].contiguous()), (7, out.cpu())):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            _lib.msa_sparse_decode_packed(*args)
    torch.cuda.synchronize()
