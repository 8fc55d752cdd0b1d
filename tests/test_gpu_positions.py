"""Rotary positions of decode steps after an eviction: the keys that stay are rotated to the
positions they had, so the new tokens' positions go on from there, whatever the caches' lengths
are.  The references hold unrotated rows with their absolute positions and rotate by those.

Outputs and log-sum-exps use the package's attention tolerances (tests/parity.py); what is only
moved, and scores of the same operands, are compared exactly."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api
from oracle import cache_ops as co
from tests.parity import check_lse, check_out, check_scores, to_np
from tests.test_gpu_packed import _i32, _rows

BF = torch.bfloat16


def _rope(dim=128, index=False):
    freqs, scale = api.rope_freqs(dim, device="cuda")
    return api.Rope(freqs, api.rope_freqs(64, device="cuda")[0] if index else None, scale)


def _at(x, positions, freqs, head_major):
    """x [n, H, 1, d] or [n, 1, H, d]: row i rotated to positions[i]."""
    return api.rope([(x.contiguous(), freqs, head_major)], _i32(positions).view(-1, 1))[0]


@pytest.mark.gpu
def test_packed_steps_after_evictions():
    """A serving loop over a paged 4-bit cache of two sequences that are cut twice; positions
    count on."""
    B, Hq, Hkv, d, cap, topk = 2, 16, 4, 128, 1024, 3
    rope = _rope()
    P = B * 8
    table = torch.randperm(P, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    table = table.to(torch.int32).view(B, 8).contiguous()
    cache = api.alloc_packed_cache(P, Hkv, d)
    pool = torch.zeros((P, 128, 128), dtype=BF, device="cuda")
    mass = torch.zeros((B, Hkv, 8), device="cuda")
    n = [890, 640]                                     # rows of each cache
    lens, positions = _i32(n), _i32(n)                 # positions: of the next token
    shape = _lib.make_shape(B, 1, cap, Hq, Hkv, d, 128, 128, topk, 1)
    n0 = max(n)
    k, v = _rows((B, Hkv, n0, d), BF, 1), _rows((B, Hkv, n0, d), BF, 2)
    ik = _rows((B, n0, 128), BF, 3)
    kr, ikr = api.rope([(k, rope.freqs, True), (ik, rope.freqs, False)], scale=rope.scale)
    _lib.msa_cache_pack(shape, n0, torch.zeros_like(lens), lens, table, P, kr, v, cache)
    for b in range(B):
        for j in range(-(-n[b] // 128)):
            part = ikr[b, 128 * j:min(n[b], 128 * (j + 1))]
            pool[table[b, j].item(), :part.shape[0]] = part
    # the reference: rows in the order of the cache, unrotated, and their positions
    rows = [dict(k=k[b, :, :n[b]].transpose(0, 1), v=v[b, :, :n[b]].transpose(0, 1),
                 ik=ik[b, :n[b]], at=list(range(n[b]))) for b in range(B)]
    for step in range(6):
        q = _rows((B, 1, Hq, d), BF, 10 + step)
        k1, v1 = (_rows((B, Hkv, 1, d), BF, 20 + 2 * step + i) for i in range(2))
        iq, ik1 = _rows((B, 1, 4, 128), BF, 40 + step), _rows((B, 1, 128), BF, 50 + step)
        lens += 1
        now = [int(x) for x in positions]
        for b, r in enumerate(rows):
            assert now[b] == max(r["at"]) + 1
            r["k"], r["v"] = torch.cat([r["k"], k1[b, :, 0][None]]), torch.cat([r["v"], v1[b, :, 0][None]])
            r["ik"] = torch.cat([r["ik"], ik1[b]])
            r["at"].append(now[b])
            n[b] += 1
            pool[table[b, (n[b] - 1) // 128].item(), (n[b] - 1) % 128] = \
                _at(ik1[b][:, None, None], [now[b]], rope.freqs, False)[0, 0, 0]
        got = api.decode_packed(q, k1, v1, cache, iq, pool, lens, table, cap, topk, rope=rope,
                                mass=mass, positions=positions)
        _lib.msa_get_device_status()
        qr, iqr = _at(q, now, rope.freqs, False), to_np(_at(iq, now, rope.freqs, False))
        held = []
        for r in rows:
            kk = to_np(_at(r["k"][:, :, None], r["at"], rope.freqs, True))[:, :, 0]
            held.append((np.moveaxis(co.pack_values(kk)[0], 0, 1),
                         np.moveaxis(co.pack_values(to_np(r["v"]))[0], 0, 1)))
        sel = to_np(got["sel"])
        o, l, _ = co.decode_mass(qr, [x for x, _ in held], [x for _, x in held], sel, n)
        check_out(got["out"], o, "bf16", f"step {step}")
        check_lse(got["lse"], l, "bf16", f"step {step}")
        for b, r in enumerate(rows):
            z = to_np(_at(r["ik"][:, None, None], r["at"], rope.freqs, False))[:, 0, 0] @ iqr[b, 0].T
            z = z * 128 ** -0.5
            want = [z[128 * j:128 * (j + 1)].max(0) for j in range(-(-n[b] // 128))]
            check_scores(to_np(got["scores"])[b, :, 0, :len(want)], np.stack(want, 1))
            assert all((n[b] - 1) // 128 in row for row in sel[b, :, 0])
        positions += 1
        if step in (1, 3):
            kept = to_np(api.evict_paged(lens, mass, table, cap, 4 if step == 1 else 3))
            for b, r in enumerate(rows):
                stay = [j for x in kept[b] if x >= 0 for j in range(128 * int(x), min(n[b], 128 * int(x) + 128))]
                for name in ("k", "v", "ik"):
                    r[name] = r[name][stay]
                r["at"] = [r["at"][j] for j in stay]
                n[b] = len(stay)
            assert n == [int(x) for x in lens] and all(now[b] + 1 > n[b] + 100 for b in range(B))


@pytest.mark.gpu
@pytest.mark.parametrize("index", [False, True])
def test_contiguous_step_after_eviction(index):
    """api.decode over cut caches with the token's own position is the decode over the kept
    blocks of the long ones, where that position is the last row's."""
    B, Hq, Hkv, d, L = 2, 16, 4, 128, 1500
    rope = _rope(index=index)
    q, k, v = (_rows(s, BF, i) for i, s in enumerate(((B, 1, Hq, d), (B, Hkv, L, d), (B, Hkv, L, d))))
    iq, ik = _rows((B, 1, 4, 128), BF, 5), _rows((B, L, 128), BF, 6)
    index_freqs = rope.index_freqs if index else rope.freqs
    k, ik = api.rope([(k, rope.freqs, True), (ik, index_freqs, False)])
    mass = torch.zeros((B, Hkv, 12), device="cuda")
    long = api.decode(q, k, v, iq, ik, top_k=5, mass=mass, rope=rope)
    same = api.decode(q, k, v, iq, ik, top_k=5, rope=rope, positions=_i32([L - 1] * B))
    for name in ("scores", "sel", "out", "lse"):
        assert torch.equal(long[name], same[name])
    cut = api.evict(k, v, ik, mass, keep=6)
    kept = to_np(cut["kept"])
    step = api.decode(q, cut["k"], cut["v"], iq, cut["idx_k"], top_k=6, rope=rope,
                      positions=_i32([L - 1] * B))
    sel = torch.from_numpy(np.repeat(kept[:, None, None], Hkv, 1).astype(np.int32)).cuda().contiguous()
    shape = _lib.make_shape(B, 1, L, Hq, Hkv, d, 128, 128, 6, 1)
    qr = _at(q, [L - 1] * B, rope.freqs, False)
    out, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")
    ws = torch.empty(_lib.msa_workspace_bytes(shape, 1) // 4 + 4, device="cuda")
    _lib.msa_sparse_decode(shape, qr, k, v, sel, out, lse, ws)
    check_out(step["out"], to_np(out), "bf16")
    check_lse(step["lse"], to_np(lse), "bf16")
    gathered = np.take_along_axis(to_np(long["scores"])[:, :, 0], np.repeat(kept[:, None], Hkv, 1), 2)
    assert np.array_equal(to_np(step["scores"])[:, :, 0], gathered)


@pytest.mark.gpu
def test_positions_of_each_sequence():
    """Every sequence has a position of its own, up to the largest."""
    B, Hq, Hkv, d, L = 3, 8, 2, 64, 400
    rope = _rope(64)
    q, k, v = (_rows(s, BF, i) for i, s in enumerate(((B, 1, Hq, d), (B, Hkv, L, d), (B, Hkv, L, d))))
    iq, ik = _rows((B, 1, Hkv, 64), BF, 5), _rows((B, L, 64), BF, 6)
    at = [0, 5_000_000, 2 ** 31 - 1]
    got = api.decode(q, k, v, iq, ik, top_k=2, rope=rope, positions=_i32(at))
    want = api.decode(_at(q, at, rope.freqs, False), k, v, _at(iq, at, rope.freqs, False), ik, top_k=2)
    for name in ("scores", "sel", "out", "lse"):
        assert torch.equal(got[name], want[name])


@pytest.mark.parametrize("bad", ["shape", "long", "no_rope"])
def test_refused_positions(bad):
    B, H, L, d = 2, 4, 1000, 128
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt)  # noqa: E731
    positions = {"shape": z(B, 2, dt=torch.int32), "long": z(B + 1, dt=torch.int32),
                 "no_rope": z(B, dt=torch.int32)}[bad]
    rope = None if bad == "no_rope" else api.Rope(api.rope_freqs(d)[0])
    q, k, new = z(B, 1, 16, d), z(B, H, L, d), z(B, H, 1, d)
    with pytest.raises(ValueError, match="positions"):
        api.decode(q, k, k, z(B, 1, H, d), z(B, L, d), rope=rope, positions=positions)
    with pytest.raises(ValueError, match="positions"):
        api.decode_packed(q, new, new, z(20, H, 160 * d, dt=torch.uint8), z(B, 1, H, d),
                          z(20, 128, d), z(B, dt=torch.int32), z(B, 8, dt=torch.int32), L, rope=rope,
                          positions=positions)
