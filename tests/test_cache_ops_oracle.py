"""Pins of the fp64 references in oracle/cache_ops.py (CPU): each is checked against what its
definition fixes, by other means than its own code."""
import itertools
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from block_sparse_gqa_02_gb300 import api
from oracle import cache_ops as co


def _freqs(rot, **kw):
    return api.rope_freqs(rot, **kw)[0].numpy()


# ------------------------------------------------------------------------------- rotary

@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_pairs_by_hand(interleaved):
    """Every pair turned by plain-loop trigonometry of pos * base^(-2 i / rot)."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 5, 3, 48))
    pos = rng.integers(0, 1000, (2, 5))
    y = co.rope(x, pos, _freqs(32), scale=1.5, interleaved=interleaved)
    for b, t, h in itertools.product(range(2), range(5), range(3)):
        for i in range(16):
            a = pos[b, t] * 10000.0 ** (-2 * i / 32)
            j0, j1 = (2 * i, 2 * i + 1) if interleaved else (i, i + 16)
            x0, x1 = x[b, t, h, j0], x[b, t, h, j1]
            assert abs(y[b, t, h, j0] - 1.5 * (x0 * math.cos(a) - x1 * math.sin(a))) < 1e-11
            assert abs(y[b, t, h, j1] - 1.5 * (x0 * math.sin(a) + x1 * math.cos(a))) < 1e-11
    assert np.array_equal(y[..., 32:], x[..., 32:])


def test_rope_scores_depend_on_distance_only():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 1, 64))
    f = _freqs(64)
    dots = [float((co.rope(q, [[p + 17]], f) * co.rope(k, [[p]], f)).sum())
            for p in (0, 5, 4096, 1 << 20, -3)]
    assert np.ptp(dots) < 1e-9


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_inverse_is_the_gradient(interleaved):
    """inverse = transpose: central differences of sum(dy . rope(x))."""
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((2, 1, 2, 1, 32))
    f, pos = _freqs(16), [[7, 900]]
    kw = dict(scale=0.7, interleaved=interleaved)
    dx = co.rope(dy, pos, f, inverse=True, **kw)
    for t, i in itertools.product(range(2), range(32)):
        e = np.zeros_like(x)
        e[0, t, 0, i] = 1e-5
        num = ((co.rope(x + e, pos, f, **kw) - co.rope(x - e, pos, f, **kw)) * dy).sum() / 2e-5
        # dims from rotary_dim on are copied, so their gradient is copied too
        assert abs(num - dx[0, t, 0, i]) < 1e-8


def test_rope_freq_table():
    """The table is 2^64 times the frequency in turns; each scaling by its own property."""
    f, scale = api.rope_freqs(64)
    for i, v in enumerate(f.tolist()):
        want = Fraction(10000.0 ** (-2 * i / 64) / (2 * math.pi)) * 2 ** 64
        assert abs(v - want) <= 2 + want * Fraction(1, 2 ** 50) and scale == 1.0
    lin, _ = api.rope_freqs(64, scaling="linear", factor=4.0)
    assert np.allclose(lin.double() * 4, f.double(), rtol=1e-14)
    ntk, _ = api.rope_freqs(64, scaling="ntk", factor=4.0)
    assert int(ntk[0]) == int(f[0])                       # the highest frequency stays
    assert abs(float(ntk[-1]) * 4 / float(f[-1]) - 1) < 1e-12   # the lowest is divided
    yarn, s = api.rope_freqs(64, scaling="yarn", factor=4.0, original_len=4096)
    turns = f.double() / 2.0 ** 64 * 4096
    assert torch.equal(yarn[turns > 32], f[turns > 32])
    assert np.allclose(yarn[turns < 1].double() * 4, f[turns < 1].double(), rtol=1e-14)
    assert abs(s - (0.1 * math.log(4.0) + 1)) < 1e-15
    for bad in (dict(rotary_dim=24), dict(rotary_dim=0), dict(rotary_dim=32, scaling="nope"),
                dict(rotary_dim=32, factor=0.5), dict(rotary_dim=32, base=1.0),
                dict(rotary_dim=32, scaling="yarn", factor=2.0)):
        with pytest.raises(ValueError):
            api.rope_freqs(**bad)


# ------------------------------------------------------------------------- the 4-bit cache

@pytest.mark.parametrize("scale,shift", [(1.0, 0.0), (1e-6, 0.0), (1e30, 0.0), (0.1, 5.0),
                                         (1e-3, 100.0)])
def test_pack_error_bound(scale, shift):
    """|value - x| <= step / 2, and where the group's ends are clipped because step and mid are
    bf16, 8 steps' and the middle's rounding more."""
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((50, 128)) * scale + shift).astype(np.float32)
    v, step, mid = co.pack_values(x)
    err = np.abs(v - x).reshape(50, 4, 32)
    bound = step / 2 + 2.0 ** -8 * np.abs(mid) + 8 * 2.0 ** -8 * step
    assert np.all(err <= bound[..., None] * (1 + 1e-6))


def test_pack_special_groups():
    x = np.zeros((6, 32), dtype=np.float32)
    x[1] = 3.14159
    x[2] = np.linspace(-1, 1, 32)
    x[3, 5] = np.nan
    x[4, 7] = -np.inf
    x[5] = np.linspace(0, 1e-38, 32)
    v, step, _ = co.pack_values(x)
    assert np.all(v[0] == 0) and np.all(v[1] == co.round_bf16(np.float32(3.14159)))
    assert np.isnan(v[3]).all() and np.isnan(v[4]).all()
    assert step[5, 0] == 0 and np.all(np.abs(v[5]) <= 2e-38)
    assert np.abs(v[2] - x[2]).max() <= 2 / 15 / 2 * 1.02


def test_round_bf16_is_torch():
    x = np.random.default_rng(4).standard_normal(10000).astype(np.float32) * 1e3
    assert np.array_equal(co.round_bf16(x), torch.from_numpy(x).bfloat16().float().numpy())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("is_v", [False, True])
def test_record_is_a_bijection(d, is_v):
    byte, half = co.record_offsets(d, is_v)
    slots = byte * 2 + half
    assert np.array_equal(np.sort(slots.reshape(-1)), np.arange(128 * d))


# ----------------------------------------------------------------- weights and eviction

def test_mass_sums_to_the_heads_and_matches_attention():
    rng = np.random.default_rng(5)
    q = rng.standard_normal((2, 1, 8, 64))
    k, v = rng.standard_normal((2, 2, 2, 300, 64))
    sel = np.array([[[[0, 2, -1]], [[1, 2, -1]]], [[[0, 1, 2]], [[-1, -1, -1]]]], dtype=np.int32)
    out, lse, mass = co.decode_mass(q, k, v, sel, [300, 257])
    ref_o, ref_l = oracle.sparse_attention(q[:1], k[:1], v[:1], sel[:1], 128, 1, None, 299)
    assert np.allclose(out[0], ref_o[0]) and np.allclose(lse[0], ref_l[0])
    assert np.allclose(mass.sum(-1)[0], 4) and np.allclose(mass.sum(-1)[1], [4, 0])
    assert np.isneginf(lse[1, 4:]).all() and np.all(out[1, 0, 4:] == 0)
    # one block: all of a head's weight is there
    one = np.where(sel == 2, 2, -1)
    _, _, m1 = co.decode_mass(q, k, v, one, [300, 257])
    assert np.allclose(m1[0, :, 2], 4) and np.allclose(m1[1, 0, 2], 4)


def test_evict_against_enumeration():
    """On tiny rows the kept set is the one subset of its size that holds the forced blocks and
    has, of those, the lexicographically best (score, -index) list."""
    rng = np.random.default_rng(6)
    for case in range(30):
        nB = int(rng.integers(1, 8))
        L = int(rng.integers(0, nB * 128 + 1))
        first, recent = int(rng.integers(0, 2)), int(rng.integers(1, 3))
        keep = first + recent + int(rng.integers(0, 3))
        mass = rng.integers(0, 3, (1, 2, nB)).astype(np.float32)      # many ties
        table = rng.permutation(50)[:nB].astype(np.int32)[None]
        kept, lens, moved, rows = co.evict(mass, [L], keep, first, recent, table=table)
        n = -(-L // 128)
        score = mass[0].sum(0)
        forced = {i for i in range(n) if i < first or i >= n - recent}
        best = max((c for c in itertools.combinations(range(n), min(n, keep)) if forced <= set(c)),
                   key=lambda c: sorted(((score[i], -i) for i in c if i not in forced), reverse=True))
        got = [int(x) for x in kept[0] if x >= 0]
        assert got == sorted(best)
        assert lens[0] == L - 128 * (n - len(got))
        assert np.array_equal(moved[0, :, :len(got)], mass[0][:, got])
        assert np.all(moved[0, :, len(got):] == 0)
        gone = [i for i in range(n) if i not in got]
        assert rows[0].tolist() == table[0][got + gone + list(range(n, nB))].tolist()
