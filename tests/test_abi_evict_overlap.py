"""Buffers of msa_cache_evict that share memory: an output may be its own input, and nothing else."""
import ctypes
import itertools

import pytest

from block_sparse_gqa_02_gb300 import _lib

BASE, APART = 1 << 40, 1 << 30      # never dereferenced: the host has no GPU, or the call is refused
B, HKV, NB, KEEP = 3, 2, 8, 5
SIZES = dict(kept=B * KEEP * 4, new_lens=B * 4, mass_out=B * HKV * NB * 4, table_out=B * NB * 4,
             seq_lens=B * 4, mass=B * HKV * NB * 4, block_table=B * NB * 4)
OWN = dict(mass_out="mass", table_out="block_table", new_lens="seq_lens")
OUT = ("kept", "new_lens", "mass_out", "table_out")


def _call(**at):
    a = {n: BASE + i * APART for i, n in enumerate(SIZES)}
    a.update(at)
    lib = _lib.load()
    s = _lib.make_shape(B, 1, NB * 128, 4, HKV, 128, 128, 128, 1, 1)
    return lib.msa_cache_evict(ctypes.byref(s), KEEP, 1, 2, a["seq_lens"], a["mass"], a["block_table"],
                               a["kept"], a["new_lens"], a["mass_out"], a["table_out"], None), a


PAIRS = [(x, y) for x, y in itertools.product(OUT, SIZES) if x != y]


@pytest.mark.parametrize("x,y", PAIRS)
def test_overlaps_are_refused(x, y):
    lib = _lib.load()
    base = BASE + 100 * APART
    at = [base + 16, base + (SIZES[y] - 1) // 16 * 16]    # y starts at base: inside it, in its last 16 bytes
    at += [base - (SIZES[x] - 1) // 16 * 16]              # ... and x reaching into y's first
    if OWN.get(x) != y:
        at.append(base)
    for place in at:
        if OWN.get(x) == y and place == base or not base - SIZES[x] < place < base + SIZES[y]:
            continue
        status, _ = _call(**{x: place, y: base})
        assert status == _lib.MSA_ERR_INVALID_ARG, (x, y, place - base)
        assert b"overlaps" in lib.msa_last_error()


def test_neighbours_and_own_inputs_are_not(monkeypatch):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    base = BASE + 100 * APART
    for x, y in PAIRS:
        after = (SIZES[y] + 15) // 16 * 16
        assert _call(**{x: base + after, y: base})[0] == _lib.MSA_ERR_CUDA, (x, y)      # no device
        before = (SIZES[x] + 15) // 16 * 16
        assert _call(**{x: base - before, y: base})[0] == _lib.MSA_ERR_CUDA, (x, y)
    for x, y in OWN.items():
        assert _call(**{x: base, y: base})[0] == _lib.MSA_ERR_CUDA
