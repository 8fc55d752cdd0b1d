"""Decode with attention weights when a split gives up a bounded wait.  The test hook lets the CTA
of a row's first split copy one block only, so the wait for its second runs out (a flag that
nothing sets); no copy is in flight then.  The call reports MSA_ERR_TIMEOUT, and the caller's
accumulated weights, which outlive the call, are as they were for every row that failed."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api
from oracle import cache_ops as co
from tests.parity import check_lse, check_out, to_np
from tests.test_gpu_packed import _i32, _rows, _weight_tol

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _sel(B, Hkv, topk, nB):
    """Sequence 0: topk blocks; sequence 1: one block, in a first split that does not fail."""
    rng = np.random.default_rng(5)
    sel = np.full((B, Hkv, 1, topk), -1, dtype=np.int32)
    for g in range(Hkv):
        sel[0, g, 0] = np.sort(rng.permutation(nB)[:topk])
        sel[1, g, 0, 0] = g
    return sel


def _faulty(call):
    _lib.msa_get_device_status()
    _lib.msa_debug_set_fault(2)
    try:
        call()
        with pytest.raises(_lib.MsaError) as e:
            _lib.msa_get_device_status()
        assert e.value.status == _lib.MSA_ERR_TIMEOUT
    finally:
        _lib.msa_debug_set_fault(0)
    _lib.msa_get_device_status()


def _check(call, out, lse, mass, o, l, w, tol):
    _faulty(call)
    assert bool((mass[0] == 3).all())                  # nothing added for the rows that failed
    assert bool((out[0] == 0).all()) and bool(torch.isneginf(lse[0]).all())
    # an addition to 3 rounds once more; a wide group makes two
    bound = tol * w + 2 * 2.0 ** -24 * (3 + w)
    assert np.all(np.abs(to_np(mass) - 3 - w)[1] <= bound[1])
    check_out(out[1:], o[1:], "bf16")
    check_lse(lse[1:], l[1:], "bf16")
    mass.fill_(3)
    call()                                             # and the next call is right
    _lib.msa_get_device_status()
    check_out(out, o, "bf16")
    check_lse(lse, l, "bf16")
    assert np.all(np.abs(to_np(mass) - 3 - w) <= bound)


@pytest.mark.parametrize("paged", [False, True])
def test_16_bit_cache(paged):
    B, Hq, Hkv, d, L, topk = 2, 32, 4, 128, 64 * 128, 60
    shape = _lib.make_shape(B, 1, L, Hq, Hkv, d, 128, 128, topk, 1)
    q, k, v = (_rows(s, BF, i) for i, s in enumerate(((B, 1, Hq, d), (B, Hkv, L, d), (B, Hkv, L, d))))
    sel_np = _sel(B, Hkv, topk, 64)
    sel = torch.from_numpy(sel_np).cuda()
    out, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")
    mass = torch.full((B, Hkv, 64), 3.0, device="cuda")
    # what an earlier call may have left: log-sums that would add infinite weights
    ws = torch.full((_lib.msa_workspace_bytes(shape, 4) // 4 + 4,), 200.0, device="cuda")
    pool = [None, None, 0, k, v]
    if paged:
        table = torch.randperm(B * 64, device="cuda").to(torch.int32).view(B, 64)
        pools = []
        for x in (k, v):
            p = torch.empty((B * 64, Hkv, 128, d), dtype=BF, device="cuda")
            p[table.long()] = x.view(B, Hkv, 64, 128, d).transpose(1, 2)
            pools.append(p)
        pool = [_i32([L] * B), table, B * 64, *pools]
    o, l, w = co.decode_mass(q, list(to_np(k)), list(to_np(v)), sel_np, [L] * B)
    _check(lambda: _lib.msa_sparse_decode_mass(shape, *pool[:3], q, *pool[3:], sel, out, lse, mass, ws),
           out, lse, mass, o, l, w, _weight_tol(to_np(q), to_np(k), d ** -0.5, d))


@pytest.mark.parametrize("heads", [8, 20])             # a group in one pass, and in two
def test_4_bit_cache(heads):
    B, Hkv, d, L, topk = 2, 2, 128, 64 * 128, 60
    Hq = heads * Hkv
    shape = _lib.make_shape(B, 1, L, Hq, Hkv, d, 128, 128, topk, 1)
    q, k, v = (_rows(s, BF, i) for i, s in enumerate(((B, 1, Hq, d), (B, Hkv, L, d), (B, Hkv, L, d))))
    cache = api.alloc_packed_cache(B * 64, Hkv, d)
    _lib.msa_cache_pack(shape, L, None, None, None, B * 64, k, v, cache)
    sel_np = _sel(B, Hkv, topk, 64)
    sel = torch.from_numpy(sel_np).cuda()
    out, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")
    mass = torch.full((B, Hkv, 64), 3.0, device="cuda")
    kv = [list(co.pack_values(to_np(x))[0]) for x in (k, v)]
    o, l, w = co.decode_mass(q, *kv, sel_np, [L] * B)
    _check(lambda: _lib.msa_sparse_decode_packed(shape, None, None, B * 64, q, cache, sel, out, lse, mass),
           out, lse, mass, o, l, w, _weight_tol(to_np(q), np.stack(kv[0]), d ** -0.5, d))
