"""Index scores and attention of drafted tokens in a call that gave up a wait."""
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api
from tests.test_gpu_packed import _i32, _rows
from tests.test_gpu_tree_step import BF, D, HKV, _drafts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("B,L,gives_up", [(1, 60000, True), (2, 20 * 128, False), (160, 384, True), (160, 300, True)])
def test_given_up_scores_are_written(packed, B, L, gives_up):
    """The CTA of a sequence's first range copies one tile only and gives up its wait, if it has more
    (20 blocks on 75 CTAs: it has not).  Every score is written all the same: the right one, or -inf."""
    N = 4
    cap = L + 140                                           # a block that only drafts, or nothing, can be in
    nB = -(-cap // 128)
    x, lens = _drafts(B, N, 5), _i32([L] * B)
    parents = _i32([[-1, 0, 1, 2]] * B)
    shape = _lib.make_shape(B, N, cap, 32, HKV, D, D, 128, 4, 1)
    mask = torch.empty((B, N), dtype=torch.int64, device="cuda")
    _lib.msa_tree_mask(shape, lens, parents, mask)
    keys, drafts, n_phys = _rows((B, cap, D), BF, 3), x["idx_k"], B * nB
    if packed:
        cache = api.alloc_index_cache(n_phys)
        api.pack_index(keys, cache, starts=torch.zeros_like(lens), capacity=cap)
        keys, drafts = cache, api.alloc_index_cache(B)
        api.pack_index(x["idx_k"], drafts, capacity=N)

    def run(scores):
        _lib.msa_index_scores_tree(shape, lens, None, n_phys, mask, x["idx_q"], keys, drafts, scores, packed=packed)
    good, got = (torch.full((B, HKV, N, nB), 7.0, device="cuda") for _ in range(2))
    run(good)
    _lib.msa_get_device_status()
    assert not (good == 7.0).any()
    _lib.msa_debug_set_fault(2)
    try:
        run(got)
        if gives_up:
            with pytest.raises(_lib.MsaError) as e:
                _lib.msa_get_device_status()
            assert e.value.status == _lib.MSA_ERR_TIMEOUT
        else:
            _lib.msa_get_device_status()
    finally:
        _lib.msa_debug_set_fault(0)
    assert ((got == good) | torch.isneginf(got)).all()
    assert (got != good).any() == gives_up
    run(got)
    _lib.msa_get_device_status()
    assert torch.equal(got, good)


@pytest.mark.parametrize("B,L,topk", [(1, 60000, 120), (40, 700, 4)])
def test_given_up_attention_is_written(B, L, topk):
    """The CTAs of the first splits give up; every row and log-sum, and every partial one that they are
    joined from, is written: without the lost blocks, or zeros and -inf."""
    N, cap = 4, L + 4
    x, lens = _drafts(B, N, 5), _i32([L] * B)
    kc, vc, ic = _rows((B, HKV, cap, D), BF, 1), _rows((B, HKV, cap, D), BF, 2), _rows((B, cap, D), BF, 3)
    good = api.decode_tree(**x, k_cache=kc, v_cache=vc, idx_cache=ic, seq_lens=lens, parents=_i32([[-1, 0, 1, 2]] * B), top_k=topk)
    shape = _lib.make_shape(B, N, cap, 32, HKV, D, D, 128, topk, 1)
    ws = torch.full((_lib.msa_workspace_bytes(shape, 5) // 4 + 4,), float("nan"), device="cuda")
    out, lse = torch.full_like(good["out"], float("nan")), torch.full_like(good["lse"], float("nan"))
    args = (shape, lens, None, 0, good["mask"], x["q"], kc, vc, good["k"], good["v"], good["sel"], out, lse, ws)
    _lib.msa_get_device_status()
    _lib.msa_debug_set_fault(2)
    try:
        _lib.msa_sparse_decode_tree(*args)
        with pytest.raises(_lib.MsaError) as e:
            _lib.msa_get_device_status()
        assert e.value.status == _lib.MSA_ERR_TIMEOUT
    finally:
        _lib.msa_debug_set_fault(0)
    assert not torch.isnan(out).any() and not torch.isnan(lse).any()
    assert not torch.equal(out, good["out"])
    _lib.msa_sparse_decode_tree(*args)
    _lib.msa_get_device_status()
    assert torch.equal(out, good["out"]) and torch.equal(lse, good["lse"])
