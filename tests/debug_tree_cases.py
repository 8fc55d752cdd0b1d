"""Cases of the calls over drafted tokens for the debug library, run by
tests/test_gpu_debug_tree.py in a process of its own (MSA_LIBRARY_VARIANT=debug): whole steps stay
clean, and a selection entry, table entry or length out of range is reported."""
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib
from tests.test_gpu_tree_step import PARENTS, _drafts, _run, _state
from tests.tree_cases import Tree
from tests.test_gpu_packed import _i32

pytestmark = pytest.mark.gpu


def _status():
    try:
        _lib.msa_get_device_status()
        return _lib.MSA_OK
    except _lib.MsaError as e:
        return e.status


def test_variant():
    assert _lib.load().msa_debug_build() == 1


@pytest.mark.parametrize("paged", [False, True])
def test_whole_steps_stay_clean(paged):
    s = _state(paged)
    s["parents"] = _i32(PARENTS)
    for i in range(3):
        _run(s, _drafts(3, 7, i), _i32([[0, 1, -1], [1, 2, -1], [0, 1, 2]]))
        assert _status() == _lib.MSA_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_indices(dtype):
    t = Tree(lens=[700, 300], n=9, cap=800, paged=True, topk=4, dtype=dtype, kind="chain")
    s, d = t.shape, t.dev
    out = torch.empty_like(d["q"])
    ws = torch.empty(_lib.msa_workspace_bytes(s, 5) // 4 + 4, device="cuda")

    def attend(sel, table=t.table, lens=t.seq_lens):
        _lib.msa_sparse_decode_tree(s, lens, table, t.n_phys, t.mask, d["q"], d["k"], d["v"], d["kd"], d["vd"], sel, out, None, ws)
        return _status()
    assert attend(d["sel"]) == _lib.MSA_OK
    good = out.clone()
    bad = d["sel"].clone()
    bad[1, :, 2, -1] = 3                                    # past the token's own block (300 + 2) // 128
    assert attend(bad) == _lib.MSA_ERR_BOUNDS
    assert attend(d["sel"]) == _lib.MSA_OK and torch.equal(out, good)
    wrong = t.table.clone()
    wrong[0, 1] = t.n_phys + 5
    scores = torch.empty(s.batch, s.n_heads_kv, t.n, t.nB, device="cuda")
    _lib.msa_index_scores_tree(s, t.seq_lens, wrong, t.n_phys, t.mask, d["iq"], d["ik"], d["ikd"], scores, packed=True)
    assert _status() == _lib.MSA_ERR_BOUNDS
    _lib.msa_index_scores_tree(s, _i32([9000, 300]), t.table, t.n_phys, t.mask, d["iq"], d["ik"], d["ikd"], scores, packed=True)
    assert _status() == _lib.MSA_ERR_BOUNDS
