"""Lists of accepted tokens that name a token which the tree does not have: its rows may hold anything
and must not reach the caches."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api
from tests.canary import guarded_like
from tests.test_gpu_packed import _i32
from tests.test_gpu_tree_step import PARENTS, _drafts, _state
from tests.tree_cases import Tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("paged", [False, True])
def test_absent_tokens_are_not_committed(paged):
    s = _state(paged)
    s["lens"][0] = s["cap"] - 2                             # tokens 0, 1, 2, 5, 6 fit, 3 and 4 (depth 2) do not
    x = _drafts(3, 7, 90)
    absent = [(0, 3), (0, 4), (1, 6)]
    for b, i in absent:
        x["k"][b, :, i] = x["v"][b, :, i] = float("nan")
        x["idx_k"][b, i] = float("nan")
    step = api.decode_tree(x["q"], x["k"], x["v"], x["idx_q"], x["idx_k"], s["kc"], s["vc"], s["ic"], s["lens"],
                           _i32(PARENTS), s["table"], s["cap"], top_k=4, rope=s["rope"])
    assert (step["mask"] == 0).nonzero().tolist() == [list(p) for p in absent]
    caches = ("kc", "vc", "ic")

    def commit(accepted):
        t = {k: s[k].clone() for k in caches + ("lens",)}
        api.commit_tree(step, _i32(accepted), t["kc"], t["vc"], t["ic"], t["lens"], s["table"], s["cap"])
        _lib.msa_get_device_status()
        return t
    # the same as lists that end before the absent token
    got = commit([[3, 0, 1], [1, 6, 2], [0, 1, 2]])
    want = commit([[-1, 0, 1], [1, -1, 2], [0, 1, 2]])
    assert got["lens"].tolist() == [s["cap"] - 2, 250 + 1, 3]
    for k in caches + ("lens",):
        assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), k
    assert not torch.isnan(got["kc"]).any() and not torch.isnan(got["vc"]).any()


@pytest.mark.parametrize("n", [1, 33, 64])
@pytest.mark.parametrize("dtype,paged", [("bf16", True), ("f32", False)])
def test_lists_end_at_absent_tokens(n, dtype, paged):
    """Random lists over trees with absent tokens (NaN rows), with the masks and, where the list is cut
    by hand, without: the same bytes and lengths."""
    t = Tree(lens=[0, 100, 290, 300, 255, 260], n=n, cap=300, paged=paged, kind="bad", hkv=2, group=1, dim=64, dtype=dtype,
             seed=n)
    s, d = t.shape, t.dev
    rng = np.random.default_rng(n)
    acc = rng.integers(0, n, (6, min(64, n + 3)))
    acc[rng.random(acc.shape) < 0.02] = -1
    cut = acc.copy()
    for b in range(6):
        for i, a in enumerate(acc[b]):
            if a >= 0 and not t.paths[b][a]:
                cut[b, i:] = -1
                break
    if n > 1:
        assert (cut != acc).any()

    def commit(accepted, mask):
        dst = {k: guarded_like(d[k].shape, d[k].dtype) for k in ("k", "v", "ik")}
        for k, g in dst.items():
            g.tensor.copy_(d[k])
        new = torch.full_like(t.seq_lens, -5)
        tensors = _lib.make_commit_tensors([(d["kd"], dst["k"].tensor), (d["vd"], dst["v"].tensor)], [(d["ikd"], dst["ik"].tensor)])
        _lib.msa_tree_commit(s, t.seq_lens, t.table, t.n_phys, _i32(accepted.tolist()), tensors, new, mask=mask)
        _lib.msa_get_device_status()
        for k, g in dst.items():
            g.check(k)
        return [g.tensor.view(torch.uint8) for g in dst.values()] + [new]
    for got, want in zip(commit(acc, t.mask), commit(cut, None)):
        assert torch.equal(got, want)
