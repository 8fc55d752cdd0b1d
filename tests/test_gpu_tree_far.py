"""Drafted tokens at the far end of the longest caches the calls take: positions up to 2^31 - 2, where a
length and a depth add up to more than 32 bits hold."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib
from oracle import tree_ops
from tests.canary import guarded_like
from tests.test_gpu_packed import _i32

pytestmark = pytest.mark.gpu

CAP, BLOCK = 2 ** 31 - 1, 1 << 16


@pytest.mark.parametrize("n", [1, 5, 64])
def test_mask_and_selection(n):
    lens = [CAP, CAP - 1, CAP - 3, CAP - 64, CAP - 70, 0]
    parents = np.array([[i - 1 for i in range(n)]] * len(lens))
    shape = _lib.make_shape(len(lens), n, CAP, 1, 1, 64, 64, BLOCK, 3, 1)
    mask, pos = guarded_like((len(lens), n), torch.int64), guarded_like((len(lens), n), torch.int32)
    _lib.msa_tree_mask(shape, _i32(lens), _i32(parents.tolist()), mask.tensor, pos.tensor)
    paths = [tree_ops.paths(parents[b], lens[b], CAP) for b in range(len(lens))]
    at = [[lens[b] + len(p) - 1 if p else -1 for p in paths[b]] for b in range(len(lens))]
    assert [[x % (1 << 64) for x in row] for row in mask.tensor.tolist()] == [[tree_ops.word(p) for p in row] for row in paths]
    assert pos.tensor.tolist() == at
    x = np.random.default_rng(n).standard_normal((len(lens), 1, n, shape.n_blocks)).astype(np.float32)
    # words of every token, as a caller may pass them: those past the capacity count as absent
    words = [tree_ops.word(range(i + 1)) for i in range(n)]
    every = torch.tensor([[w - (1 << 64) if w >> 63 else w for w in words]] * len(lens)).cuda()
    for m in (mask.tensor, every):
        sel = guarded_like((len(lens), 1, n, 3), torch.int32)
        _lib.msa_block_topk_tree(shape, _i32(lens), m, torch.tensor(x).cuda(), sel.tensor)
        _lib.msa_get_device_status()
        for b in range(len(lens)):
            for i in range(n):
                assert sel.tensor[b, 0, i].tolist() == tree_ops.select(x[b, 0, i], at[b][i], BLOCK, 3)
        sel.check("sel")
    mask.check("mask")
    pos.check("positions")


@pytest.mark.parametrize("masked", [False, True])
def test_commit(masked):
    B, n, d = 3, 8, 16
    lens = [CAP - 3, CAP, CAP - 100]
    shape = _lib.make_shape(B, n, CAP, 1, 1, 64, 64, BLOCK, 1, 1)
    src = torch.randn(B, n, d, device="cuda").bfloat16()
    pool = guarded_like((3, BLOCK, d), torch.bfloat16, fill=2.0)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].repeat(1, shape.n_blocks).contiguous()
    acc = _i32([[7, 6, 5, 4, 3, 2]] * B)
    mask = torch.tensor([[1 << i for i in range(n)]] * B).cuda() if masked else None     # all children of the last cached token
    lens_t, new = _i32(lens), torch.zeros(B, dtype=torch.int32, device="cuda")
    _lib.msa_tree_commit(shape, lens_t, table, 3, acc, _lib.make_commit_tensors([(src, pool.tensor)]), new, mask=mask)
    _lib.msa_get_device_status()
    assert new.tolist() == [CAP, CAP, CAP - 94]
    want = torch.full_like(pool.tensor, 2.0)
    for b, count in enumerate([3, 0, 6]):
        for i in range(count):
            want[b, (lens[b] + i) % BLOCK] = src[b, 7 - i]
    assert torch.equal(pool.tensor, want)
    pool.check()
