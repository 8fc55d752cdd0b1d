"""Block top-k of rows around the sizes where its shared memory needs an opt-in."""
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("blocks", [10240, 10241, 11900, 12288, 12289])
def test_topk_just_below_48_kib(blocks):
    """The candidates and the kernel's own arrays together pass the default limit of 48 KiB before
    the candidates alone do."""
    shape = _lib.make_shape(1, 1, 128 * blocks, 4, 4, 128, 128, 128, 64, 1)
    g = torch.Generator("cuda").manual_seed(blocks)
    scores = torch.rand((1, 4, 1, blocks), generator=g, device="cuda")
    sel = torch.empty((1, 4, 1, 64), dtype=torch.int32, device="cuda")
    _lib.msa_block_topk(shape, scores, sel)
    _lib.msa_get_device_status()
    # the 63 best of the blocks before the query's, and that
    best = scores[..., :-1].topk(63, dim=-1).indices.sort(-1).values
    assert torch.equal(sel[..., :63].long(), best) and bool((sel[..., 63] == blocks - 1).all())
