"""api.evict: K, V and index keys are cut alike, so they have the same rows."""
import pytest
import torch

from block_sparse_gqa_02_gb300 import api

BF = torch.bfloat16


@pytest.mark.parametrize("name,shape", [
    ("v_cache", (2, 4, 900, 128)), ("v_cache", (2, 2, 1000, 128)), ("v_cache", (1, 4, 1000, 128)),
    ("idx_k", (2, 900, 128)), ("idx_k", (1, 1000, 128)), ("idx_k", (2, 1, 1000, 128)), ("idx_k", (2, 1000))])
def test_other_rows_are_refused(name, shape):
    """A shorter cache would leave the rows that it lacks as the allocation found them."""
    t = dict(k_cache=torch.zeros((2, 4, 1000, 128), dtype=BF), v_cache=torch.zeros((2, 4, 1000, 128), dtype=BF),
             idx_k=torch.zeros((2, 1000, 128), dtype=BF), mass=torch.zeros((2, 4, 8)))
    t[name] = torch.zeros(shape, dtype=BF)
    with pytest.raises(ValueError, match=f"{name} is"):
        api.evict(**t, keep=4)


@pytest.mark.gpu
def test_rows_of_other_widths():
    """Index keys of their own dims, and V of another head size than K."""
    g = torch.Generator("cuda").manual_seed(1)
    z = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    k, v, ik = z(2, 4, 1000, 128), z(2, 4, 1000, 64), z(2, 1000, 32)
    cut = api.evict(k, v, ik, torch.rand((2, 4, 8), generator=g, device="cuda"), keep=4)
    for b in range(2):
        rows = [j for x in cut["kept"][b].tolist() for j in range(128 * x, min(1000, 128 * x + 128))]
        assert torch.equal(cut["k"][b], k[b, :, rows]) and torch.equal(cut["v"][b], v[b, :, rows])
        assert torch.equal(cut["idx_k"][b], ik[b, rows])
