"""Attention weights of the 4-bit decode in groups of more than 16 heads, which it takes sixteen at
a time."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api
from tests.test_gpu_packed import DT, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [1, 16, 17, 40, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_one_addition_a_call(heads, dtype, d):
    """A block's entry gets one fp32 addition however many heads the group has: the weights of a
    call on zeros, added to what was there and rounded once."""
    B, Hkv, L, topk = 2, 2, 4000, 20
    shape = _lib.make_shape(B, 1, L, heads * Hkv, Hkv, d, 128, 128, topk, 1, dtype)
    q, k, v = (_rows(s, DT[dtype], i) for i, s in enumerate(((B, 1, heads * Hkv, d), (B, Hkv, L, d), (B, Hkv, L, d))))
    cache = api.alloc_packed_cache(B * 32, Hkv, d)
    _lib.msa_cache_pack(shape, L, None, None, None, B * 32, k, v, cache)
    rng = np.random.default_rng(heads)
    sel = torch.from_numpy(np.stack([rng.permutation(32)[:topk] for _ in range(B * Hkv)]).astype(np.int32))
    sel = sel.view(B, Hkv, 1, topk).cuda()
    out = torch.empty_like(q)

    def weights(before):
        m = before.clone()
        _lib.msa_sparse_decode_packed(shape, None, None, B * 32, q, cache, sel, out, None, m)
        _lib.msa_get_device_status()
        return m
    zero = torch.zeros((B, Hkv, 32), device="cuda")
    w = weights(zero)
    assert abs(float(w.double().sum()) - B * Hkv * heads) <= 1e-3 * B * Hkv * heads
    for base in (1.0, 1000.0, 2.0 ** 20):
        before = base * (1 + torch.rand((B, Hkv, 32), generator=torch.Generator("cuda").manual_seed(1), device="cuda"))
        assert torch.equal(weights(before), before + w)
