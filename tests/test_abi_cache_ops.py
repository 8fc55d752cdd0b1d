"""Host-side refusals of the rotary, 4-bit cache and eviction calls: every bad argument is
rejected before anything is launched (no GPU needed)."""
import ctypes

import pytest

from block_sparse_gqa_02_gb300 import _lib
from block_sparse_gqa_02_gb300._lib import (MSA_ERR_INVALID_ARG, MSA_ERR_UNSUPPORTED, MsaGatherTensor,
                                            MsaRope, MsaRopeTensor, make_shape)

FAKE = 1 << 30          # 16-byte aligned, never dereferenced
FAR = 1 << 44


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _rope(lib, desc=None, tensors=None, n=None, positions=None):
    d = MsaRope(2, 10, _lib.MSA_BF16, 0, 0, 0, 1.0)
    for k, v in (desc or {}).items():
        setattr(d, k, v)
    rows = tensors if tensors is not None else [{}]
    arr = (MsaRopeTensor * max(1, len(rows)))()
    for i, row in enumerate(rows):
        t = dict(x=FAKE + i * FAR, y=FAKE + i * FAR + FAR // 2, freqs=FAKE, n_heads=4, head_dim=64,
                 rotary_dim=64, head_major=0)
        t.update(row)
        arr[i] = MsaRopeTensor(**t)
    return lib.msa_rope(ctypes.byref(d), arr, len(rows) if n is None else n, positions, None)


@pytest.mark.parametrize("desc", [dict(batch=0), dict(seq=0), dict(dtype=5), dict(interleaved=2),
                                  dict(inverse=-1), dict(scale=float("nan")),
                                  dict(scale=float("inf"))])
def test_rope_desc(lib, desc):
    assert _rope(lib, desc) == MSA_ERR_INVALID_ARG and lib.msa_last_error()


@pytest.mark.parametrize("row,status", [
    (dict(x=None), MSA_ERR_INVALID_ARG), (dict(y=None), MSA_ERR_INVALID_ARG),
    (dict(freqs=None), MSA_ERR_INVALID_ARG), (dict(x=FAKE + 8), MSA_ERR_INVALID_ARG),
    (dict(n_heads=0), MSA_ERR_INVALID_ARG), (dict(head_major=2), MSA_ERR_INVALID_ARG),
    (dict(head_dim=72, rotary_dim=64), MSA_ERR_UNSUPPORTED),
    (dict(head_dim=2048), MSA_ERR_UNSUPPORTED), (dict(rotary_dim=0), MSA_ERR_UNSUPPORTED),
    (dict(rotary_dim=24), MSA_ERR_UNSUPPORTED), (dict(rotary_dim=80), MSA_ERR_UNSUPPORTED),
    (dict(x=FAKE, y=FAKE + 128), MSA_ERR_INVALID_ARG),           # partly over its own input
])
def test_rope_tensor(lib, row, status):
    assert _rope(lib, tensors=[row]) == status and lib.msa_last_error()


def test_rope_call(lib):
    assert _rope(lib, n=0) == MSA_ERR_INVALID_ARG
    assert _rope(lib, tensors=[{}] * 9) == MSA_ERR_INVALID_ARG
    assert _rope(lib, positions=FAKE + 4) == MSA_ERR_INVALID_ARG
    # one tensor's output over another's input, and two outputs in one place
    assert _rope(lib, tensors=[dict(x=FAKE, y=FAR), dict(x=FAR + 64, y=3 * FAR)]) == MSA_ERR_INVALID_ARG
    assert b"overlaps x" in lib.msa_last_error()
    assert _rope(lib, tensors=[dict(x=FAKE, y=FAR), dict(x=5 * FAR, y=FAR + 64)]) == MSA_ERR_INVALID_ARG
    assert b"overlaps y" in lib.msa_last_error()
    assert lib.msa_rope(None, (MsaRopeTensor * 1)(), 1, None, None) == MSA_ERR_INVALID_ARG


def _shape(**kw):
    d = dict(batch=2, seq_q=1, seq_k=1000, n_heads_q=16, n_heads_kv=4, head_dim=128, index_dim=128,
             block_size=128, top_k=4, q_tile=1, dtype="bf16")
    d.update(kw)
    return make_shape(**d)


def _packed_calls(lib, s, lens=FAKE, table=FAKE, n_phys=99, ptr=FAKE, mass=None):
    r = ctypes.byref(s)
    return [lib.msa_cache_pack(r, 3, None, lens, table, n_phys, ptr, FAKE, FAKE, None),
            lib.msa_cache_unpack(r, 3, None, lens, table, n_phys, ptr, FAKE, FAKE, None),
            lib.msa_sparse_decode_packed(r, lens, table, n_phys, ptr, FAKE, FAKE, FAKE, None, mass,
                                         None)]


@pytest.mark.parametrize("shape,status", [
    (dict(block_size=64), MSA_ERR_UNSUPPORTED), (dict(head_dim=96), MSA_ERR_UNSUPPORTED),
    (dict(batch=0), MSA_ERR_INVALID_ARG), (dict(seq_k=1 << 23), MSA_ERR_UNSUPPORTED),
    (dict(seq_q=1000, q_tile=64), MSA_ERR_INVALID_ARG),          # a prefill shape
])
def test_packed_shapes(lib, shape, status):
    assert _packed_calls(lib, _shape(**shape)) == [status] * 3


def test_packed_arguments(lib):
    s = _shape()
    bad = [MSA_ERR_INVALID_ARG] * 3
    assert _packed_calls(lib, s, ptr=None) == bad
    assert _packed_calls(lib, s, ptr=FAKE + 2) == bad
    assert _packed_calls(lib, s, lens=FAKE + 4) == bad
    assert _packed_calls(lib, s, n_phys=0) == bad
    # without a table the cache holds exactly batch * n_blocks blocks
    assert _packed_calls(lib, s, table=None, n_phys=15) == bad
    assert b"n_blocks" in lib.msa_last_error()
    r = ctypes.byref(s)
    assert lib.msa_cache_pack(r, 0, None, FAKE, FAKE, 9, FAKE, FAKE, FAKE, None) == MSA_ERR_INVALID_ARG
    assert lib.msa_cache_unpack(r, -1, None, FAKE, FAKE, 9, FAKE, FAKE, FAKE, None) == MSA_ERR_INVALID_ARG
    big = _shape(top_k=1025)
    assert lib.msa_sparse_decode_packed(ctypes.byref(big), FAKE, FAKE, 9, FAKE, FAKE, FAKE, FAKE, None,
                                        FAKE, None) == MSA_ERR_UNSUPPORTED
    wide = _shape(n_heads_q=4 * 65)
    assert lib.msa_sparse_decode_packed(ctypes.byref(wide), FAKE, FAKE, 9, FAKE, FAKE, FAKE, FAKE, None,
                                        None, None) == MSA_ERR_UNSUPPORTED


def test_decode_mass_arguments(lib):
    def call(s, lens=None, table=None, mass=FAKE, ws=FAKE, ws_bytes=1 << 30):
        return lib.msa_sparse_decode_mass(ctypes.byref(s), lens, table, 9, FAKE, FAKE, FAKE, FAKE,
                                          FAKE, None, mass, ws, ws_bytes, None)
    s = _shape()
    need = lib.msa_workspace_bytes(ctypes.byref(s), 4)
    assert need >= lib.msa_workspace_bytes(ctypes.byref(s), 1) + 2 * 16 * 4
    assert call(s, ws_bytes=need - 1) == MSA_ERR_INVALID_ARG and b"workspace" in lib.msa_last_error()
    assert call(s, ws=None) == MSA_ERR_INVALID_ARG
    assert call(s, mass=None) == MSA_ERR_INVALID_ARG
    assert call(s, lens=FAKE) == MSA_ERR_INVALID_ARG               # lengths without a table
    assert call(s, table=FAKE) == MSA_ERR_INVALID_ARG
    assert call(_shape(n_heads_q=8, n_heads_kv=2), lens=FAKE, table=FAKE) == MSA_ERR_UNSUPPORTED
    assert call(_shape(seq_q=1000, q_tile=64)) == MSA_ERR_INVALID_ARG
    assert call(_shape(n_heads_q=4 * 65)) == MSA_ERR_UNSUPPORTED
    assert lib.msa_workspace_bytes(ctypes.byref(_shape(seq_q=1000, q_tile=64)), 4) == 0
    for kw in (dict(), dict(dtype="f32"), dict(head_dim=64)):
        assert call(_shape(top_k=(1 << 20) + 1, **kw), ws_bytes=1 << 50) == MSA_ERR_UNSUPPORTED


def test_evict_arguments(lib):
    def call(s, keep=5, first=1, recent=2, mass=FAKE, table=FAKE, kept=FAKE, out=FAKE, t_out=FAKE):
        return lib.msa_cache_evict(ctypes.byref(s), keep, first, recent, FAKE, mass, table, kept, FAKE,
                                   out, t_out, None)
    s = _shape()
    assert call(s, keep=2) == MSA_ERR_INVALID_ARG
    assert call(s, first=-1) == MSA_ERR_INVALID_ARG
    assert call(s, recent=0) == MSA_ERR_INVALID_ARG
    assert call(s, first=1 << 30, recent=(1 << 30) + (1 << 29), keep=1 << 30) == MSA_ERR_INVALID_ARG
    assert call(s, mass=None) == MSA_ERR_INVALID_ARG
    assert call(s, kept=FAKE + 4) == MSA_ERR_INVALID_ARG
    assert call(s, t_out=None) == MSA_ERR_INVALID_ARG
    assert call(s, table=None) == MSA_ERR_INVALID_ARG
    assert call(s, out=FAKE + 16) == MSA_ERR_INVALID_ARG and b"mass_out" in lib.msa_last_error()
    assert call(s, t_out=FAKE - 16) == MSA_ERR_INVALID_ARG and b"table_out" in lib.msa_last_error()
    assert call(_shape(seq_q=1000, q_tile=64)) == MSA_ERR_INVALID_ARG
    assert call(_shape(seq_k=(1 << 22) + 1)) == MSA_ERR_UNSUPPORTED  # 32769 blocks
    assert call(s, keep=(1 << 20) + 1) == MSA_ERR_UNSUPPORTED


@pytest.mark.parametrize("row,status", [
    (dict(src=None), MSA_ERR_INVALID_ARG), (dict(dst=FAKE + FAR + 8), MSA_ERR_INVALID_ARG),
    (dict(n_heads=0), MSA_ERR_INVALID_ARG), (dict(src_rows=0), MSA_ERR_INVALID_ARG),
    (dict(row_bytes=24), MSA_ERR_UNSUPPORTED), (dict(row_bytes=0), MSA_ERR_UNSUPPORTED),
    (dict(row_bytes=1 << 17), MSA_ERR_UNSUPPORTED), (dict(dst=FAKE + 256), MSA_ERR_INVALID_ARG),
])
def test_gather_tensor(lib, row, status):
    t = dict(src=FAKE, dst=FAKE + FAR, src_rows=1000, dst_rows=500, n_heads=4, row_bytes=256)
    t.update(row)
    arr = (MsaGatherTensor * 1)(MsaGatherTensor(**t))
    assert lib.msa_cache_gather(2, arr, 1, FAKE, 4, 128, None) == status and lib.msa_last_error()


def test_gather_call(lib):
    arr = (MsaGatherTensor * 1)(MsaGatherTensor(FAKE, FAKE + FAR, 1000, 500, 4, 256))
    for batch, n, kept, keep, block in ((0, 1, FAKE, 4, 128), (2, 0, FAKE, 4, 128),
                                        (2, 9, FAKE, 4, 128), (2, 1, None, 4, 128),
                                        (2, 1, FAKE, 0, 128), (2, 1, FAKE, 4, 0)):
        assert lib.msa_cache_gather(batch, arr, n, kept, keep, block, None) == MSA_ERR_INVALID_ARG
    assert lib.msa_cache_gather(2, None, 1, FAKE, 4, 128, None) == MSA_ERR_INVALID_ARG


def test_binding_refuses_tensors_off_the_device(lib):
    import torch
    s = _shape()
    q = torch.zeros(2, 1, 16, 128, dtype=torch.bfloat16)             # on the host
    with pytest.raises(ValueError, match="current CUDA device"):
        _lib.msa_sparse_decode_packed(s, None, None, 16, q, FAKE, FAKE, FAKE, stream=0)


def test_api_refuses_arrays_of_another_stride():
    """Arrays with an entry per block are indexed by the call's number of blocks: one with room
    for more would be read in the wrong rows."""
    import torch
    from block_sparse_gqa_02_gb300 import api
    B, H, L, d, bf = 2, 4, 1000, 128, torch.bfloat16
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)  # noqa: E731
    q, k, iq, ik = z(B, 1, 16, d), z(B, H, L, d), z(B, 1, H, d), z(B, L, d)
    lens, mass, table = z(B, dt=torch.int32), z(B, H, 8, dt=torch.float32), z(B, 8, dt=torch.int32)
    cache, pool = z(20, H, 160 * d, dt=torch.uint8), z(20, 128, d)
    wide, long = z(B, H, 9, dt=torch.float32), z(B, 9, dt=torch.int32)
    with pytest.raises(ValueError, match="mass is"):
        api.decode(q, k, k, iq, ik, mass=wide)
    with pytest.raises(ValueError, match="mass is"):
        api.evict(k, k, ik, wide, 4)
    with pytest.raises(ValueError, match="mass is"):
        api.evict_paged(lens, wide, table, L, 4)
    with pytest.raises(ValueError, match="block_table is"):
        api.evict_paged(lens, mass, long, L, 4)
    new = z(B, H, 1, d)
    with pytest.raises(ValueError, match="mass is"):
        api.decode_packed(q, new, new, cache, iq, pool, lens, table, L, mass=wide)
    with pytest.raises(ValueError, match="block_table is"):
        api.decode_packed(q, new, new, cache, iq, pool, lens, long, L)
    with pytest.raises(ValueError, match="idx_k_pool is"):
        api.decode_packed(q, new, new, cache, iq, pool[:19], lens, table, L)
