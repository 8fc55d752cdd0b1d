"""Cases of the cache calls for the debug library, run by tests/test_gpu_debug_cache.py in a
process of its own (MSA_LIBRARY_VARIANT=debug): clean inputs stay clean, and a selection entry,
table entry or length out of range is reported, with the output of the call without it."""
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api
from tests.test_gpu_packed import DT, _filled, _i32, _rows, _shape

pytestmark = pytest.mark.gpu


def _status():
    try:
        _lib.msa_get_device_status()
        return _lib.MSA_OK
    except _lib.MsaError as e:
        return e.status


def _decode(lens, cap, cache, table, P, sel, mass):
    shape = _shape(len(lens), cap, 16, 4, 128, sel.shape[-1])
    q = _rows((len(lens), 1, 16, 128), DT["bf16"], 1)
    out = torch.empty_like(q)
    _lib.msa_sparse_decode_packed(shape, _i32(lens), table, P, q, cache, sel, out, None, mass)
    return out


def test_variant():
    assert _lib.load().msa_debug_build() == 1


def test_packed_indices():
    lens, cap = [700, 300], 700
    cache, table, P, _, _ = _filled(2, cap, 4, 128, lens, "bf16", True, 4)
    assert _status() == _lib.MSA_OK
    sel = _i32([[[[0, 3, 5]]] * 4, [[[0, 2, -1]]] * 4]).contiguous()
    mass = torch.zeros((2, 4, 6), device="cuda")
    good = _decode(lens, cap, cache, table, P, sel, mass)
    assert _status() == _lib.MSA_OK
    bad = sel.clone()
    bad[1, :, 0, 2] = 3                                    # past the second sequence's blocks
    assert torch.equal(_decode(lens, cap, cache, table, P, bad, mass), good)
    assert _status() == _lib.MSA_ERR_BOUNDS
    assert torch.equal(_decode([700, 300], cap, cache, table, P, sel, mass), good)
    assert _status() == _lib.MSA_OK                        # the report cleared the word
    wrong = table.clone()
    wrong[0, 1] = P + 7                                    # a block that no entry selects
    assert torch.equal(_decode(lens, cap, cache, wrong, P, sel, mass), good)
    assert _status() == _lib.MSA_ERR_BOUNDS
    _decode([9000, 300], cap, cache, table, P, sel, mass)
    assert _status() == _lib.MSA_ERR_BOUNDS


def test_other_calls_stay_clean():
    lens = _i32([700, 300])
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6).contiguous()
    api.evict_paged(lens, torch.rand((2, 4, 6), device="cuda"), table, 700, 4)
    freqs, _ = api.rope_freqs(64, device="cuda")
    api.rope([(_rows((2, 3, 4, 64), DT["bf16"], 1), freqs, False)])
    q, k, v = (_rows(s, DT["bf16"], i) for i, s in enumerate(
        ((2, 1, 16, 128), (2, 4, 700, 128), (2, 4, 700, 128))))
    iq, ik = _rows((2, 1, 4, 128), DT["bf16"], 5), _rows((2, 700, 128), DT["bf16"], 6)
    api.decode(q, k, v, iq, ik, top_k=3, mass=torch.zeros((2, 4, 6), device="cuda"))
    assert _status() == _lib.MSA_OK
