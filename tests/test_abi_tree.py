"""Host-side refusals of the calls over drafted tokens: every bad argument is rejected before
anything is launched (no GPU needed)."""
import ctypes

import pytest

from block_sparse_gqa_02_gb300 import _lib
from block_sparse_gqa_02_gb300._lib import (MSA_ERR_INVALID_ARG, MSA_ERR_UNSUPPORTED, MsaCommitTensor,
                                            make_shape)

FAKE = 1 << 30          # 16-byte aligned, never dereferenced
FAR = 1 << 44


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _shape(**kw):
    d = dict(batch=2, seq_q=7, seq_k=1000, n_heads_q=16, n_heads_kv=4, head_dim=128, index_dim=128,
             block_size=128, top_k=4, q_tile=1, dtype="bf16")
    d.update(kw)
    return make_shape(**d)


def _commit(lib, s, lens=FAKE, table=None, n_phys=16, accepted=FAKE + (1 << 20), n=3, rows=({},), new=FAKE, n_rows=None):
    arr = (MsaCommitTensor * max(1, len(rows)))()
    for i, row in enumerate(rows):
        t = dict(src=FAR * (2 * i + 1), dst=FAR * (2 * i + 2), n_heads=4, row_bytes=256, packed=0)
        t.update(row)
        arr[i] = MsaCommitTensor(**t)
    return lib.msa_tree_commit(ctypes.byref(s), lens, table, n_phys, accepted, n, arr, len(rows) if n_rows is None else n_rows,
                               new, None)


def _calls(lib, s, lens=FAKE, mask=FAKE, table=FAKE, n_phys=99, ptr=FAKE, packed=0):
    """mask, scores, selection, attention."""
    r = ctypes.byref(s)
    return [lib.msa_tree_mask(r, lens, ptr, mask, None, None),
            lib.msa_index_scores_tree(r, lens, table, n_phys, mask, ptr, FAKE, FAKE, packed, FAKE, None),
            lib.msa_block_topk_tree(r, lens, mask, ptr, FAKE, None),
            lib.msa_sparse_decode_tree(r, lens, table, n_phys, mask, ptr, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE,
                                       1 << 40, None)]


@pytest.mark.parametrize("shape,status", [
    (dict(seq_q=65), MSA_ERR_UNSUPPORTED), (dict(seq_q=0), MSA_ERR_INVALID_ARG), (dict(q_tile=7), MSA_ERR_INVALID_ARG),
    (dict(batch=0), MSA_ERR_INVALID_ARG), (dict(head_dim=96), MSA_ERR_UNSUPPORTED), (dict(seq_k=1 << 23), MSA_ERR_UNSUPPORTED),
    (dict(n_heads_q=17), MSA_ERR_INVALID_ARG), (dict(index_dim=32), MSA_ERR_UNSUPPORTED),
    (dict(sm_scale=float("nan")), MSA_ERR_INVALID_ARG)])
def test_shapes(lib, shape, status):
    s = _shape(**shape)
    assert _calls(lib, s) == [status] * 4
    assert _commit(lib, s) == status and lib.msa_last_error()
    assert lib.msa_workspace_bytes(ctypes.byref(s), 5) == 0


def test_arguments(lib):
    s = _shape()
    bad = [MSA_ERR_INVALID_ARG] * 4
    for kw in (dict(lens=None), dict(lens=FAKE + 4), dict(mask=None), dict(mask=FAKE + 8), dict(ptr=None), dict(ptr=FAKE + 2)):
        assert _calls(lib, s, **kw) == bad, kw
    r = ctypes.byref(s)
    for kw in (dict(table=FAKE + 4), dict(n_phys=0)):
        got = _calls(lib, s, **kw)
        assert got[1] == got[3] == MSA_ERR_INVALID_ARG, kw
    # 8-bit keys without a table: one record for every block
    args = FAKE, None, 15, FAKE, FAKE, FAKE, FAKE, 1, FAKE, None
    assert lib.msa_index_scores_tree(r, *args) == MSA_ERR_INVALID_ARG and b"n_blocks" in lib.msa_last_error()
    assert lib.msa_index_scores_tree(r, FAKE, None, 16, FAKE, FAKE, FAKE, FAKE, 2, FAKE, None) == MSA_ERR_INVALID_ARG
    odd = _shape(block_size=64)
    assert lib.msa_index_scores_tree(ctypes.byref(odd), FAKE, FAKE, 9, FAKE, FAKE, FAKE, FAKE, 1, FAKE, None) == MSA_ERR_UNSUPPORTED
    many = _shape(n_heads_kv=65, n_heads_q=65)
    assert lib.msa_index_scores_tree(ctypes.byref(many), FAKE, FAKE, 9, FAKE, FAKE, FAKE, FAKE, 0, FAKE, None) == MSA_ERR_UNSUPPORTED
    decode = lambda s, ws: lib.msa_sparse_decode_tree(ctypes.byref(s), FAKE, FAKE, 9, FAKE, *[FAKE] * 7, None, FAKE, ws, None)  # noqa: E731
    need = lib.msa_workspace_bytes(r, 5)
    assert need > 0 and decode(s, need - 1) == MSA_ERR_INVALID_ARG and b"workspace" in lib.msa_last_error()
    assert decode(_shape(n_heads_q=4 * 65), 1 << 40) == MSA_ERR_UNSUPPORTED
    assert decode(_shape(top_k=(1 << 20) + 1), 1 << 40) == MSA_ERR_UNSUPPORTED


def test_index_cache(lib):
    def both(s, n=3, lens=FAKE, starts=None, table=FAKE, n_phys=99, x=FAKE, cache=FAKE):
        r = ctypes.byref(s)
        return [lib.msa_index_pack(r, n, starts, lens, table, n_phys, x, cache, None),
                lib.msa_index_unpack(r, n, starts, lens, table, n_phys, cache, x, None)]
    s = _shape()
    bad = [MSA_ERR_INVALID_ARG] * 2
    for kw in (dict(n=0), dict(n=-4), dict(lens=FAKE + 4), dict(starts=FAKE + 8), dict(table=FAKE + 2), dict(n_phys=0),
               dict(table=None, n_phys=15), dict(x=None), dict(cache=None), dict(x=FAKE + 1), dict(cache=FAKE + 8)):
        assert both(s, **kw) == bad, kw
    assert both(_shape(block_size=64)) == [MSA_ERR_UNSUPPORTED] * 2
    assert both(_shape(index_dim=96)) == [MSA_ERR_UNSUPPORTED] * 2
    assert lib.msa_index_pack(None, 1, None, None, None, 16, FAKE, FAKE, None) == MSA_ERR_INVALID_ARG


def test_commit(lib):
    s = _shape()
    for kw in (dict(lens=None), dict(accepted=None), dict(accepted=FAKE + 4), dict(n=0), dict(n=65), dict(new=None), dict(rows=({},) * 9),
               dict(n_rows=0), dict(n_phys=15), dict(table=FAKE + 2), dict(table=FAKE + FAR, n_phys=0), dict(rows=(dict(src=None),)),
               dict(rows=(dict(dst=FAR + 8),)), dict(rows=(dict(n_heads=0),)), dict(rows=(dict(row_bytes=0),)), dict(rows=(dict(packed=2),))):
        assert _commit(lib, s, **kw) == MSA_ERR_INVALID_ARG, kw
        assert lib.msa_last_error()
    for row in (dict(row_bytes=24), dict(n_heads=1 << 20, row_bytes=4096), dict(packed=1), dict(packed=1, n_heads=1, row_bytes=96)):
        assert _commit(lib, s, rows=(row,)) == MSA_ERR_UNSUPPORTED, row
    assert _commit(lib, _shape(block_size=64, seq_k=1000), n_phys=32, rows=(dict(packed=1, n_heads=1, row_bytes=128),)) == MSA_ERR_UNSUPPORTED
    # destinations clear of everything: of a source, of one another, of the list, of the lengths
    size = 2 * 4 * 1000 * 256
    for rows in ((dict(src=FAR, dst=FAR + 256),), (dict(), dict(dst=2 * FAR + size - 16)), (dict(dst=FAKE - size + 16),),
                 (dict(dst=FAKE + (1 << 20) - 16),)):
        assert _commit(lib, s, rows=rows) == MSA_ERR_INVALID_ARG and b"overlaps" in lib.msa_last_error(), rows
    assert _commit(lib, s, new=FAKE + (1 << 20)) == MSA_ERR_INVALID_ARG           # over the list
    # a length that is another sequence's (new_lens over seq_lens, but not in its place)
    assert _commit(lib, _shape(batch=8), n_phys=64, new=FAKE + 16) == MSA_ERR_INVALID_ARG
