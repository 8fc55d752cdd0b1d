"""Host-side refusals of the commit with the tree's masks (no GPU needed)."""
import ctypes

import pytest

from block_sparse_gqa_02_gb300 import _lib
from block_sparse_gqa_02_gb300._lib import MSA_ERR_INVALID_ARG, MSA_ERR_UNSUPPORTED, MsaCommitTensor, make_shape

FAKE = 1 << 30          # 16-byte aligned, never dereferenced
FAR = 1 << 44


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _commit(lib, mask=FAKE + (1 << 21), new=FAKE, n=3, dst=2 * FAR, seq_q=7):
    s = make_shape(2, seq_q, 1000, 16, 4, 128, 128, 128, 4, 1, "bf16")
    arr = (MsaCommitTensor * 1)(MsaCommitTensor(FAR, dst, 4, 256, 0))
    return lib.msa_tree_commit_masked(ctypes.byref(s), FAKE, None, 16, mask, FAKE + (1 << 20), n, arr, 1, new, None)


def test_masks(lib):
    for kw in (dict(mask=FAKE + (1 << 21) + 8), dict(n=0), dict(n=65), dict(dst=None), dict(seq_q=0)):
        assert _commit(lib, **kw) == MSA_ERR_INVALID_ARG and lib.msa_last_error(), kw
    assert _commit(lib, seq_q=65) == MSA_ERR_UNSUPPORTED
    # an output over the masks: the lengths, the cache's first and last bytes
    size = 2 * 4 * 1000 * 256
    for kw in (dict(new=FAKE + (1 << 21)), dict(new=FAKE + (1 << 21) + 96), dict(mask=2 * FAR), dict(mask=2 * FAR + size - 16),
               dict(mask=2 * FAR - 96)):
        assert _commit(lib, **kw) == MSA_ERR_INVALID_ARG and b"overlaps mask" in lib.msa_last_error(), kw
