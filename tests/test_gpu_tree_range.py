"""Index scores of drafted tokens whose queries' dims differ widely in size, against fp64: a large dim
must not take digits from the others, whatever form the keys are held in."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib
from oracle import tree_ops
from tests.canary import guarded_like
from tests.tree_cases import Tree

pytestmark = pytest.mark.gpu

LARGE = [5, 77, 40]                     # dims of the large values; the keys are zero there


def _with_queries(t, make):
    """The tree's case with other queries and keys: make(queries), and keys without the large dims."""
    s = t.shape
    large = [j for j in LARGE if j < s.index_dim]
    t.iq = make(t.iq.float(), large).to(t.dt)
    t.ik[..., large] = 0
    t.ikd[..., large] = 0
    there = torch.tensor([[bool(p) for p in row] for row in t.paths])
    iq = t.iq.clone()
    iq[~there] = float("nan")
    t.dev["iq"] = iq.cuda()
    if t.packed:
        t.dev["ik"] = t._pack(t.ik, 128).cuda()
        codes, exps, t.ikd64 = tree_ops.quantise(t.ikd.float().numpy())
        rec, n, d = t.dev["ikd"], t.n, s.index_dim
        rec[:, :n * d] = torch.tensor(codes).reshape(s.batch, -1).cuda()
        rec[:, 128 * d:128 * d + n] = torch.tensor(exps).cuda()
        t.ik64 = tree_ops.quantise(t.ik.float().numpy())[2]
    else:
        t.dev["ik"], t.dev["ikd"] = t._store(t.ik, s.block_size, float("nan")).cuda(), t.ikd.cuda()
        t.ikd64, t.ik64 = t.ikd.double().numpy(), t.ik.double().numpy()


def _bound(t):
    """Per (b, h, token): the products are summed in fp32 (each of up to three parts of a query's dim
    with its key; an addition is off by 2^-24 of the sum's magnitude, twice that where it truncates;
    parts of 3 bits add up to 1 + 2^-3 + 2^-6 of the dim), and the tensor-core form with 8-bit keys
    may miss 2^-31 of the query's largest dim in the dims below 2^-23 of it."""
    s = t.shape
    d = s.index_dim
    split = t.packed and t.dt == torch.bfloat16 and d == 128
    terms, spread = (3 * d, 1.15) if split else (d, 1.0)
    out = np.zeros((s.batch, s.n_heads_kv, t.n, 1))
    for b, length in enumerate(t.lens):
        k = np.abs(np.concatenate([t.ik64[b][:length], t.ikd64[b]]))
        q = np.abs(t.iq[b].double().numpy())                              # [N, H, d]
        top = q.max(-1, keepdims=True)
        lost = np.where(q < 2.0 ** -23 * top, 2.0 ** -31 * top, 0.0) if split else np.zeros_like(q)
        e = 2 * (terms + 2) * 2.0 ** -24 * spread * (q @ k.T).max(-1) + (lost @ k.T).max(-1)
        out[b, :, :, 0] = (e * d ** -0.5 * 1.001).T
    return out


def _outliers(ratio):
    def make(q, large):
        q[..., large] *= ratio
        return q
    return make


def _spread(q, large):
    g = torch.Generator().manual_seed(9)
    return q * (4 * torch.randn(q.shape, generator=g)).exp()


QUERIES = {"plain": _outliers(1.0), "300": _outliers(300.0), "1e4": _outliers(1e4), "1e6": _outliers(1e6),
           "spread": _spread, "tiny": lambda q, large: _outliers(1e4)(q * 2.0 ** -60, large),
           "huge": lambda q, large: _outliers(1e4)(q * 2.0 ** 60, large)}


@pytest.mark.parametrize("queries", list(QUERIES))
@pytest.mark.parametrize("c", [
    dict(lens=[1000, 129, 0], n=5, cap=1100), dict(lens=[1500, 250], n=32, cap=1600, paged=True, kind="bad"),
    dict(lens=[700, 126], n=64, cap=800, kind="chain"), dict(lens=[600], n=1, cap=601, hkv=1),
    dict(lens=[1000, 129], n=9, cap=1100, packed=False), dict(lens=[500, 127], n=9, cap=600, idim=64)],
    ids=["five", "paged32", "chain64", "one", "16-bit", "dim64"])
def test_scores_of_wide_queries(c, queries):
    t = Tree(seed=21, **c)
    _with_queries(t, QUERIES[queries])
    s, d = t.shape, t.dev
    out = guarded_like((s.batch, s.n_heads_kv, t.n, t.nB), torch.float32)
    _lib.msa_index_scores_tree(s, t.seq_lens, t.table, t.n_phys, t.mask, d["iq"], d["ik"], d["ikd"],
                               out.tensor, packed=t.packed)
    _lib.msa_get_device_status()
    got, want = out.tensor.cpu().double().numpy(), t.scores()
    assert np.array_equal(np.isneginf(got), np.isneginf(want)) and not np.isnan(got).any()
    fine = np.isfinite(want)
    err = np.abs(np.where(fine, got, 0) - np.where(fine, want, 0))
    bound = _bound(t) + 2.0 ** -23 * np.abs(np.where(fine, want, 0))
    assert (err <= bound).all(), (err.max(), (err / np.maximum(bound, 1e-300)).max())
    out.check("scores")
