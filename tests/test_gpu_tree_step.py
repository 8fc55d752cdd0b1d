"""Whole steps over drafted tokens through the Python calls: against decode on the linear caches,
over several steps with commits, captured in a graph, and on other streams."""
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api
from tests.test_gpu_packed import _i32, _rows

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HQ, HKV, D = 32, 4, 128


def _close(a, b, tol):
    return float((a.double() - b.double()).norm()) <= tol * float(b.double().norm())


def _drafts(B, N, seed):
    return dict(q=_rows((B, N, HQ, D), BF, seed), k=_rows((B, HKV, N, D), BF, seed + 1), v=_rows((B, HKV, N, D), BF, seed + 2),
                idx_q=_rows((B, N, HKV, D), BF, seed + 3), idx_k=_rows((B, N, D), BF, seed + 4))


@pytest.mark.parametrize("with_rope", [False, True])
@pytest.mark.parametrize("L", [600, 1021])
def test_chain_is_sequential_decode(with_rope, L):
    """Token i of a chain gets what decode gives it over the caches with tokens 0 .. i appended: the
    same scores (both exact products, summed in fp32), selection and attention."""
    B, N, topk = 2, 6, 4
    rope = None
    if with_rope:
        freqs, scale = api.rope_freqs(D, scaling="yarn", factor=4.0, original_len=512, device="cuda")
        rope = api.Rope(freqs, scale=scale)
    cap = L + N
    kc, vc, ic = _rows((B, HKV, cap, D), BF, 1), _rows((B, HKV, cap, D), BF, 2), _rows((B, cap, D), BF, 3)
    x = _drafts(B, N, 10)
    lens = _i32([L] * B)
    parents = _i32([[i - 1 for i in range(N)]] * B)
    step = api.decode_tree(**x, k_cache=kc, v_cache=vc, idx_cache=ic, seq_lens=lens, parents=parents, top_k=topk, rope=rope)
    assert step["positions"].tolist() == [[L + i for i in range(N)]] * B
    kc2, vc2, ic2, lens2 = kc.clone(), vc.clone(), ic.clone(), lens.clone()
    api.commit_tree(step, _i32([list(range(N))] * B), kc2, vc2, ic2, lens2)
    assert lens2.tolist() == [cap] * B
    assert torch.equal(kc2[:, :, :L], kc[:, :, :L]) and torch.equal(kc2[:, :, L:], step["k"])
    assert torch.equal(vc2[:, :, L:], x["v"]) and torch.equal(ic2[:, L:], step["idx_k"])
    if not with_rope:
        assert torch.equal(step["k"], x["k"])
    for i in range(N):
        one = lambda y: y[:, i:i + 1].contiguous()  # noqa: E731
        d = api.decode(one(x["q"]), kc2[:, :, :L + i + 1].contiguous(), vc2[:, :, :L + i + 1].contiguous(),
                       one(x["idx_q"]), ic2[:, :L + i + 1].contiguous(), top_k=topk, rope=rope)
        n = d["scores"].shape[-1]
        assert _close(step["scores"][:, :, i, :n], d["scores"][:, :, 0], 1e-6)
        assert torch.isneginf(step["scores"][:, :, i, n:]).all()
        assert torch.equal(step["sel"][:, :, i], d["sel"][:, :, 0])
        assert _close(step["out"][:, i], d["out"][:, 0], 8e-3)             # two bf16 roundings of P and out
        assert _close(step["lse"][:, :, i], d["lse"][:, :, 0], 1e-5)
    _lib.msa_get_device_status()


def _state(paged, seed=0):
    B, cap, nB = 3, 1100, 9
    P = B * nB + (2 if paged else 0)
    g = torch.Generator("cuda").manual_seed(seed)
    s = dict(lens=_i32([900, 250, 0]), table=None, cap=cap)
    if paged:
        s["table"] = torch.randperm(P, generator=g, device="cuda")[:B * nB].to(torch.int32).view(B, nB).contiguous()
    s["kc"], s["vc"] = (_rows((P, HKV, 128, D) if paged else (B, HKV, cap, D), BF, seed + i) for i in (1, 2))
    s["ic"] = api.alloc_index_cache(P)
    api.pack_index(_rows((B, 900, D), BF, seed + 3), s["ic"], s["lens"], s["table"], _i32([0] * B), cap)
    freqs, scale = api.rope_freqs(D, device="cuda")
    s["rope"] = api.Rope(freqs, scale=scale)
    return s


PARENTS = [[-1, 0, 0, 1, 2, -1, 5], [-1, -1, 1, 1, 2, 2, -2], [-1, 0, 1, 2, 3, 4, 5]]


def _run(s, x, acc):
    step = api.decode_tree(x["q"], x["k"], x["v"], x["idx_q"], x["idx_k"], s["kc"], s["vc"], s["ic"], s["lens"], s["parents"],
                           s["table"], s["cap"], top_k=4, rope=s["rope"])
    api.commit_tree(step, acc, s["kc"], s["vc"], s["ic"], s["lens"], s["table"], s["cap"])
    return step


@pytest.mark.parametrize("paged", [False, True])
def test_captured_steps(paged):
    """Several steps, each with its commit, eager and as replays of one graph: the same bits."""
    one, two = _state(paged), _state(paged)
    accepted = [[[0, 1, 3, -1], [1, 2, 4, -1], [0, 1, 2, 3]], [[5, 6, -1, -1], [-1] * 4, [0, 1, -1, -1]],
                [[0, 2, 4, -1], [0, -1, -1, -1], [0, 1, 2, 3]]]
    x, acc = _drafts(3, 7, 50), _i32(accepted[0])
    for s in (one, two):
        s["parents"] = _i32(PARENTS)
    backup = {k: two[k].clone() for k in ("kc", "vc", "ic", "lens")}
    _run(two, x, acc)                                       # warm-up outside the capture
    for k, v in backup.items():
        two[k].copy_(v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = _run(two, x, acc)
    for k, v in backup.items():
        two[k].copy_(v)
    for i in range(4):
        fresh = _drafts(3, 7, 100 + 10 * i)
        for n in x:
            x[n].copy_(fresh[n])
        acc.copy_(_i32(accepted[i % 3]))
        eager = _run(one, x, acc)
        graph.replay()
        torch.cuda.synchronize()
        for n in ("out", "lse", "scores", "sel", "mask", "positions"):
            assert torch.equal(eager[n], replayed[n]), (i, n)
        for n in ("kc", "vc", "ic", "lens"):
            assert torch.equal(one[n].view(torch.uint8), two[n].view(torch.uint8)), (i, n)
    assert one["lens"].tolist() == [900 + 3 + 2 + 3 + 3, 250 + 3 + 0 + 1 + 3, 4 + 2 + 4 + 4]
    _lib.msa_get_device_status()


def test_two_streams_at_once():
    """Steps on two streams, issued in turn without waiting: the bits of the steps run alone."""
    states = [_state(True, 0), _state(False, 7)]
    xs = [_drafts(3, 7, 20), _drafts(3, 7, 40)]
    for s in states:
        s["parents"] = _i32(PARENTS)
    acc = _i32([[-1, -1]] * 3)
    want = [_run(s, x, acc) for s, x in zip(states, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                got[j].append(_run(states[j], xs[j], acc))
    torch.cuda.synchronize()
    for j in range(2):
        for g in got[j]:
            for n in ("out", "lse", "scores", "sel"):
                assert torch.equal(g[n], want[j][n]), (j, n)
    _lib.msa_get_device_status()


def test_positions_after_an_eviction():
    """With positions, rotation goes on from them and not from the shortened lengths."""
    s = _state(False)
    x = _drafts(3, 7, 60)
    s["parents"] = _i32(PARENTS)
    pos = s["lens"] + _i32([1000, 0, 7])
    step = api.decode_tree(x["q"], x["k"], x["v"], x["idx_q"], x["idx_k"], s["kc"], s["vc"], s["ic"], s["lens"], s["parents"],
                           s["table"], s["cap"], top_k=4, rope=s["rope"], positions=pos)
    at = step["positions"] + (pos - s["lens"])[:, None]
    want, = api.rope([(x["k"], s["rope"].freqs, True)], at.contiguous(), scale=s["rope"].scale)
    there = step["mask"] != 0
    assert torch.equal(step["k"].transpose(1, 2)[there], want.transpose(1, 2)[there])
    assert (step["mask"][1, 6] == 0) and there.sum() == 20


def test_refusals():
    s = _state(True)
    x = _drafts(3, 7, 70)
    args = dict(x, k_cache=s["kc"], v_cache=s["vc"], idx_cache=s["ic"], seq_lens=s["lens"], parents=_i32(PARENTS),
                block_table=s["table"], top_k=4, capacity=s["cap"])
    api.decode_tree(**args)
    for name, bad in (("k", x["k"][:, :, :5].contiguous()), ("idx_k", x["idx_k"].unsqueeze(1)), ("parents", _i32(PARENTS)[:, :6].contiguous()),
                      ("block_table", s["table"][:, :8].contiguous()), ("v_cache", s["vc"][:-1]), ("idx_cache", s["ic"][:, :-128].contiguous()),
                      ("seq_lens", s["lens"].cpu()), ("seq_lens", s["lens"].long()), ("idx_cache", _rows((5, 128, 128), BF, 1)),
                      ("positions", s["lens"]), ("q", x["q"].transpose(1, 2))):
        with pytest.raises((ValueError, _lib.MsaError)):
            api.decode_tree(**{**args, name: bad})
    step = api.decode_tree(**args)
    keep = s["lens"].clone()
    with pytest.raises(ValueError):
        api.commit_tree(step, _i32([[0], [1]]), s["kc"], s["vc"], s["ic"], s["lens"], s["table"])
    with pytest.raises(ValueError):
        api.commit_tree(step, _i32([[0]] * 3), s["kc"], s["vc"][:-1], s["ic"], s["lens"], s["table"])
    assert torch.equal(keep, s["lens"])
    _lib.msa_get_device_status()


@pytest.mark.parametrize("call", ["scores", "attention"])
def test_given_up_wait(call):
    """The CTA of a row's first split (or range) copies one block only: its wait runs out, the call
    reports it, and the next one is right."""
    B, N, cap = 1, 4, 60000
    x, lens, parents = _drafts(B, N, 5), _i32([cap - N]), _i32([[-1, 0, 1, 2]])
    kc, vc, ic = _rows((B, HKV, cap, D), BF, 1), _rows((B, HKV, cap, D), BF, 2), _rows((B, cap, D), BF, 3)
    good = api.decode_tree(**x, k_cache=kc, v_cache=vc, idx_cache=ic, seq_lens=lens, parents=parents, top_k=120)
    shape = _lib.make_shape(B, N, cap, HQ, HKV, D, D, 128, 120, 1)
    ws = torch.empty(_lib.msa_workspace_bytes(shape, 5) // 4 + 4, device="cuda")
    out, lse, scores = (torch.empty_like(good[n]) for n in ("out", "lse", "scores"))

    def run():
        if call == "scores":
            _lib.msa_index_scores_tree(shape, lens, None, 0, good["mask"], x["idx_q"], ic, good["idx_k"], scores)
        else:
            _lib.msa_sparse_decode_tree(shape, lens, None, 0, good["mask"], x["q"], kc, vc, good["k"], good["v"], good["sel"], out, lse, ws)
    _lib.msa_get_device_status()
    _lib.msa_debug_set_fault(2)
    try:
        run()
        with pytest.raises(_lib.MsaError) as e:
            _lib.msa_get_device_status()
        assert e.value.status == _lib.MSA_ERR_TIMEOUT
    finally:
        _lib.msa_debug_set_fault(0)
    run()
    _lib.msa_get_device_status()
    assert torch.equal(scores, good["scores"]) if call == "scores" else torch.equal(out, good["out"])
