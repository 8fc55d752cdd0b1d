"""A whole decode step over the 4-bit cache captured once and replayed on new tokens, lengths and
positions, across an eviction: the bits of the same steps run one by one."""
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api
from tests.test_gpu_packed import _i32, _rows

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
B, HQ, HKV, D, CAP, NB = 3, 32, 4, 128, 2048, 16


def _state():
    P = B * NB
    freqs, scale = api.rope_freqs(D, scaling="yarn", factor=4.0, original_len=512, device="cuda")
    table = torch.randperm(P, generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    s = dict(table=table.to(torch.int32).view(B, NB).contiguous(), cache=api.alloc_packed_cache(P, HKV, D),
             pool=_rows((P, 128, 128), BF, 3), lens=_i32([1500, 640, 1]), pos=_i32([1500, 640, 1]),
             mass=torch.zeros((B, HKV, NB), device="cuda"), rope=api.Rope(freqs, scale=scale))
    s["q"], s["iq"] = (torch.empty(n, dtype=BF, device="cuda") for n in ((B, 1, HQ, D), (B, 1, HKV, 128)))
    s["k"], s["v"] = (torch.empty((B, HKV, 1, D), dtype=BF, device="cuda") for _ in range(2))
    shape = _lib.make_shape(B, 1, CAP, HQ, HKV, D, 128, 128, 4, 1)
    rows = [_rows((B, HKV, 1500, D), BF, i) for i in range(2)]
    _lib.msa_cache_pack(shape, 1500, _i32([0] * B), s["lens"], s["table"], P, *rows, s["cache"])
    return s


def _token(s, i):
    for j, name in enumerate(("q", "iq", "k", "v")):
        s[name].copy_(_rows(tuple(s[name].shape), BF, 100 + 10 * i + j))
    s["lens"] += 1


def _step(s):
    return api.decode_packed(s["q"], s["k"], s["v"], s["cache"], s["iq"], s["pool"], s["lens"], s["table"],
                             CAP, 4, rope=s["rope"], mass=s["mass"], positions=s["pos"])


def _after(s, i):
    s["pos"] += 1
    if i == 2:
        api.evict_paged(s["lens"], s["mass"], s["table"], CAP, 5)


def test_captured_step():
    one, two = _state(), _state()
    _token(two, 0)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        replayed = _step(two)
    two["lens"] -= 1
    for i in range(6):
        _token(one, i)
        eager = _step(one)
        _token(two, i)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("out", "lse", "sel"):
            assert torch.equal(eager[name], replayed[name]), (i, name)
        for name in ("cache", "mass", "lens"):
            assert torch.equal(one[name], two[name]), (i, name)
        _after(one, i)
        _after(two, i)
    _lib.msa_get_device_status()
    assert one["lens"].tolist()[0] < one["pos"].tolist()[0] - 500      # the cut was a real one
