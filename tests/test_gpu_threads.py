"""Calls from host threads at once, on streams of their own and with sizes that take one kernel
with different amounts of shared memory: every call succeeds, with the results that it has alone,
bit for bit.  The C entry points are called directly, without work between the calls: what one
thread sets for a kernel must not reach another between its own setting and its launch."""
import ctypes
import sys
import threading

import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api
from tests.test_gpu_packed import _i32, _rows

pytestmark = pytest.mark.gpu

BF, CALLS = torch.bfloat16, 3000


class Call:
    """A C call on prepared arguments (tensors by their address, the stream last)."""

    def __init__(self, name, shape, args, outputs):
        self.fn, self.hold = getattr(_lib.load(), name), (shape, args)
        self.args = [ctypes.byref(shape)] + [x.data_ptr() if torch.is_tensor(x) else x for x in args]
        self.outputs = outputs

    def __call__(self, stream):
        return self.fn(*self.args, stream.cuda_stream)


def _packed(topk, mass):
    B, Hq, Hkv, d, cap = 1, 16, 4, 128, 128 * 1024
    shape = _lib.make_shape(B, 1, cap, Hq, Hkv, d, 128, 128, topk, 1)
    g = torch.Generator("cuda").manual_seed(topk)
    cache = api.alloc_packed_cache(1024, Hkv, d)
    k, v = _rows((B, Hkv, 128 * 20, d), BF, 1), _rows((B, Hkv, 128 * 20, d), BF, 2)
    _lib.msa_cache_pack(shape, 128 * 20, _i32([0]), _i32([cap]), None, 1024, k, v, cache)
    sel = torch.full((B, Hkv, 1, topk), -1, dtype=torch.int32, device="cuda")
    sel[..., :15] = torch.randperm(20, generator=g, device="cuda")[:15].to(torch.int32)
    q = _rows((B, 1, Hq, d), BF, 3)
    out, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")
    w = torch.zeros((B, Hkv, 1024), device="cuda") if mass else None
    return Call("msa_sparse_decode_packed", shape, [None, None, 1024, q, cache, sel, out, lse, w], [out, lse])


def _evict(blocks):
    shape = _lib.make_shape(1, 1, 128 * blocks, 2, 2, 128, 128, 128, 1, 1)
    mass = torch.rand((1, 2, blocks), generator=torch.Generator("cuda").manual_seed(blocks), device="cuda")
    kept, lens, out = _i32([0] * 100), _i32([0]), torch.empty_like(mass)
    return Call("msa_cache_evict", shape, [100, 1, 2, None, mass, None, kept, lens, out, None],
                [kept, lens, out])


def _topk(blocks):
    shape = _lib.make_shape(1, 1, 128 * blocks, 4, 4, 128, 128, 128, 64, 1)
    scores = torch.rand((1, 4, 1, blocks), generator=torch.Generator("cuda").manual_seed(blocks), device="cuda")
    sel = torch.empty((1, 4, 1, 64), dtype=torch.int32, device="cuda")
    return Call("msa_block_topk", shape, [scores, sel], [sel])


def _scores(block):
    T = 2 * block
    shape = _lib.make_shape(1, T, T, 2, 2, 64, 64, block, 1, block // 2, "f32")
    iq, ik = _rows((1, T, 2, 64), torch.float32, 1), _rows((1, T, 64), torch.float32, 2)
    out = torch.empty((1, 2, shape.n_rows, shape.n_blocks), device="cuda")
    return Call("msa_index_scores", shape, [iq, ik, out], [out])


PAIRS = {
    "packed": (lambda: _packed(16, False), lambda: _packed(16 * 900, False)),
    "packed_mass": (lambda: _packed(16, True), lambda: _packed(1024, True)),
    "evict_small": (lambda: _evict(10), lambda: _evict(1024)),
    "evict": (lambda: _evict(8200), lambda: _evict(32768)),
    "topk": (lambda: _topk(12400), lambda: _topk(32768)),
    "index_scores": (lambda: _scores(32), lambda: _scores(256)),
}


@pytest.mark.parametrize("name", list(PAIRS))
def test_host_threads(name):
    work = [make() for make in PAIRS[name]]
    alone = []
    for call in work:
        assert call(torch.cuda.current_stream()) == _lib.MSA_OK
        torch.cuda.synchronize()
        alone.append([x.clone() for x in call.outputs])
        for x in call.outputs:
            x.zero_()
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(work)), []

    def loop(call, stream):
        start.wait()
        failed.append(sum(call(stream) != _lib.MSA_OK for _ in range(CALLS)))
    threads = [threading.Thread(target=loop, args=pair) for pair in zip(work, streams)]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    assert failed == [0, 0], f"{failed} of {CALLS} calls were refused"
    _lib.msa_get_device_status()
    for call, want in zip(work, alone):
        for x, y in zip(call.outputs, want):
            assert torch.equal(x, y)
