"""Rotary positions (msa_rope, api.rope, the rope argument of api.prefill and api.decode) against
the fp64 reference.

Tolerance, from the arithmetic: the angle reaches sincospif as an fp32 fraction of at most 1/4
half turn, off by 2^-26 half turns (pi 2^-26 < 2^-24 radians); sine and cosine are within 2 ulp
(2^-23) and are multiplied by scale (2^-24 more); the two products and their sum add 2 * 2^-24 of
|x0| + |x1|.  Together 6 * 2^-24 * scale * (|x0| + |x1|) and the result's rounding, half a step of
its type (bf16 2^-8 of the value, fp32 2^-24)."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api
from oracle import cache_ops as co
from tests.canary import guarded_like
from tests.parity import to_np

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _check(y, x, pos, freqs, dtype, scale=1.0, **kw):
    ref = co.rope(x, pos, freqs.cpu(), scale=scale, **kw)
    n = 2 * freqs.numel()
    ax = np.abs(to_np(x))
    pair = np.zeros_like(ax)
    if kw.get("interleaved"):
        pair[..., 0:n:2] = pair[..., 1:n:2] = ax[..., 0:n:2] + ax[..., 1:n:2]
    else:
        pair[..., :n // 2] = pair[..., n // 2:n] = ax[..., :n // 2] + ax[..., n // 2:n]
    arith = 6 * 2.0 ** -24 * abs(scale) * pair
    bound = arith + HALF_STEP[dtype] * (np.abs(ref) + arith)
    err = np.abs(to_np(y) - ref)
    assert np.all(err <= bound), (err - bound).max()
    assert np.array_equal(to_np(y)[..., n:], to_np(x)[..., n:])


CASES = [  # batch, seq, heads, d, rot
    (1, 1, 1, 16, 16), (3, 1, 64, 128, 128), (2, 7, 5, 64, 16), (1, 33, 3, 80, 48),
    (2, 513, 4, 128, 64), (1, 100, 2, 1024, 1024), (5, 3, 9, 112, 96), (1, 1000, 1, 128, 128),
    (2, 129, 16, 64, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("head_major", [False, True])
def test_rope_shapes(dtype, interleaved, head_major):
    for i, (B, S, H, d, rot) in enumerate(CASES):
        shape = (B, H, S, d) if head_major else (B, S, H, d)
        x = torch.randn(shape, generator=_gen(i), device="cuda").to(DT[dtype])
        freqs, _ = api.rope_freqs(rot, device="cuda")
        pos = torch.randint(0, 1 << 20, (B, S), generator=_gen(i), device="cuda", dtype=torch.int32)
        y = guarded_like(shape, DT[dtype])
        args = _lib.make_rope_tensors([(x, y.tensor, freqs, head_major)])
        inverse = bool(i % 2)
        desc = _lib.make_rope(B, S, dtype, pos_offset=-1, scale=1.25, interleaved=interleaved,
                              inverse=inverse)
        _lib.msa_rope(desc, args, pos)
        _lib.msa_get_device_status()
        y.check(f"rope {shape}")
        kw = dict(interleaved=interleaved, inverse=inverse, head_major=head_major, scale=1.25)
        _check(y.tensor, x, pos.cpu().numpy().astype(np.int64) - 1, freqs, dtype, **kw)
        # in place: the same bits
        z = x.clone()
        _lib.msa_rope(desc, _lib.make_rope_tensors([(z, z, freqs, head_major)]), pos)
        assert torch.equal(z, y.tensor)


@pytest.mark.parametrize("positions", [
    [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 20, 123456789],
])
def test_rope_far_and_negative_positions(positions):
    """Angles of any 32-bit position are exact; sums with the offset wrap as 32-bit integers."""
    n = len(positions)
    x = torch.randn((1, n, 2, 64), generator=_gen(1), device="cuda")
    freqs, _ = api.rope_freqs(64, device="cuda")
    pos = torch.tensor([positions], dtype=torch.int32, device="cuda")
    for off in (0, 3, -7):
        y, = api.rope([(x, freqs, False)], pos, pos_offset=off)
        want = ((np.array([positions], dtype=np.int64) + off + 2 ** 31) % 2 ** 32) - 2 ** 31
        _check(y, x, want, freqs, "f32")


def test_rope_several_tensors_one_launch():
    """q, k, idx_q and idx_k of a batch in one call give each the bits of its own call."""
    B, S = 3, 77
    g = _gen(2)
    f128, scale = api.rope_freqs(128, scaling="yarn", factor=4.0, original_len=4096, device="cuda")
    f64, _ = api.rope_freqs(64, scaling="ntk", factor=2.0, device="cuda")
    rows = [(torch.randn((B, S, 16, 128), generator=g, device="cuda").bfloat16(), f128, False),
            (torch.randn((B, 4, S, 128), generator=g, device="cuda").bfloat16(), f128, True),
            (torch.randn((B, S, 4, 64), generator=g, device="cuda").bfloat16(), f64, False),
            (torch.randn((B, S, 64), generator=g, device="cuda").bfloat16(), f64, False)]
    pos = torch.randint(0, 5000, (B, S), generator=g, device="cuda", dtype=torch.int32)
    got = api.rope(rows, pos, scale=scale)
    for y, row in zip(got, rows):
        one, = api.rope([row], pos, scale=scale)
        assert torch.equal(y, one)
    _check(got[1], rows[1][0], pos.cpu().numpy(), f128, "bf16", scale=scale, head_major=True)
    _check(got[3][:, :, None], rows[3][0][:, :, None], pos.cpu().numpy(), f64, "bf16", scale=scale)


def test_rope_gradient():
    """Forward and inverse against each other and against differences: <dy, R x> = <R' dy, x>,
    and central differences of <dy, R x> along a direction."""
    B, S, H, d = 2, 65, 3, 64
    g = _gen(3)
    freqs, _ = api.rope_freqs(32, device="cuda")
    x, dy, e = (torch.randn((B, S, H, d), generator=g, device="cuda") for _ in range(3))
    f = lambda t: api.rope([(t, freqs, False)], scale=0.5)[0].double()  # noqa: E731
    dx = api.rope([(dy, freqs, False)], scale=0.5, inverse=True)[0].double()
    fwd, back = (dy.double() * f(x)).sum(), (dx * x.double()).sum()
    norm = float(dy.double().norm() * x.double().norm())
    # each element is off by 7 * 2^-24 of its pair (above), |pair| <= sqrt 2 of its 2-norm
    assert abs(float(fwd - back)) <= 2 * 10 * 2.0 ** -24 * norm
    num = ((f(x + e) - f(x - e)) * dy.double()).sum() / 2
    # the map is linear, so a step of 1 has no truncation error: only the arithmetic's, of two
    # calls on values of norm |x| + |e|, and the rounding of x + e and x - e
    room = 12 * 2.0 ** -24 * float(dy.double().norm()) * float(x.norm() + e.norm())
    assert abs(float(num - (dx * e.double()).sum())) <= 2 * room


def test_rope_past_32_bit_offsets():
    """2.4 G elements: byte and element offsets past 32 bits, checked at the end."""
    B, S, H, d = 1, 290_001, 64, 128
    x = torch.zeros((B, S, H, d), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((B, 5, H, d), generator=_gen(4), device="cuda").bfloat16()
    x[:, -5:] = tail
    freqs, _ = api.rope_freqs(128, device="cuda")
    _lib.msa_rope(_lib.make_rope(B, S), _lib.make_rope_tensors([(x, x, freqs, False)]))
    _check(x[:, -5:], tail, np.arange(S - 5, S)[None], freqs, "bf16")
    assert not x[:, :-5].any()


def test_rope_stream_and_graph():
    """On a side stream and replayed from a graph on new inputs."""
    freqs, _ = api.rope_freqs(64, device="cuda")
    x = torch.randn((4, 1, 8, 64), generator=_gen(5), device="cuda").bfloat16()
    y = torch.zeros_like(x)
    pos = torch.tensor([[5], [6], [7], [8]], dtype=torch.int32, device="cuda")
    desc, args = _lib.make_rope(4, 1), _lib.make_rope_tensors([(x, y, freqs, False)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _lib.msa_rope(desc, args, pos)
    side.synchronize()
    _check(y, x, pos.cpu().numpy(), freqs, "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.msa_rope(desc, args, pos)
    x.copy_(torch.randn(x.shape, generator=_gen(6), device="cuda"))
    pos += 100000
    graph.replay()
    torch.cuda.synchronize()
    _check(y, x, pos.cpu().numpy(), freqs, "bf16")


def test_prefill_and_decode_with_rope():
    """api.prefill and api.decode with a Rope are the calls on tensors rotated beforehand."""
    from block_sparse_gqa_02_gb300.configs import CONFIGS
    from block_sparse_gqa_02_gb300.inputs import make_inputs
    cfg = CONFIGS["p32k"].with_(seq=700, top_k=3, n_plants=0)
    x = make_inputs(cfg, device="cuda")
    freqs, scale = api.rope_freqs(128, scaling="linear", factor=2.0, device="cuda")
    half, _ = api.rope_freqs(64, device="cuda")
    rope = api.Rope(freqs, index_freqs=half, scale=scale)
    got = api.prefill(x["q"], x["k"], x["v"], x["idx_q"], x["idx_k"], top_k=3, rope=rope)
    q, k = api.rope([(x["q"], freqs, False), (x["k"], freqs, True)])
    iq, ik = api.rope([(x["idx_q"], half, False), (x["idx_k"], half, False)])
    ref = api.prefill(q, k, x["v"], iq, ik, top_k=3)
    for n in ("scores", "sel", "out", "lse"):
        assert torch.equal(got[n], ref[n])
    assert torch.equal(got["k"], k) and torch.equal(got["idx_k"], ik)
    # one more token: the caches hold rotated keys, the query is rotated to the last position
    last = slice(699, 700)
    step = api.decode(x["q"][:, last], k, x["v"], x["idx_q"][:, last], ik, top_k=3, rope=rope)
    again = api.decode(q[:, last], k, x["v"], iq[:, last], ik, top_k=3)
    for n in ("scores", "sel", "out", "lse"):
        assert torch.equal(step[n], again[n])


def test_rope_binding_refuses():
    freqs, _ = api.rope_freqs(64, device="cuda")
    x = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="shape and type"):
        _lib.make_rope_tensors([(x, x.float(), freqs, False)])
    with pytest.raises(ValueError, match="contiguous"):
        _lib.make_rope_tensors([(x.transpose(1, 2), x.transpose(1, 2), freqs, False)])
    with pytest.raises(ValueError, match="expected torch.int64"):
        _lib.make_rope_tensors([(x, x, freqs.double(), False)])
    args = _lib.make_rope_tensors([(x, x, freqs, False)])
    with pytest.raises(ValueError, match="the call"):
        _lib.msa_rope(_lib.make_rope(2, 4), args)
    with pytest.raises(ValueError, match="the call"):
        _lib.msa_rope(_lib.make_rope(2, 3, "f32"), args)
    with pytest.raises(ValueError, match="positions"):
        _lib.msa_rope(_lib.make_rope(2, 3), args, torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(_lib.MsaError) as err:
        _lib.msa_rope(_lib.make_rope(2, 3), _lib.make_rope_tensors([]))
    assert err.value.status == _lib.MSA_ERR_INVALID_ARG
