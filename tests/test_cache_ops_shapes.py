"""Tensors of another stride than the call's: an array whose later axes are longer than the call
indexes holds every row but the first in another place.  Such calls are refused; a longer first
axis and flat buffers are not."""
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api

BF, I32, F32, U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
B, HQ, HKV, D, CAP, NB, P, K, N = 2, 16, 4, 128, 1000, 8, 20, 3, 5


def _z(*shape, dt=BF, device="cpu"):
    return torch.zeros(shape, dtype=dt, device=device)


def _shape(**kw):
    return _lib.make_shape(B, 1, CAP, HQ, HKV, D, 128, 128, K, 1, **kw)


def _pack(name, device="cpu", **t):
    a = dict(starts=_z(B, dt=I32), seq_lens=_z(B, dt=I32), block_table=_z(B, NB, dt=I32),
             k=_z(B, HKV, N, D), v=_z(B, HKV, N, D), cache=_z(P, HKV, 160 * D, dt=U8))
    a.update(t)
    a = {n: x.to(device) for n, x in a.items()}
    order = ("k", "v", "cache") if name == "msa_cache_pack" else ("cache", "k", "v")
    getattr(_lib, name)(_shape(), N, a["starts"], a["seq_lens"], a["block_table"], P, *(a[n] for n in order))


def _packed(device="cpu", **t):
    a = dict(seq_lens=_z(B, dt=I32), block_table=_z(B, NB, dt=I32), q=_z(B, 1, HQ, D),
             cache=_z(P, HKV, 160 * D, dt=U8), sel=_z(B, HKV, 1, K, dt=I32), out=_z(B, 1, HQ, D),
             lse=_z(B, HQ, 1, dt=F32), mass=_z(B, HKV, NB, dt=F32))
    a.update(t)
    a = {n: x.to(device) for n, x in a.items()}
    _lib.msa_sparse_decode_packed(_shape(), a["seq_lens"], a["block_table"], P, a["q"], a["cache"],
                                  a["sel"], a["out"], a["lse"], a["mass"])


def _weights(paged, device="cpu", **t):
    kv = (P, HKV, 128, D) if paged else (B, HKV, CAP, D)
    a = dict(seq_lens=_z(B, dt=I32), block_table=_z(B, NB, dt=I32), q=_z(B, 1, HQ, D), k=_z(*kv), v=_z(*kv),
             sel=_z(B, HKV, 1, K, dt=I32), out=_z(B, 1, HQ, D), lse=_z(B, HQ, 1, dt=F32),
             mass=_z(B, HKV, NB, dt=F32), ws=_z(1 << 20, dt=F32))
    a.update(t)
    a = {n: x.to(device) for n, x in a.items()}
    lead = (a["seq_lens"], a["block_table"], P) if paged else (None, None, 0)
    _lib.msa_sparse_decode_mass(_shape(), *lead, a["q"], a["k"], a["v"], a["sel"], a["out"], a["lse"],
                                a["mass"], a["ws"])


def _evict(device="cpu", **t):
    a = dict(seq_lens=_z(B, dt=I32), mass=_z(B, HKV, NB, dt=F32), block_table=_z(B, NB, dt=I32),
             kept=_z(B, 4, dt=I32), new_lens=_z(B, dt=I32), mass_out=_z(B, HKV, NB, dt=F32),
             table_out=_z(B, NB, dt=I32))
    a.update(t)
    a = {n: x.to(device) for n, x in a.items()}
    _lib.msa_cache_evict(_shape(), 4, 1, 2, a["seq_lens"], a["mass"], a["block_table"], a["kept"],
                         a["new_lens"], a["mass_out"], a["table_out"])


def _rope(device="cpu", positions=None):
    x = _z(B, N, HQ, D, device=device)
    freqs = api.rope_freqs(D, device=device)[0]
    _lib.msa_rope(_lib.make_rope(B, N), _lib.make_rope_tensors([(x, torch.empty_like(x), freqs, False)]),
                  positions.to(device))


def _step(device="cpu", **t):
    a = dict(q=_z(B, 1, HQ, D), k=_z(B, HKV, 1, D), v=_z(B, HKV, 1, D), cache=_z(P, HKV, 160 * D, dt=U8),
             idx_q=_z(B, 1, HKV, 128), idx_k_pool=_z(P, 128, 128), seq_lens=_z(B, dt=I32),
             block_table=_z(B, NB, dt=I32))
    a.update(t)
    api.decode_packed(**{n: x.to(device) for n, x in a.items()}, capacity=CAP, top_k=K)


WIDE = {
    "pack k": (lambda **t: _pack("msa_cache_pack", **t), dict(k=_z(B, HKV, N + 3, D))),
    "pack v": (lambda **t: _pack("msa_cache_pack", **t), dict(v=_z(B, HKV + 1, N, D))),
    "pack cache": (lambda **t: _pack("msa_cache_pack", **t), dict(cache=_z(P, HKV, 320 * D, dt=U8))),
    "pack cache heads": (lambda **t: _pack("msa_cache_pack", **t), dict(cache=_z(P, 8, 160 * D, dt=U8))),
    "pack starts": (lambda **t: _pack("msa_cache_pack", **t), dict(starts=_z(B, 2, dt=I32))),
    "unpack k": (lambda **t: _pack("msa_cache_unpack", **t), dict(k=_z(B, HKV, N + 1, D))),
    "unpack block_table": (lambda **t: _pack("msa_cache_unpack", **t), dict(block_table=_z(B, NB + 1, dt=I32))),
    "packed q": (_packed, dict(q=_z(B, 2, HQ, D))),
    "packed sel": (_packed, dict(sel=_z(B, HKV, 1, K + 1, dt=I32))),
    "packed cache": (_packed, dict(cache=_z(P, HKV, 320 * D, dt=U8))),
    "packed mass": (_packed, dict(mass=_z(B, HKV, NB + 1, dt=F32))),
    "packed lse": (_packed, dict(lse=_z(B, HQ, 2, dt=F32))),
    "packed seq_lens": (_packed, dict(seq_lens=_z(B, 2, dt=I32))),
    "weights k": (lambda **t: _weights(False, **t), dict(k=_z(B, HKV, CAP + 24, D))),
    "weights v": (lambda **t: _weights(True, **t), dict(v=_z(P, HKV, 256, D))),
    "weights sel": (lambda **t: _weights(True, **t), dict(sel=_z(B, HKV, 1, 64, dt=I32))),
    "weights block_table": (lambda **t: _weights(True, **t), dict(block_table=_z(B, 64, dt=I32))),
    "evict mass": (_evict, dict(mass=_z(B, HKV, NB + 1, dt=F32))),
    "evict kept": (_evict, dict(kept=_z(B, 5, dt=I32))),
    "evict table_out": (_evict, dict(table_out=_z(B, NB + 8, dt=I32))),
    "rope positions": (_rope, dict(positions=_z(B, N + 3, dt=I32))),
    "step q": (_step, dict(q=_z(B, 2, HQ, D))),
    "step k": (_step, dict(k=_z(B, HKV, 2, D))),
    "step cache": (_step, dict(cache=_z(P, HKV, 320 * D, dt=U8))),
    "step idx_q": (_step, dict(idx_q=_z(B, 2, HKV, 128))),
    "step seq_lens": (_step, dict(seq_lens=_z(B, 2, dt=I32))),
}


class NoLibrary:
    """Takes every call and launches nothing."""

    def __getattr__(self, name):
        return lambda *args: _lib.MSA_OK


@pytest.fixture
def host_only(monkeypatch):
    """The binding's checks on host tensors."""
    _lib._get_torch()
    monkeypatch.setattr(_lib, "_device", lambda: -1)
    monkeypatch.setattr(_lib, "_place", lambda stream: (-1, 0))
    monkeypatch.setattr(_lib, "load", lambda *a, **kw: NoLibrary())


@pytest.mark.parametrize("name", list(WIDE))
def test_another_stride_is_refused(host_only, name):
    call, t = WIDE[name]
    with pytest.raises(ValueError, match=f"{next(iter(t))} is .* expected"):
        call(**t)


LONG = {
    "pack": (lambda **t: _pack("msa_cache_pack", **t),
             dict(k=_z(B + 1, HKV, N, D), v=_z(B * HKV * N * D + 7), cache=_z(P + 1, HKV, 160 * D, dt=U8))),
    "packed": (_packed, dict(q=_z(B + 1, 1, HQ, D), sel=_z(B * HKV * K + 5, dt=I32), lse=_z(B + 3, HQ, dt=F32),
                             cache=_z(P + 1, HKV, 160 * D, dt=U8))),
    "weights": (lambda **t: _weights(False, **t), dict(k=_z(B + 1, HKV, CAP, D))),
    "evict": (_evict, dict(mass=_z(B + 1, HKV, NB, dt=F32), kept=_z(100, dt=I32))),
    "rope": (_rope, dict(positions=_z(B * N + 4, dt=I32))),
}


@pytest.mark.parametrize("name", list(LONG))
def test_longer_arrays_pass_the_checks(host_only, name):
    call, t = LONG[name]
    call(**t)


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(LONG))
def test_longer_arrays_are_taken(name):
    call, t = LONG[name]
    call(device="cuda", **t)
    _lib.msa_get_device_status()
