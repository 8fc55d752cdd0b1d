"""What api.decode_packed refuses, it refuses before the new token is written into the cache."""
import pytest
import torch

from block_sparse_gqa_02_gb300 import _lib, api

BF = torch.bfloat16


def _step(device, Hq=16, Hkv=4, d=128, dtype=BF, dI=128, top_k=3, with_mass=False, **other):
    """Arguments of a step of two sequences on filled caches, and the cache."""
    B, P, cap = 2, 20, 1000
    z = lambda *s, dt=dtype: torch.ones(s, dtype=dt, device=device)  # noqa: E731
    cache = torch.full((P, Hkv, 160 * d), 7, dtype=torch.uint8, device=device)
    args = dict(q=z(B, 1, Hq, d), k=z(B, Hkv, 1, d), v=z(B, Hkv, 1, d), cache=cache, idx_q=z(B, 1, Hkv, dI),
                idx_k_pool=z(P, 128, dI), seq_lens=z(B, dt=torch.int32) * 300,
                block_table=torch.arange(16, dtype=torch.int32, device=device).view(B, 8), capacity=cap,
                top_k=top_k, mass=z(B, Hkv, 8, dt=torch.float32) if with_mass else None)
    args.update(other)
    return args, cache


UNSUPPORTED = {
    "fp32": dict(dtype=torch.float32), "head_dim_64": dict(d=64), "two_kv_heads": dict(Hkv=2),
    "eight_kv_heads": dict(Hkv=8), "wide_group": dict(Hq=68), "index_dim_64": dict(dI=64),
    "weights_of_1025": dict(top_k=1025, with_mass=True),
}


@pytest.mark.parametrize("name", list(UNSUPPORTED))
def test_unsupported_steps(name):
    args, _ = _step("cpu", **UNSUPPORTED[name])
    with pytest.raises(_lib.MsaError) as e:
        api.decode_packed(**args)
    assert e.value.status == _lib.MSA_ERR_UNSUPPORTED


def test_steps_off_the_device():
    args, _ = _step("cpu")
    with pytest.raises(ValueError, match="current CUDA device"):
        api.decode_packed(**args)


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(UNSUPPORTED))
def test_unsupported_steps_leave_the_cache(name):
    args, cache = _step("cuda", **UNSUPPORTED[name])
    with pytest.raises(_lib.MsaError) as e:
        api.decode_packed(**args)
    assert e.value.status == _lib.MSA_ERR_UNSUPPORTED
    assert bool((cache == 7).all())


def _off(*shape, dt=BF):
    """A contiguous tensor that starts 8 bytes into its memory."""
    n = 1
    for x in shape:
        n *= x
    item = torch.empty((), dtype=dt).element_size()
    return torch.ones(n + 8 // item, dtype=dt, device="cuda")[8 // item:].view(shape)


BAD = {
    "q": lambda: _off(2, 1, 16, 128), "idx_q": lambda: _off(2, 1, 4, 128),
    "idx_k_pool": lambda: _off(20, 128, 128), "mass": lambda: _off(2, 4, 8, dt=torch.float32),
    "v": lambda: _off(2, 4, 1, 128), "seq_lens": lambda: _off(2, dt=torch.int32),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(BAD))
def test_unaligned_arguments_leave_the_cache(name):
    args, cache = _step("cuda", **{name: BAD[name]()})
    with pytest.raises((ValueError, _lib.MsaError), match="align"):
        api.decode_packed(**args)
    assert bool((cache == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("name,dtype", [("idx_q", torch.float32), ("idx_k_pool", torch.float16),
                                        ("idx_k_pool", torch.float32), ("mass", torch.float64),
                                        ("seq_lens", torch.int64), ("block_table", torch.int64),
                                        ("k", torch.float16), ("cache", torch.int8)])
def test_other_types_leave_the_cache(name, dtype):
    args, cache = _step("cuda", with_mass=True)
    args[name] = args[name].to(dtype)
    with pytest.raises(ValueError, match=f"{name} is"):
        api.decode_packed(**args)
    assert bool((cache == 7).all())


@pytest.mark.gpu
def test_a_step_changes_the_tokens_bytes_only():
    args, cache = _step("cuda", with_mass=True)
    api.decode_packed(**args)
    _lib.msa_get_device_status()
    touched = (cache != 7).view(20, 4, -1).any(-1)
    assert touched.nonzero()[:, 0].unique().tolist() == [2, 10]   # block 2 of each sequence
    assert float(args["mass"].double().sum()) == pytest.approx(2 * 4 * 8 + 2 * 16, rel=1e-3)
