"""Whole-pass helpers over the C ABI: allocate the outputs with torch, then run the three
MSA stages (index block scores -> per-KV-head block top-k -> sparse attention) as
library calls on the current stream, with no host synchronisation in between."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import (make_gather_tensors, make_rope, make_rope_tensors, make_shape, msa_block_topk,
                   msa_block_topk_ragged, msa_cache_evict, msa_cache_gather, msa_cache_pack,
                   msa_index_scores, msa_index_scores_paged, msa_rope, msa_sparse_decode,
                   msa_sparse_decode_mass, msa_sparse_decode_packed, msa_sparse_prefill,
                   msa_workspace_bytes)

_DT = {torch.float32: "f32", torch.bfloat16: "bf16"}


def _shape_of(q, k, idx_q, block_size, top_k, q_tile, sm_scale, index_scale):
    B, Sq, Hq, d = q.shape
    _, Hkv, Sk, _ = k.shape
    return make_shape(B, Sq, Sk, Hq, Hkv, d, idx_q.shape[-1], block_size, top_k, q_tile,
                      _DT[q.dtype], sm_scale, index_scale)


def alloc_prefill_outputs(shape, device, dtype):
    B, Hkv = shape.batch, shape.n_heads_kv
    return dict(
        scores=torch.empty((B, Hkv, shape.n_rows, shape.n_blocks), device=device,
                           dtype=torch.float32),
        sel=torch.empty((B, Hkv, shape.n_rows, shape.top_k), device=device, dtype=torch.int32),
        out=torch.empty((B, shape.seq_q, shape.n_heads_q, shape.head_dim), device=device,
                        dtype=dtype),
        lse=torch.empty((B, shape.n_heads_q, shape.seq_q), device=device, dtype=torch.float32))


def run_prefill(shape, q, k, v, idx_q, idx_k, bufs, stream=None):
    """One prefill pass into preallocated buffers (dict from alloc_prefill_outputs)."""
    msa_index_scores(shape, idx_q, idx_k, bufs["scores"], stream)
    msa_block_topk(shape, bufs["scores"], bufs["sel"], stream)
    msa_sparse_prefill(shape, q, k, v, bufs["sel"], bufs["out"], bufs["lse"], None, 0, stream)


def run_decode(shape, q, k_cache, v_cache, idx_q, idx_k, bufs, stream=None):
    """One decode step into preallocated buffers (alloc_prefill_outputs + 'ws')."""
    msa_index_scores(shape, idx_q, idx_k, bufs["scores"], stream)
    msa_block_topk(shape, bufs["scores"], bufs["sel"], stream)
    msa_sparse_decode(shape, q, k_cache, v_cache, bufs["sel"], bufs["out"], bufs["lse"],
                      bufs["ws"], None, stream)


@dataclass(frozen=True)
class Rope:
    """Rotary positions of a model: frequencies of the main heads (int64 [rotary_dim / 2],
    turns per position in units of 2^-64 turns, see rope_freqs), of the index heads (None: the
    same), the factor on the rotated dims, and the pairing of the dims."""
    freqs: torch.Tensor
    index_freqs: torch.Tensor | None = None
    scale: float = 1.0
    interleaved: bool = False


def rope_freqs(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_len=0,
               ramp=(1.0, 32.0), device=None):
    """Frequencies base^(-2 i / rotary_dim) radians per position as a table for msa_rope, and
    the factor for the rotated dims: (int64 [rotary_dim / 2], scale).  For contexts `factor`
    times the trained length: scaling "linear" divides the positions, "ntk" raises the base so
    that the lowest frequency is divided by `factor`, "yarn" divides the frequencies that turn
    less than ramp[0] times in original_len positions, keeps those that turn more than ramp[1]
    times, ramps in between, and gives the scale 0.1 ln(factor) + 1."""
    if rotary_dim < 16 or rotary_dim % 16:
        raise ValueError(f"rotary_dim {rotary_dim} is not a multiple of 16")
    if not (factor >= 1.0 and math.isfinite(factor)) or not (base > 1.0 and math.isfinite(base)):
        raise ValueError("factor must be >= 1 and base > 1")
    scale = 1.0
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    turns = base ** (-i / rotary_dim) / (2 * math.pi)
    if scaling == "linear":
        turns = turns / factor
    elif scaling == "yarn":
        if original_len < 1 or not 0 < ramp[0] < ramp[1]:
            raise ValueError("yarn needs original_len >= 1 and an ascending ramp")
        keep = ((turns * original_len - ramp[0]) / (ramp[1] - ramp[0])).clamp(0, 1)
        turns = turns * keep + turns / factor * (1 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return (turns * 2.0 ** 64).to(torch.int64).to(device), scale


def rope(tensors, positions=None, pos_offset=0, scale=1.0, interleaved=False, inverse=False):
    """Rotates tensors that share their positions in one launch: rows (x, freqs, head_major),
    x [batch, seq, heads, d] or [batch, seq, d], or [batch, heads, seq, d] with head_major.
    Returns new tensors; inverse=True is the gradient of the same call without it."""
    rows = [(x, torch.empty_like(x), freqs, head_major) for x, freqs, head_major in tensors]
    x, _, _, head_major = rows[0]
    seq = x.shape[2] if head_major and x.dim() == 4 else x.shape[1]
    msa_rope(make_rope(x.shape[0], seq, _DT[x.dtype], pos_offset, scale, interleaved, inverse),
             make_rope_tensors(rows), positions)
    return [y for _, y, _, _ in rows]


def _rotate(rope_, q, k, idx_q, idx_k, pos_offset=0, positions=None):
    """The given tensors (None: left out) at positions pos_offset, pos_offset + 1, ..., or, one
    token a sequence, at pos_offset + positions [B]."""
    index = rope_.freqs if rope_.index_freqs is None else rope_.index_freqs
    rows = [(q, rope_.freqs, False), (k, rope_.freqs, True), (idx_q, index, False),
            (idx_k, index, False)]
    got = iter(rope([r for r in rows if r[0] is not None], positions, pos_offset, rope_.scale,
                    rope_.interleaved))
    return [None if r[0] is None else next(got) for r in rows]


def _check_positions(positions, rope_, batch):
    if positions is None:
        return
    if rope_ is None:
        raise ValueError("positions are those of a Rope, and rope is None")
    _check_shape(positions, "positions", (batch,))


def _check_shape(x, name, want):
    """A per-block array is indexed by its shape, so a larger one is not a longer one."""
    if x is not None and tuple(x.shape) != want:
        raise ValueError(f"{name} is {tuple(x.shape)}, expected {want}")


def prefill(q, k, v, idx_q, idx_k, block_size=128, top_k=16, q_tile=64, sm_scale=0.0,
            index_scale=0.0, rope=None):
    """MSA prefill.  q [B,T,Hq,d], k/v [B,Hkv,T,d], idx_q [B,T,Hkv,dI], idx_k [B,T,dI].
    With a Rope, q, k, idx_q and idx_k are rotated to positions 0 .. T-1 first (copies).

    Returns a dict with out [B,T,Hq,d], lse [B,Hq,T], scores and sel, and with a Rope the
    rotated keys for the caches (k, idx_k)."""
    shape = _shape_of(q, k, idx_q, block_size, top_k, q_tile, sm_scale, index_scale)
    bufs = alloc_prefill_outputs(shape, q.device, q.dtype)
    if rope is not None:
        q, k, idx_q, idx_k = _rotate(rope, q, k, idx_q, idx_k)
        bufs.update(k=k, idx_k=idx_k)
    run_prefill(shape, q, k, v, idx_q, idx_k, bufs)
    return bufs


def alloc_decode_outputs(shape, device, dtype, mass=False):
    """Outputs and workspace of a decode step (of msa_sparse_decode_mass with mass)."""
    bufs = alloc_prefill_outputs(shape, device, dtype)
    nbytes = max(16, msa_workspace_bytes(shape, 4 if mass else 1))
    bufs["ws"] = torch.empty((nbytes + 15) // 16 * 4, device=device, dtype=torch.float32)
    return bufs


def decode(q, k_cache, v_cache, idx_q, idx_k, block_size=128, top_k=64, sm_scale=0.0,
           index_scale=0.0, rope=None, mass=None, positions=None):
    """One MSA decode step.  q [B,1,Hq,d], caches [B,Hkv,L,d], idx_q [B,1,Hkv,dI],
    idx_k [B,L,dI]; the new token is the last of the caches' L and already in them.  With a
    Rope, q and idx_q are rotated (the caches hold rotated keys) to positions (int32 [B]: the
    new tokens' absolute positions), or without them to L-1.  That is right while nothing has
    been evicted: the keys that evict leaves stay rotated to the positions they had, so after it
    the positions go on counting from where they were, past L.  With mass (float32
    [B,Hkv,blocks]) the attention weight of every selected block is added to it."""
    shape = _shape_of(q, k_cache, idx_q, block_size, top_k, 1, sm_scale, index_scale)
    _check_shape(mass, "mass", (shape.batch, shape.n_heads_kv, shape.n_blocks))
    _check_positions(positions, rope, shape.batch)
    bufs = alloc_decode_outputs(shape, q.device, q.dtype, mass is not None)
    if rope is not None:
        q, _, idx_q, _ = _rotate(rope, q, None, idx_q, None,
                                 shape.seq_k - 1 if positions is None else 0, positions)
    if mass is None:
        run_decode(shape, q, k_cache, v_cache, idx_q, idx_k, bufs)
    else:
        msa_index_scores(shape, idx_q, idx_k, bufs["scores"])
        msa_block_topk(shape, bufs["scores"], bufs["sel"])
        msa_sparse_decode_mass(shape, None, None, 0, q, k_cache, v_cache, bufs["sel"], bufs["out"],
                               bufs["lse"], mass, bufs["ws"])
    return bufs


def _check_step(x, name, rows, numel, dtype, dev):
    """What a call would refuse a tensor for, ahead of the step's first launch."""
    if _lib._arg(x, name, dtype, numel, dev, rows) % 16:
        raise ValueError(f"{name} is not 16-byte aligned")


def alloc_packed_cache(n_phys, n_heads_kv, head_dim, device="cuda"):
    """A 4-bit cache of n_phys blocks of 128 keys (layout in include/msa.h)."""
    return torch.zeros((n_phys, n_heads_kv, 160 * head_dim), dtype=torch.uint8, device=device)


def decode_packed(q, k, v, cache, idx_q, idx_k_pool, seq_lens, block_table, capacity, top_k=64,
                  sm_scale=0.0, index_scale=0.0, rope=None, mass=None, positions=None):
    """One MSA decode step over a paged cache whose K and V are held in 4 bits.  q [B,1,Hq,d];
    k, v [B,Hkv,1,d]: the new token's rows, packed into the cache as its row seq_lens - 1;
    cache from alloc_packed_cache; idx_q [B,1,Hkv,128]; idx_k_pool [P,128,128] 16-bit index keys
    (rotated, the new token's among them); seq_lens int32 [B] (the new token counted);
    block_table int32 [B, ceil(capacity / 128)].  With a Rope, q, k and idx_q are rotated first,
    to positions (int32 [B]: the new tokens' absolute positions), or without them to
    seq_lens - 1.  That is right while nothing has been evicted: evict_paged shortens seq_lens,
    but the keys that stay are rotated to the positions they had, so positions are then a count
    of its own that evictions leave alone.  With mass, the blocks' attention weights are added
    to it (top_k at most 1024).

    The paged index scores set the step's limits: bf16, head_dim 128, 4 KV heads, at most 16
    query heads per KV head.  (msa_cache_pack and msa_sparse_decode_packed take more, with a
    selection from elsewhere.)  A step that is refused has not changed the cache."""
    B, _, Hq, d = q.shape
    Hkv, n_phys = cache.shape[1], cache.shape[0]
    shape = make_shape(B, 1, capacity, Hq, Hkv, d, idx_q.shape[-1], 128, top_k, 1, _DT[q.dtype],
                       sm_scale, index_scale)
    if q.dtype is not torch.bfloat16 or d != 128 or idx_q.shape[-1] != 128 or Hkv != 4 or Hq > 64:
        raise _lib.MsaError(_lib.MSA_ERR_UNSUPPORTED, "decode_packed",
                            "a step over the 4-bit cache runs bf16, head_dim = index_dim = 128, 4 KV "
                            "heads, at most 16 query heads per KV head")
    if mass is not None and top_k > 1024:
        raise _lib.MsaError(_lib.MSA_ERR_UNSUPPORTED, "decode_packed", "mass needs top_k <= 1024")
    _check_shape(block_table, "block_table", (B, shape.n_blocks))
    _check_shape(idx_k_pool, "idx_k_pool", (n_phys, 128, idx_q.shape[-1]))
    _check_shape(mass, "mass", (B, Hkv, shape.n_blocks))
    _check_positions(positions, rope, B)
    # packing checks its own arguments ahead of its launch; these are those of the calls after it
    dev = _lib._place(None)[0]
    _check_step(q, "q", B, B * Hq * d, q.dtype, dev)
    _check_step(idx_q, "idx_q", B, B * Hkv * d, q.dtype, dev)
    _check_step(idx_k_pool, "idx_k_pool", n_phys, n_phys * 128 * d, q.dtype, dev)
    if mass is not None:
        _check_step(mass, "mass", B, B * Hkv * shape.n_blocks, torch.float32, dev)
    bufs = alloc_prefill_outputs(shape, q.device, q.dtype)
    if rope is not None:
        index = rope.freqs if rope.index_freqs is None else rope.index_freqs
        rows = [(x, torch.empty_like(x), f, h)
                for x, f, h in ((q, rope.freqs, False), (k, rope.freqs, True), (idx_q, index, False))]
        msa_rope(make_rope(B, 1, _DT[q.dtype], -1 if positions is None else 0, rope.scale,
                           rope.interleaved), make_rope_tensors(rows),
                 seq_lens if positions is None else positions)
        q, k, idx_q = (y for _, y, _, _ in rows)
    msa_cache_pack(shape, 1, None, seq_lens, block_table, n_phys, k, v, cache)
    msa_index_scores_paged(shape, seq_lens, block_table, n_phys, idx_q, idx_k_pool, bufs["scores"])
    msa_block_topk_ragged(shape, seq_lens, bufs["scores"], bufs["sel"])
    msa_sparse_decode_packed(shape, seq_lens, block_table, n_phys, q, cache, bufs["sel"],
                             bufs["out"], bufs["lse"], mass)
    return bufs


def evict_paged(seq_lens, mass, block_table, capacity, keep, n_first=1, n_recent=2, block_size=128):
    """Cuts every sequence of a paged cache to at most `keep` blocks, in place: seq_lens, mass
    [B,Hkv,blocks] and block_table are updated (the dropped physical blocks follow the kept
    ones in the table).  Returns kept int32 [B, keep], the old indices of what stays.  Keys keep
    their rotation: later steps with a Rope need positions that did not shrink with seq_lens."""
    B, Hkv, _ = mass.shape
    shape = make_shape(B, 1, capacity, Hkv, Hkv, 128, 128, block_size, 1, 1)
    _check_shape(mass, "mass", (B, Hkv, shape.n_blocks))
    _check_shape(block_table, "block_table", (B, shape.n_blocks))
    kept = torch.empty((B, keep), dtype=torch.int32, device=mass.device)
    msa_cache_evict(shape, keep, n_first, n_recent, seq_lens, mass, block_table, kept, seq_lens,
                    mass, block_table)
    return kept


def evict(k_cache, v_cache, idx_k, mass, keep, n_first=1, n_recent=2, block_size=128):
    """Cuts contiguous caches (k, v [B,Hkv,L,d], idx_k [B,L,dI]) to at most `keep` blocks.
    Returns a dict with the shorter caches k, v, idx_k, their mass, and kept int32 [B, keep].
    Keys keep their rotation: later steps with a Rope need positions that go on from L."""
    B, Hkv, L, d = k_cache.shape
    shape = make_shape(B, 1, L, Hkv, Hkv, d, 128, block_size, 1, 1)
    n = shape.n_blocks
    _check_shape(mass, "mass", (B, Hkv, n))
    if tuple(v_cache.shape[:-1]) != (B, Hkv, L):
        raise ValueError(f"v_cache is {tuple(v_cache.shape)}, expected {(B, Hkv, L, d)}")
    if idx_k.dim() != 3 or tuple(idx_k.shape[:2]) != (B, L):
        raise ValueError(f"idx_k is {tuple(idx_k.shape)}, expected {(B, L, 'dI')}")
    rows = L - (n - min(n, keep)) * block_size
    new = lambda x: torch.empty((*x.shape[:-2], rows, x.shape[-1]), dtype=x.dtype, device=x.device)  # noqa: E731
    kept = torch.empty((B, keep), dtype=torch.int32, device=mass.device)
    lens = torch.empty((B,), dtype=torch.int32, device=mass.device)
    out = torch.empty_like(mass)
    msa_cache_evict(shape, keep, n_first, n_recent, None, mass, None, kept, lens, out)
    pairs = [(x, new(x)) for x in (k_cache, v_cache, idx_k)]
    msa_cache_gather(B, make_gather_tensors(pairs), kept, block_size)
    blocks = -(-rows // block_size)
    return dict(k=pairs[0][1], v=pairs[1][1], idx_k=pairs[2][1],
                mass=out[:, :, :blocks].contiguous(), kept=kept)


__all__ = ["prefill", "decode", "run_prefill", "run_decode", "alloc_prefill_outputs",
           "alloc_decode_outputs", "Rope", "rope", "rope_freqs", "alloc_packed_cache",
           "decode_packed", "evict", "evict_paged", "_lib"]
