"""ctypes binding of libmsa.so: the C ABI in include/msa.h, argument marshalling only.

Every computation runs in the library's CUDA kernels.  Tensors are passed as raw device
pointers (``tensor.data_ptr()``) together with the current torch CUDA stream; a missing
library or CUDA device raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import threading

(MSA_OK, MSA_ERR_INVALID_ARG, MSA_ERR_UNSUPPORTED, MSA_ERR_CUDA, MSA_ERR_TIMEOUT,
 MSA_ERR_BOUNDS) = range(6)
MSA_F32, MSA_BF16 = 0, 1
_DTYPE_CODES = {"f32": MSA_F32, "bf16": MSA_BF16}

# Every function include/msa.h declares, with its ctypes signature.
_vp, _i32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t


class MsaShape(ctypes.Structure):
    """Mirror of ``msa_shape``."""
    _fields_ = [("batch", _i32), ("seq_q", _i32), ("seq_k", _i32), ("n_heads_q", _i32),
                ("n_heads_kv", _i32), ("head_dim", _i32), ("index_dim", _i32),
                ("block_size", _i32), ("top_k", _i32), ("q_tile", _i32), ("dtype", _i32),
                ("sm_scale", ctypes.c_float), ("index_scale", ctypes.c_float)]

    @property
    def n_blocks(self) -> int:
        return -(-self.seq_k // self.block_size)

    @property
    def n_rows(self) -> int:
        return -(-self.seq_q // self.q_tile)

    def __repr__(self):
        return "MsaShape(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class MsaRope(ctypes.Structure):
    """Mirror of ``msa_rope_desc``."""
    _fields_ = [("batch", _i32), ("seq", _i32), ("dtype", _i32), ("pos_offset", _i32),
                ("interleaved", _i32), ("inverse", _i32), ("scale", ctypes.c_float)]


class MsaRopeTensor(ctypes.Structure):
    """Mirror of ``msa_rope_tensor``."""
    _fields_ = [("x", _vp), ("y", _vp), ("freqs", _vp), ("n_heads", _i32), ("head_dim", _i32),
                ("rotary_dim", _i32), ("head_major", _i32)]


class MsaCommitTensor(ctypes.Structure):
    """Mirror of ``msa_commit_tensor``."""
    _fields_ = [("src", _vp), ("dst", _vp), ("n_heads", _i32), ("row_bytes", _i32),
                ("packed", _i32)]


class MsaGatherTensor(ctypes.Structure):
    """Mirror of ``msa_gather_tensor``."""
    _fields_ = [("src", _vp), ("dst", _vp), ("src_rows", ctypes.c_int64),
                ("dst_rows", ctypes.c_int64), ("n_heads", _i32), ("row_bytes", _i32)]


_SHAPE_P = ctypes.POINTER(MsaShape)
SIGNATURES = {
    "msa_index_scores": (_i32, [_SHAPE_P, _vp, _vp, _vp, _vp]),
    "msa_block_topk": (_i32, [_SHAPE_P, _vp, _vp, _vp]),
    "msa_index_topk_fused": (_i32, [_SHAPE_P, _vp, _vp, _vp, _vp, _vp]),
    "msa_block_topk_shared": (_i32, [_SHAPE_P, _vp, _vp, _vp]),
    "msa_sparse_prefill": (_i32, [_SHAPE_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "msa_sparse_decode": (_i32, [_SHAPE_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "msa_sparse_prefill_backward": (_i32, [_SHAPE_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                           _vp, _vp, _vp, _sz, _vp]),
    "msa_index_kl_loss": (_i32, [_SHAPE_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _sz, _vp]),
    "msa_sparse_decode_static": (_i32, [_SHAPE_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "msa_index_scores_paged": (_i32, [_SHAPE_P, _vp, _vp, _i32, _vp, _vp, _vp, _vp]),
    "msa_block_topk_ragged": (_i32, [_SHAPE_P, _vp, _vp, _vp, _vp]),
    "msa_sparse_decode_paged": (_i32, [_SHAPE_P, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _vp, _sz, _vp]),
    "msa_rope": (_i32, [ctypes.POINTER(MsaRope), ctypes.POINTER(MsaRopeTensor), _i32, _vp, _vp]),
    "msa_cache_pack": (_i32, [_SHAPE_P, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp]),
    "msa_cache_unpack": (_i32, [_SHAPE_P, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp]),
    "msa_sparse_decode_packed": (_i32, [_SHAPE_P, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                        _vp]),
    "msa_sparse_decode_mass": (_i32, [_SHAPE_P, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _sz, _vp]),
    "msa_cache_evict": (_i32, [_SHAPE_P, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                               _vp]),
    "msa_cache_gather": (_i32, [_i32, ctypes.POINTER(MsaGatherTensor), _i32, _vp, _i32, _i32,
                                _vp]),
    "msa_tree_mask": (_i32, [_SHAPE_P, _vp, _vp, _vp, _vp, _vp]),
    "msa_index_pack": (_i32, [_SHAPE_P, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp]),
    "msa_index_unpack": (_i32, [_SHAPE_P, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp]),
    "msa_index_scores_tree": (_i32, [_SHAPE_P, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp,
                                     _vp]),
    "msa_block_topk_tree": (_i32, [_SHAPE_P, _vp, _vp, _vp, _vp, _vp]),
    "msa_sparse_decode_tree": (_i32, [_SHAPE_P, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _vp, _vp, _sz, _vp]),
    "msa_tree_commit": (_i32, [_SHAPE_P, _vp, _vp, _i32, _vp, _i32,
                               ctypes.POINTER(MsaCommitTensor), _i32, _vp, _vp]),
    "msa_tree_commit_masked": (_i32, [_SHAPE_P, _vp, _vp, _i32, _vp, _vp, _i32,
                                      ctypes.POINTER(MsaCommitTensor), _i32, _vp, _vp]),
    "msa_workspace_bytes": (_sz, [_SHAPE_P, ctypes.c_int]),
    "msa_get_device_status": (_i32, [_vp]),
    "msa_status_string": (ctypes.c_char_p, [_i32]),
    "msa_last_error": (ctypes.c_char_p, []),
    "msa_abi_version": (_i32, []),
    "msa_debug_build": (_i32, []),
    "msa_debug_set_fault": (_i32, [_i32]),
}

_lock = threading.Lock()
_libs = {}                 # variant -> loaded library
# The variant the calls below go through: "release" (libmsa.so), or "debug"
# (libmsa_debug.so, built with the device-side index checks) when the environment sets
# MSA_LIBRARY_VARIANT=debug.  A process loads one variant: the two libraries export the same
# symbols and device variables.
_active = os.environ.get("MSA_LIBRARY_VARIANT", "release")


class MsaError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({detail})")


def library_path(variant: str = "release") -> str:
    name = "libmsa.so" if variant == "release" else f"libmsa_{variant}.so"
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), name)


def load(build_if_missing: bool = True, variant: str | None = None):
    """The loaded library of `variant` (default: the process's variant, see
    MSA_LIBRARY_VARIANT), built in-tree with nvcc on first use if needed."""
    variant = _active if variant is None else variant
    if variant in _libs:
        return _libs[variant]
    if variant not in ("release", "debug"):
        raise ValueError(f"unknown MSA library variant {variant!r}")
    with _lock:
        if _libs and variant not in _libs:
            raise RuntimeError(f"the {next(iter(_libs))} MSA library is already loaded in this "
                               f"process; run the {variant} variant in a process of its own")
        if variant not in _libs:
            path = library_path(variant)
            if build_if_missing:
                from . import build as _build
                path = _build.build(variant=variant)
            if not os.path.exists(path):
                raise RuntimeError(f"MSA CUDA library missing at {path}; run the build first")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _libs[variant] = lib
        return _libs[variant]


def _ptr(x):
    """Device pointer of a tensor (must be contiguous), an int, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_contiguous():
        raise ValueError("MSA tensors must be contiguous")
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        return (_torch or _get_torch()).cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != MSA_OK:
        lib = load()
        detail = (lib.msa_last_error() or b"").decode() or \
            (lib.msa_status_string(status) or b"").decode()
        raise MsaError(status, where, detail)


def make_shape(batch, seq_q, seq_k, n_heads_q, n_heads_kv, head_dim, index_dim, block_size,
               top_k, q_tile, dtype="bf16", sm_scale=0.0, index_scale=0.0) -> MsaShape:
    code = _DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    return MsaShape(batch, seq_q, seq_k, n_heads_q, n_heads_kv, head_dim, index_dim,
                    block_size, top_k, q_tile, code, sm_scale, index_scale)


def shape_from_config(cfg, **override) -> MsaShape:
    kw = dict(batch=cfg.batch, seq_q=cfg.seq_q, seq_k=cfg.seq_k, n_heads_q=cfg.n_heads_q,
              n_heads_kv=cfg.n_heads_kv, head_dim=cfg.head_dim, index_dim=cfg.index_dim,
              block_size=cfg.block_size, top_k=cfg.top_k, q_tile=cfg.q_tile, dtype=cfg.dtype)
    kw.update(override)
    return make_shape(**kw)


# ------------------------------------------------------------- the C-ABI calls

def msa_index_scores(shape: MsaShape, idx_q, idx_k, block_scores, stream=None):
    _check(load().msa_index_scores(ctypes.byref(shape), _ptr(idx_q), _ptr(idx_k),
                                   _ptr(block_scores), _stream(stream)), "msa_index_scores")


def msa_block_topk(shape: MsaShape, block_scores, sel, stream=None):
    _check(load().msa_block_topk(ctypes.byref(shape), _ptr(block_scores), _ptr(sel),
                                 _stream(stream)), "msa_block_topk")


def msa_block_topk_shared(shape: MsaShape, block_scores, sel, stream=None):
    """Ablation: one selection per row from the KV heads' summed scores, shared by all heads."""
    _check(load().msa_block_topk_shared(ctypes.byref(shape), _ptr(block_scores), _ptr(sel),
                                        _stream(stream)), "msa_block_topk_shared")


def msa_index_topk_fused(shape: MsaShape, idx_q, idx_k, sel, block_scores=None, stream=None):
    _check(load().msa_index_topk_fused(ctypes.byref(shape), _ptr(idx_q), _ptr(idx_k),
                                       _ptr(block_scores), _ptr(sel), _stream(stream)),
           "msa_index_topk_fused")


def msa_sparse_prefill(shape: MsaShape, q, k, v, sel, out, lse=None, workspace=None,
                       ws_bytes=0, stream=None):
    _check(load().msa_sparse_prefill(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(sel),
                                     _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
                                     _stream(stream)), "msa_sparse_prefill")


def msa_sparse_prefill_backward(shape: MsaShape, q, k, v, sel, out, lse, dout, dq, dk, dv,
                                workspace=None, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().msa_sparse_prefill_backward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                              _ptr(sel), _ptr(out), _ptr(lse), _ptr(dout),
                                              _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
                                              ws_bytes, _stream(stream)),
           "msa_sparse_prefill_backward")


def msa_index_kl_loss(shape: MsaShape, q, k, lse, idx_q, idx_k, sel, loss, d_idx_q, d_idx_k,
                      workspace=None, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().msa_index_kl_loss(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(lse),
                                    _ptr(idx_q), _ptr(idx_k), _ptr(sel), _ptr(loss),
                                    _ptr(d_idx_q), _ptr(d_idx_k), _ptr(workspace), ws_bytes,
                                    _stream(stream)),
           "msa_index_kl_loss")


def msa_sparse_decode(shape: MsaShape, q, k_cache, v_cache, sel, out, lse=None, workspace=None,
                      ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().msa_sparse_decode(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(sel), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
                                    _stream(stream)), "msa_sparse_decode")


def msa_sparse_decode_static(shape: MsaShape, q, k_cache, v_cache, sel, out, lse=None,
                             stream=None):
    """msa_sparse_decode without a caller workspace: for callers that cannot allocate
    device memory where decode runs, the library's own static device scratch is used."""
    _check(load().msa_sparse_decode_static(ctypes.byref(shape), _ptr(q), _ptr(k_cache),
                                           _ptr(v_cache), _ptr(sel), _ptr(out), _ptr(lse),
                                           _stream(stream)), "msa_sparse_decode_static")


def msa_index_scores_paged(shape: MsaShape, seq_lens, block_table, n_phys, idx_q, idx_k_pool,
                           block_scores, stream=None):
    _check(load().msa_index_scores_paged(ctypes.byref(shape), _ptr(seq_lens), _ptr(block_table),
                                         int(n_phys), _ptr(idx_q), _ptr(idx_k_pool),
                                         _ptr(block_scores), _stream(stream)),
           "msa_index_scores_paged")


def msa_block_topk_ragged(shape: MsaShape, seq_lens, block_scores, sel, stream=None):
    _check(load().msa_block_topk_ragged(ctypes.byref(shape), _ptr(seq_lens), _ptr(block_scores),
                                        _ptr(sel), _stream(stream)), "msa_block_topk_ragged")


def msa_sparse_decode_paged(shape: MsaShape, seq_lens, block_table, n_phys, q, k_pool, v_pool,
                            sel, out, lse=None, workspace=None, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().msa_sparse_decode_paged(ctypes.byref(shape), _ptr(seq_lens), _ptr(block_table),
                                          int(n_phys), _ptr(q), _ptr(k_pool), _ptr(v_pool),
                                          _ptr(sel), _ptr(out), _ptr(lse), _ptr(workspace),
                                          ws_bytes, _stream(stream)), "msa_sparse_decode_paged")


# ----------------------------- rotary positions, the 4-bit cache, eviction by weight

_torch = _I32 = _I64 = _U8 = _F32 = None
_FLOATS = {}               # msa_dtype -> torch dtype


def _get_torch():
    global _torch, _I32, _I64, _U8, _F32
    if _torch is None:
        import torch
        _FLOATS.update({MSA_F32: torch.float32, MSA_BF16: torch.bfloat16})
        _I32, _I64, _U8, _F32 = torch.int32, torch.int64, torch.uint8, torch.float32
        _torch = torch
    return _torch


def _device():
    """The current CUDA device (initialising CUDA), or -2, no tensor's, on a machine without."""
    torch = _torch or _get_torch()
    return torch.cuda.current_device() if torch.cuda.is_available() else -2


_fast = []                 # torch's raw device and stream getters, once CUDA is in use


def _place(stream):
    """The current device, and the raw stream: the given one or torch's current one."""
    if _fast:
        dev = _fast[0]()
        if stream is None:
            return dev, _fast[1](dev)
    else:
        dev = _device()
        if dev >= 0:
            c = _torch._C
            if hasattr(c, "_cuda_getDevice") and hasattr(c, "_cuda_getCurrentRawStream"):
                _fast.extend((c._cuda_getDevice, c._cuda_getCurrentRawStream))
        elif stream is None:
            return dev, 0
    return dev, _stream(stream)


def _arg(x, name, dtype, numel, dev, rows=0):
    """Device pointer of a tensor that must be contiguous, of `dtype` (None: any) and at least
    `numel` elements, and on device `dev`; of an int (a raw pointer) or None as they are.
    rows: the entries of the first axis that the call indexes.  A longer first axis (or a flat
    buffer) has the call's elements at its start; with any other axis longer every row but the
    first would be read in the wrong place."""
    if x is None or type(x) is int:
        return x
    if numel and x.numel() != numel:
        _check_size(x, name, numel, rows)
    if x.get_device() != dev:
        raise ValueError(f"{name} is on {x.device}, not on the current CUDA device")
    if dtype is not None and x.dtype is not dtype:
        raise ValueError(f"{name} is {x.dtype}, expected {dtype}")
    if not x.is_contiguous():
        raise ValueError(f"{name}: MSA tensors must be contiguous")
    return x.data_ptr()


def _check_size(x, name, numel, rows):
    n = x.numel()
    if rows and x.dim() > 1 and n * rows != numel * x.shape[0]:
        raise ValueError(f"{name} is {tuple(x.shape)}: {n} elements, expected {numel} in {rows} rows")
    if n < numel:
        raise ValueError(f"{name} has {n} elements, expected {numel}")


def make_rope(batch, seq, dtype="bf16", pos_offset=0, scale=0.0, interleaved=False,
              inverse=False) -> MsaRope:
    """The description of a msa_rope call (see include/msa.h; scale 0 means 1)."""
    code = _DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    return MsaRope(batch, seq, code, pos_offset, int(interleaved), int(inverse), scale)


class RopeTensors:
    """The tensors of a msa_rope call: rows (x, y, freqs, head_major) with x and y
    [batch, seq, heads, d] (or [batch, seq, d], one head), or [batch, heads, seq, d] with
    head_major; freqs int64 [rotary_dim / 2].  Holds the tensors, and may be kept and used for
    every call on them."""

    def __init__(self, rows):
        rows = list(rows)
        self.device = dev = _device()
        self.rows = rows
        self.array = (MsaRopeTensor * max(1, len(rows)))()
        self.batch = self.seq = self.dtype = None
        for i, (x, y, freqs, head_major) in enumerate(rows):
            if x.dim() not in (3, 4) or y.shape != x.shape or y.dtype != x.dtype:
                raise ValueError(f"rope tensor {i}: x and y need the same [batch, seq, (heads,) d] "
                                 f"shape and type, got {tuple(x.shape)} and {tuple(y.shape)}")
            head_major = bool(head_major) and x.dim() == 4
            heads = 1 if x.dim() == 3 else x.shape[1 if head_major else 2]
            this = x.shape[0], x.shape[2 if head_major else 1], x.dtype
            if i and this != (self.batch, self.seq, self.dtype):
                raise ValueError(f"rope tensor {i} has (batch, seq, dtype) {this}, the others "
                                 f"{(self.batch, self.seq, self.dtype)}")
            self.batch, self.seq, self.dtype = this
            self.array[i] = MsaRopeTensor(
                _arg(x, f"x of rope tensor {i}", None, 0, dev),
                _arg(y, f"y of rope tensor {i}", None, 0, dev),
                _arg(freqs, f"freqs of rope tensor {i}", _I64, 0, dev), heads, x.shape[-1],
                2 * freqs.numel(), int(head_major))

    def __len__(self):
        return len(self.rows)


def make_rope_tensors(rows) -> RopeTensors:
    return RopeTensors(rows)


def msa_rope(desc: MsaRope, tensors: RopeTensors, positions=None, stream=None):
    dev, st = _place(stream)
    batch, seq = desc.batch, desc.seq
    if tensors.device != dev:
        raise ValueError(f"the rope tensors are on CUDA device {tensors.device}, the current one "
                         f"is {dev}")
    if tensors.rows and (tensors.batch != batch or tensors.seq != seq or
                         tensors.dtype is not _FLOATS.get(desc.dtype)):
        raise ValueError(f"the rope tensors have (batch, seq, dtype) "
                         f"{(tensors.batch, tensors.seq, tensors.dtype)}, the call "
                         f"{(batch, seq, _FLOATS.get(desc.dtype))}")
    _check(load().msa_rope(ctypes.byref(desc), tensors.array, len(tensors.rows),
                           _arg(positions, "positions", _I32, batch * seq, dev, batch), st), "msa_rope")


def _cache_args(shape, batch, hkv, d, seq_lens, block_table, n_phys, cache, dev):
    return (_arg(seq_lens, "seq_lens", _I32, batch, dev, batch),
            block_table if block_table is None else
            _arg(block_table, "block_table", _I32, batch * shape.n_blocks, dev, batch), n_phys,
            _arg(cache, "cache", _U8, n_phys * hkv * 160 * d, dev, n_phys))


def _cache_rows(call, where, shape, n, starts, seq_lens, block_table, n_phys, cache, k, v, stream):
    """The arguments of pack (cache last) and unpack (cache before k and v)."""
    dev, st = _place(stream)
    n, n_phys = int(n), int(n_phys)
    batch, hkv, d, dt = shape.batch, shape.n_heads_kv, shape.head_dim, _FLOATS.get(shape.dtype)
    rows = batch * hkv * n * d
    args = _cache_args(shape, batch, hkv, d, seq_lens, block_table, n_phys, cache, dev)
    kv = _arg(k, "k", dt, rows, dev, batch), _arg(v, "v", dt, rows, dev, batch)
    tail = kv + args[3:] if where == "msa_cache_pack" else args[3:] + kv
    _check(call(ctypes.byref(shape), n, _arg(starts, "starts", _I32, batch, dev, batch), *args[:3],
                *tail, st), where)


def msa_cache_pack(shape: MsaShape, n_new, starts, seq_lens, block_table, n_phys, k, v, cache,
                   stream=None):
    _cache_rows(load().msa_cache_pack, "msa_cache_pack", shape, n_new, starts, seq_lens,
                block_table, n_phys, cache, k, v, stream)


def msa_cache_unpack(shape: MsaShape, n_out, starts, seq_lens, block_table, n_phys, cache, k, v,
                     stream=None):
    _cache_rows(load().msa_cache_unpack, "msa_cache_unpack", shape, n_out, starts, seq_lens,
                block_table, n_phys, cache, k, v, stream)


def _decode_args(shape, batch, hkv, d, dt, q, sel, out, lse, mass, dev):
    hq = shape.n_heads_q
    n = batch * hq * d
    return (_arg(q, "q", dt, n, dev, batch),
            _arg(sel, "sel", _I32, batch * hkv * shape.top_k, dev, batch),
            _arg(out, "out", dt, n, dev, batch), _arg(lse, "lse", _F32, batch * hq, dev, batch),
            mass if mass is None else
            _arg(mass, "mass", _F32, batch * hkv * shape.n_blocks, dev, batch))


def msa_sparse_decode_packed(shape: MsaShape, seq_lens, block_table, n_phys, q, cache, sel, out,
                             lse=None, mass=None, stream=None):
    dev, st = _place(stream)
    batch, hkv, d = shape.batch, shape.n_heads_kv, shape.head_dim
    sl, bt, n_phys, c = _cache_args(shape, batch, hkv, d, seq_lens, block_table, int(n_phys), cache,
                                    dev)
    q, sel, out, lse, mass = _decode_args(shape, batch, hkv, d, _FLOATS.get(shape.dtype), q, sel,
                                          out, lse, mass, dev)
    _check(load().msa_sparse_decode_packed(ctypes.byref(shape), sl, bt, n_phys, q, c, sel, out,
                                           lse, mass, st), "msa_sparse_decode_packed")


def msa_sparse_decode_mass(shape: MsaShape, seq_lens, block_table, n_phys, q, k, v, sel, out, lse,
                           mass, workspace, ws_bytes=None, stream=None):
    dev, st = _place(stream)
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    n_phys = int(n_phys)
    batch, hkv, d, dt = shape.batch, shape.n_heads_kv, shape.head_dim, _FLOATS.get(shape.dtype)
    paged = block_table is not None
    n = (n_phys * shape.block_size if paged else batch * shape.seq_k) * hkv * d
    rows = n_phys if paged else batch
    q, sel, out, lse, mass = _decode_args(shape, batch, hkv, d, dt, q, sel, out, lse, mass, dev)
    _check(load().msa_sparse_decode_mass(
        ctypes.byref(shape), _arg(seq_lens, "seq_lens", _I32, batch, dev, batch),
        _arg(block_table, "block_table", _I32, batch * shape.n_blocks, dev, batch) if paged else None,
        n_phys, q, _arg(k, "k", dt, n, dev, rows), _arg(v, "v", dt, n, dev, rows), sel, out, lse, mass,
        _arg(workspace, "workspace", None, 0, dev), ws_bytes, st), "msa_sparse_decode_mass")


def msa_cache_evict(shape: MsaShape, keep, n_first, n_recent, seq_lens, mass, block_table, kept,
                    new_lens, mass_out, table_out=None, stream=None):
    dev, st = _place(stream)
    keep, batch = int(keep), shape.batch
    n = batch * shape.n_blocks
    m = n * shape.n_heads_kv
    _check(load().msa_cache_evict(
        ctypes.byref(shape), keep, int(n_first), int(n_recent),
        _arg(seq_lens, "seq_lens", _I32, batch, dev, batch), _arg(mass, "mass", _F32, m, dev, batch),
        _arg(block_table, "block_table", _I32, n, dev, batch),
        _arg(kept, "kept", _I32, batch * keep, dev, batch),
        _arg(new_lens, "new_lens", _I32, batch, dev, batch),
        _arg(mass_out, "mass_out", _F32, m, dev, batch),
        _arg(table_out, "table_out", _I32, n, dev, batch), st), "msa_cache_evict")


class GatherTensors:
    """The caches of a msa_cache_gather call: rows (src, dst), each [batch, heads, rows, ...]
    or [batch, rows, d] (one head).  Holds the tensors, and may be kept and used for every call
    on them."""

    def __init__(self, rows):
        rows = list(rows)
        self.device = dev = _device()
        self.rows = rows
        self.array = (MsaGatherTensor * max(1, len(rows)))()
        self.batches = []
        for i, (src, dst) in enumerate(rows):
            lead = 1 if src.dim() == 3 else 2
            if src.dim() not in (3, 4) or dst.dim() != src.dim() or dst.dtype != src.dtype or \
                    dst.shape[:lead] != src.shape[:lead] or dst.shape[-1] != src.shape[-1]:
                raise ValueError(f"gather tensor {i}: src and dst differ in more than their rows: "
                                 f"{tuple(src.shape)} and {tuple(dst.shape)}")
            self.array[i] = MsaGatherTensor(
                _arg(src, f"src of gather tensor {i}", None, 0, dev),
                _arg(dst, f"dst of gather tensor {i}", None, 0, dev),
                src.shape[lead], dst.shape[lead], 1 if lead == 1 else src.shape[1],
                src.shape[-1] * src.element_size())
            self.batches.append(src.shape[0])

    def __len__(self):
        return len(self.rows)


def make_gather_tensors(rows) -> GatherTensors:
    return GatherTensors(rows)


def msa_cache_gather(batch, tensors: GatherTensors, kept, block_size=128, stream=None):
    dev, st = _place(stream)
    if tensors.device != dev:
        raise ValueError(f"the gather tensors are on CUDA device {tensors.device}, the current one "
                         f"is {dev}")
    for i, n in enumerate(tensors.batches):
        if n != batch:
            raise ValueError(f"gather tensor {i} has batch {n}, the call {batch}")
    if kept.dim() != 2 or kept.shape[0] != batch:
        raise ValueError(f"kept is {tuple(kept.shape)}, expected [{batch}, keep]")
    _check(load().msa_cache_gather(int(batch), tensors.array, len(tensors),
                                   _arg(kept, "kept", _I32, 0, dev), kept.shape[1], int(block_size),
                                   st), "msa_cache_gather")


# ------------------------------------------- decode over a tree of drafted tokens

def msa_tree_mask(shape: MsaShape, seq_lens, parents, mask, positions=None, stream=None):
    """mask: int64 [batch, tokens] (its bits are the library's 64-bit words)."""
    dev, st = _place(stream)
    batch = shape.batch
    n = batch * shape.seq_q
    _check(load().msa_tree_mask(
        ctypes.byref(shape), _arg(seq_lens, "seq_lens", _I32, batch, dev, batch),
        _arg(parents, "parents", _I32, n, dev, batch), _arg(mask, "mask", _I64, n, dev, batch),
        _arg(positions, "positions", _I32, n, dev, batch), st), "msa_tree_mask")


def _index_rows(call, where, shape, n, starts, seq_lens, block_table, n_phys, cache, x, stream):
    """The arguments of index packing (cache last) and unpacking (cache before the rows)."""
    dev, st = _place(stream)
    n, n_phys = int(n), int(n_phys)
    batch, d = shape.batch, shape.index_dim
    c = _arg(cache, "cache", _U8, n_phys * 128 * (d + 1), dev, n_phys)
    rows = _arg(x, "x", _FLOATS.get(shape.dtype), batch * n * d, dev, batch)
    _check(call(ctypes.byref(shape), n, _arg(starts, "starts", _I32, batch, dev, batch),
                _arg(seq_lens, "seq_lens", _I32, batch, dev, batch),
                _arg(block_table, "block_table", _I32, batch * shape.n_blocks, dev, batch), n_phys,
                *((rows, c) if where == "msa_index_pack" else (c, rows)), st), where)


def msa_index_pack(shape: MsaShape, n_new, starts, seq_lens, block_table, n_phys, x, cache,
                   stream=None):
    _index_rows(load().msa_index_pack, "msa_index_pack", shape, n_new, starts, seq_lens, block_table,
                n_phys, cache, x, stream)


def msa_index_unpack(shape: MsaShape, n_out, starts, seq_lens, block_table, n_phys, cache, y,
                     stream=None):
    _index_rows(load().msa_index_unpack, "msa_index_unpack", shape, n_out, starts, seq_lens,
                block_table, n_phys, cache, y, stream)


def _tree_cache(shape, x, name, lead, d, block_table, n_phys, dtype, dev):
    """A cache of rows of d: [batch, *lead, seq_k, d], or pools [n_phys, *lead, block, d]."""
    if block_table is None:
        return _arg(x, name, dtype, shape.batch * lead * shape.seq_k * d, dev, shape.batch)
    return _arg(x, name, dtype, n_phys * lead * shape.block_size * d, dev, n_phys)


def msa_index_scores_tree(shape: MsaShape, seq_lens, block_table, n_phys, mask, idx_q, idx_k,
                          idx_draft, block_scores, packed=False, stream=None):
    dev, st = _place(stream)
    n_phys, packed = int(n_phys), int(packed)
    batch, n, hkv, d, dt = (shape.batch, shape.seq_q, shape.n_heads_kv, shape.index_dim,
                            _FLOATS.get(shape.dtype))
    if packed:
        rec = 128 * (d + 1)
        k = _arg(idx_k, "idx_k", _U8, n_phys * rec, dev, n_phys)
        kd = _arg(idx_draft, "idx_draft", _U8, batch * rec, dev, batch)
    else:
        k = _tree_cache(shape, idx_k, "idx_k", 1, d, block_table, n_phys, dt, dev)
        kd = _arg(idx_draft, "idx_draft", dt, batch * n * d, dev, batch)
    _check(load().msa_index_scores_tree(
        ctypes.byref(shape), _arg(seq_lens, "seq_lens", _I32, batch, dev, batch),
        _arg(block_table, "block_table", _I32, batch * shape.n_blocks, dev, batch), n_phys,
        _arg(mask, "mask", _I64, batch * n, dev, batch),
        _arg(idx_q, "idx_q", dt, batch * n * hkv * d, dev, batch), k, kd, packed,
        _arg(block_scores, "block_scores", _F32, batch * hkv * n * shape.n_blocks, dev, batch), st),
        "msa_index_scores_tree")


def msa_block_topk_tree(shape: MsaShape, seq_lens, mask, block_scores, sel, stream=None):
    dev, st = _place(stream)
    batch, n = shape.batch, shape.seq_q
    rows = batch * shape.n_heads_kv * n
    _check(load().msa_block_topk_tree(
        ctypes.byref(shape), _arg(seq_lens, "seq_lens", _I32, batch, dev, batch),
        _arg(mask, "mask", _I64, batch * n, dev, batch),
        _arg(block_scores, "block_scores", _F32, rows * shape.n_blocks, dev, batch),
        _arg(sel, "sel", _I32, rows * shape.top_k, dev, batch), st), "msa_block_topk_tree")


def msa_sparse_decode_tree(shape: MsaShape, seq_lens, block_table, n_phys, mask, q, k, v, k_draft,
                           v_draft, sel, out, lse, workspace, ws_bytes=None, stream=None):
    dev, st = _place(stream)
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    n_phys = int(n_phys)
    batch, n, hq, hkv, d, dt = (shape.batch, shape.seq_q, shape.n_heads_q, shape.n_heads_kv,
                                shape.head_dim, _FLOATS.get(shape.dtype))
    rows = batch * n * hq * d
    drafts = batch * hkv * n * d
    _check(load().msa_sparse_decode_tree(
        ctypes.byref(shape), _arg(seq_lens, "seq_lens", _I32, batch, dev, batch),
        _arg(block_table, "block_table", _I32, batch * shape.n_blocks, dev, batch), n_phys,
        _arg(mask, "mask", _I64, batch * n, dev, batch), _arg(q, "q", dt, rows, dev, batch),
        _tree_cache(shape, k, "k", hkv, d, block_table, n_phys, dt, dev),
        _tree_cache(shape, v, "v", hkv, d, block_table, n_phys, dt, dev),
        _arg(k_draft, "k_draft", dt, drafts, dev, batch),
        _arg(v_draft, "v_draft", dt, drafts, dev, batch),
        _arg(sel, "sel", _I32, batch * hkv * n * shape.top_k, dev, batch),
        _arg(out, "out", dt, rows, dev, batch), _arg(lse, "lse", _F32, batch * hq * n, dev, batch),
        _arg(workspace, "workspace", None, 0, dev), ws_bytes, st), "msa_sparse_decode_tree")


class CommitTensors:
    """The caches of a msa_tree_commit call.  rows: (src, dst), src [batch, heads, tokens, d] or
    [batch, tokens, d] (one head), dst with the cache's rows in place of the tokens (pools:
    [n_phys, (heads,) block, d]).  packed: (src, dst) of 8-bit index keys, uint8 [batch, 128 (d + 1)]
    and [n_phys, 128 (d + 1)].  Holds the tensors, and may be kept and used for every call."""

    def __init__(self, rows, packed=()):
        rows, packed = list(rows), list(packed)
        self.device = dev = _device()
        self.rows, self.packed = rows, packed
        self.array = (MsaCommitTensor * max(1, len(rows) + len(packed)))()
        # (batch, tokens, first axis and rows of dst) of the rows, (batch, blocks) of 8-bit keys
        self.row_shapes, self.packed_shapes = set(), set()
        for i, (src, dst) in enumerate(rows):
            heads = 1 if src.dim() == 3 else src.shape[1]
            if src.dim() not in (3, 4) or dst.dim() != src.dim() or dst.dtype != src.dtype or \
                    dst.shape[-1] != src.shape[-1] or (src.dim() == 4 and dst.shape[1] != heads):
                raise ValueError(f"commit tensor {i}: src and dst differ in more than their rows: "
                                 f"{tuple(src.shape)} and {tuple(dst.shape)}")
            self.array[i] = MsaCommitTensor(
                _arg(src, f"src of commit tensor {i}", None, 0, dev),
                _arg(dst, f"dst of commit tensor {i}", None, 0, dev), heads,
                src.shape[-1] * src.element_size(), 0)
            self.row_shapes.add((src.shape[0], src.shape[-2], dst.shape[0], dst.shape[-2]))
        for j, (src, dst) in enumerate(packed):
            i = len(rows) + j
            n = src.shape[-1]
            if src.dim() != 2 or dst.dim() != 2 or dst.shape[1] != n or n % 128 or n < 256:
                raise ValueError(f"commit tensor {i}: 8-bit index keys are [batch, 128 (d + 1)] and "
                                 f"[n_phys, 128 (d + 1)], got {tuple(src.shape)} and {tuple(dst.shape)}")
            self.array[i] = MsaCommitTensor(_arg(src, f"src of commit tensor {i}", _U8, 0, dev),
                                            _arg(dst, f"dst of commit tensor {i}", _U8, 0, dev), 1,
                                            n // 128 - 1, 1)
            self.packed_shapes.add((src.shape[0], dst.shape[0]))

    def __len__(self):
        return len(self.rows) + len(self.packed)


def make_commit_tensors(rows, packed=()) -> CommitTensors:
    return CommitTensors(rows, packed)


def msa_tree_commit(shape: MsaShape, seq_lens, block_table, n_phys, accepted,
                    tensors: CommitTensors, new_lens, stream=None, mask=None):
    """With the tree's mask (int64 [batch, tokens]) a list ends at a token that the tree does not have."""
    dev, st = _place(stream)
    batch, n_phys = shape.batch, int(n_phys)
    if tensors.device != dev:
        raise ValueError(f"the commit tensors are on CUDA device {tensors.device}, the current one "
                         f"is {dev}")
    paged = block_table is not None
    want = (batch, shape.seq_q) + ((n_phys, shape.block_size) if paged else (batch, shape.seq_k))
    if tensors.row_shapes and tensors.row_shapes != {want}:
        raise ValueError(f"commit tensors with (batch, tokens, cache axes) {tensors.row_shapes}, the "
                         f"call has {want}")
    if tensors.packed_shapes and tensors.packed_shapes != {(batch, n_phys)}:
        raise ValueError(f"8-bit index keys with (batch, blocks) {tensors.packed_shapes}, the call has "
                         f"{(batch, n_phys)}")
    if accepted.dim() != 2 or accepted.shape[0] != batch:
        raise ValueError(f"accepted is {tuple(accepted.shape)}, expected [{batch}, tokens]")
    _check(load().msa_tree_commit_masked(
        ctypes.byref(shape), _arg(seq_lens, "seq_lens", _I32, batch, dev, batch),
        _arg(block_table, "block_table", _I32, batch * shape.n_blocks, dev, batch), n_phys,
        _arg(mask, "mask", _I64, batch * shape.seq_q, dev, batch),
        _arg(accepted, "accepted", _I32, 0, dev), accepted.shape[1], tensors.array, len(tensors),
        _arg(new_lens, "new_lens", _I32, batch, dev, batch), st), "msa_tree_commit")


def msa_workspace_bytes(shape: MsaShape, which: int) -> int:
    return int(load().msa_workspace_bytes(ctypes.byref(shape), which))


def msa_get_device_status(stream=None):
    _check(load().msa_get_device_status(_stream(stream)), "msa_get_device_status")


def msa_abi_version() -> int:
    return int(load().msa_abi_version())


def msa_debug_set_fault(mode: int):
    """Test hook: mode 1 makes tensor-core prefill launches time out (see include/msa.h)."""
    _check(load().msa_debug_set_fault(mode), "msa_debug_set_fault")
