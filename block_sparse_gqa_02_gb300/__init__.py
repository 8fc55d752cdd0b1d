"""MiniMax Sparse Attention (MSA) hot path for GB300 (sm_103a).

The computation lives in libmsa.so (CUDA kernels behind the C ABI of include/msa.h);
this package only marshals arguments to it.
"""
from ._lib import (MsaError, MsaShape, make_gather_tensors, make_rope, make_rope_tensors,
                   make_shape, msa_abi_version, msa_block_topk, msa_cache_evict,
                   msa_cache_gather, msa_cache_pack, msa_cache_unpack, msa_get_device_status,
                   msa_index_scores, msa_rope, msa_sparse_decode, msa_sparse_decode_mass,
                   msa_sparse_decode_packed, msa_sparse_prefill, msa_workspace_bytes,
                   shape_from_config)
from .api import (Rope, alloc_decode_outputs, alloc_packed_cache, alloc_prefill_outputs, decode,
                  decode_packed, evict, evict_paged, prefill, rope, rope_freqs, run_decode,
                  run_prefill)
