"""Pools off a 16-byte boundary are refused on the host, before any CUDA call.

The calls have no tokens, so that one whose checks all pass launches nothing and
returns MSA_OK: the pointers are made up, and none is ever dereferenced.
"""

import ctypes

import pytest
import torch

from nvfp4_kv_block_gb300 import ops
from test_abi_cpu import _cache, lib  # noqa: F401
from test_oracle_rotary import _row_struct

FAKE = ctypes.c_void_p(16)
BIG = 1 << 32
INDEX = (FAKE, FAKE, 8, FAKE, 4, FAKE, FAKE, 1, 0, 16)
# call, its arguments behind the cache, the widest access to the K/V pool and to the index pool (1: none)
CALLS = {
    "msa_quantize_kv_insert": ((FAKE, FAKE, FAKE, FAKE, 0, None), 4, 4),
    "msa_indexer_topk": (INDEX + (FAKE, FAKE, FAKE, BIG, None), 1, 16),
    "msa_indexer_topk_range": (INDEX + (0, 4, FAKE, FAKE, BIG, None), 1, 16),
    "msa_indexer_topk_noalloc": (INDEX + (FAKE, FAKE, None), 1, 16),
    "msa_sparse_attn_decode": ((FAKE, 16, 0.1, FAKE, FAKE, FAKE, 4, FAKE, FAKE, 1, 0, 4, FAKE, FAKE, None), 16, 1),
    "msa_decode_fused": ((FAKE, FAKE, FAKE, 16, 8, 0.1, FAKE, 4, FAKE, FAKE, 1, 0, 16, FAKE, FAKE, FAKE, FAKE, BIG, None), 16, 16),
    "msa_qkv_project_insert": ((FAKE, FAKE, 0, 64, FAKE, FAKE, FAKE, FAKE, 8, FAKE, FAKE, 1e-6, FAKE, None, None), 4, 16),
    "msa_rotary_insert": ((ctypes.byref(_row_struct()), 0, FAKE, 8, 64, 0, FAKE, FAKE, FAKE, FAKE, None), 16, 16),
    "msa_read_kv": ((FAKE, 0, 1, FAKE, FAKE, FAKE, None), 16, 16),
    "msa_tree_attn": ((FAKE, 16, 0.1, FAKE, 4, FAKE, FAKE, 1, 0, None, None, None, 1, FAKE, FAKE, FAKE, BIG, None), 16, 1),
}


@pytest.mark.parametrize("name", CALLS)
def test_misaligned_pools_are_refused(lib, name):  # noqa: F811
    args, kv, idx = CALLS[name]

    def call(kv_pool, idx_pool):
        return getattr(lib, name)(ctypes.byref(_cache(kv_pool=kv_pool, idx_pool=idx_pool, n_pages=4)), *args)

    # every check passes (the call with scratch of its own asks the device for its address first)
    fine = (0, -4) if name == "msa_indexer_topk_noalloc" else (0,)
    assert call(160, 160) in fine
    for off in (1, 2, 4, 8):
        assert call(160 + off, 160) in ((-1,) if off % kv else fine), off
        assert call(160, 160 + off) in ((-1,) if off % idx else fine), off


def test_from_pools_refuses_views_off_16_bytes():
    """A slice that begins inside a larger buffer (the check comes before the device's)."""
    kv = torch.zeros(ops.KV_PAGE_BYTES + 16, dtype=torch.uint8)
    ix = torch.zeros(ops.IDX_PAGE_BYTES + 16, dtype=torch.uint8)
    assert kv.data_ptr() % 16 == 0 and ix.data_ptr() % 16 == 0

    def make(a, b):
        return ops.KVCache.from_pools(kv[a:a + ops.KV_PAGE_BYTES].view(1, -1), ix[b:b + ops.IDX_PAGE_BYTES].view(1, -1), 1.0, 1.0)

    for off in (1, 2, 4, 8):
        with pytest.raises(ValueError, match="kv_pool must begin on a 16-byte"):
            make(off, 0)
        with pytest.raises(ValueError, match="idx_pool must begin on a 16-byte"):
            make(0, off)
    for off in (0, 16):
        with pytest.raises(ValueError, match="CUDA"):
            make(off, off)
