"""Lengths near 2^31 are refused before they are rounded up in 32 bits (no GPU: refused
calls return before any device work; addresses are never dereferenced)."""
import ctypes

import numpy as np
import pytest

import pagedattention_decode_03_b200 as pa
from pagedattention_decode_03_b200.binding import lib, pa_pool_desc


@pytest.fixture(scope="module", autouse=True)
def built():
    from pagedattention_decode_03_b200 import build
    build.build()


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("kv,blocks", [(2 ** 31 - 255, 1 << 27), (2 ** 31 - 1, 1 << 27), (161, 10)])
def test_attention_refuses_lengths_past_the_last(tree, kv, blocks):
    d = pa_pool_desc()
    d.num_layers, d.num_kv_heads, d.head_dim, d.block_size = 1, 2, 128, 16
    d.num_blocks, d.max_seqs, d.max_blocks_per_seq = 64, 1, blocks
    d.kv_dtype = d.act_dtype = pa.binding.PA_BF16
    d.k_cache, d.v_cache, d.workspace = 4096, 8192, 1 << 20
    d.workspace_bytes = lib().pa_workspace_size(ctypes.byref(d))
    h = ctypes.c_void_p()
    assert lib().pa_pool_create(ctypes.byref(d), ctypes.byref(h)) == pa.PA_OK
    try:
        lens, q = np.array([kv], np.int32), np.array([1], np.int32)
        a = [h, 0, 1, None, 4096, lens.ctypes.data, q.ctypes.data] + ([4096] if tree else [])
        st = (lib().pa_tree_attention if tree else lib().pa_prefill_attention)(*a, 8, 4096, 4096, 0.1, None)
        assert st == pa.PA_ERR_INVALID_ARG and "2^31 - 256" in pa.pa_last_error()
    finally:
        lib().pa_pool_destroy(h)
