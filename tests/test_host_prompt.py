"""Refusals of the prompt-side entry points (no GPU: every refused call returns
before any device work; addresses are never dereferenced)."""
import ctypes

import numpy as np
import pytest

import pagedattention_decode_03_b200 as pa
from pagedattention_decode_03_b200.binding import lib, pa_pool_desc


@pytest.fixture(scope="module", autouse=True)
def built():
    from pagedattention_decode_03_b200 import build
    build.build()


class Fake:
    """A pool over addresses that are never touched."""

    def __init__(self, host_only=False):
        d = pa_pool_desc()
        d.num_layers, d.num_kv_heads, d.head_dim, d.block_size = 2, 2, 128, 16
        d.num_blocks, d.max_seqs, d.max_blocks_per_seq = 64, 4, 10
        d.kv_dtype = d.act_dtype = pa.binding.PA_BF16
        if not host_only:
            d.k_cache, d.v_cache, d.workspace = 4096, 8192, 1 << 20
            d.workspace_bytes = lib().pa_workspace_size(ctypes.byref(d))
        self.h = ctypes.c_void_p()
        assert lib().pa_pool_create(ctypes.byref(d), ctypes.byref(self.h)) == pa.PA_OK

    def __del__(self):
        lib().pa_pool_destroy(self.h)


def arr(*x):
    return np.array(x, np.int32)


def attend(f, tree=False, layer=0, n=1, seqs=None, tables=4096, kv=(100,), lens=(20,), mask=4096, hq=8, q=4096,
           out=4096, scale=0.1, handle=True):
    seqs, kv, lens = (None if x is None else arr(*x) for x in (seqs, kv, lens))
    ptr = [x.ctypes.data if x is not None else None for x in (seqs, kv, lens)]
    a = [f.h if handle else None, layer, n, ptr[0], tables, ptr[1], ptr[2]] + ([mask] if tree else [])
    return (lib().pa_tree_attention if tree else lib().pa_prefill_attention)(*a, hq, q, out, scale, None)


ATTEND = [dict(handle=False), dict(layer=-1), dict(layer=2), dict(n=-1), dict(lens=None), dict(tables=None),
          dict(tables=None, kv=None), dict(seqs=(0,)), dict(kv=None), dict(hq=0), dict(hq=3), dict(hq=6), dict(hq=32),
          dict(q=4104), dict(out=4100), dict(tables=4098), dict(scale=float("inf")), dict(scale=float("nan")),
          dict(kv=(-1,)), dict(kv=(161,)), dict(lens=(-1,)), dict(lens=(101,)), dict(q=None), dict(out=None),
          dict(tables=None, kv=(100,), seqs=(0,))]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("bad", ATTEND, ids=[str(b) for b in ATTEND])
def test_attention_refusals(tree, bad):
    assert attend(Fake(), tree, **bad) == pa.PA_ERR_INVALID_ARG
    assert pa.pa_last_error()


def test_tree_refusals():
    f = Fake()
    assert attend(f, True, lens=(65,)) == pa.PA_ERR_INVALID_ARG
    assert attend(f, True, mask=None) == pa.PA_ERR_INVALID_ARG
    assert attend(f, True, mask=4100) == pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("tree", [False, True])
def test_sequences_of_the_pool(tree):
    f = Fake()
    own = dict(tables=None, kv=None)
    assert attend(f, tree, seqs=(4,), **own) == pa.PA_ERR_INVALID_ARG
    assert attend(f, tree, seqs=(1,), **own) == pa.PA_ERR_NO_SEQ
    assert lib().pa_alloc_blocks(f.h, 1, 19, None) == pa.PA_OK
    assert attend(f, tree, seqs=(1,), **own) == pa.PA_ERR_INVALID_ARG       # 20 query tokens, 19 cached


@pytest.mark.parametrize("tree", [False, True])
def test_nothing_to_do(tree):
    f = Fake()
    assert attend(f, tree, n=0, tables=None, kv=None, lens=None, q=None, out=None, mask=None) == pa.PA_OK
    assert attend(f, tree, n=2, kv=(0, 7), lens=(0, 0), q=None, out=None, mask=None) == pa.PA_OK
    assert lib().pa_append_kv_slots(f.h, 0, 0, None, None, None, None) == pa.PA_OK
    assert lib().pa_launch_count(f.h) == 0


def test_too_many_rows():
    f = Fake()
    big = dict(n=2 ** 12, kv=[160] * 2 ** 12, lens=[160] * 2 ** 12)
    assert attend(f, hq=16, q=None, **big) == pa.PA_ERR_INVALID_ARG
    many = 2 ** 20
    assert attend(f, n=many, kv=[160] * many, lens=[160] * many, hq=16) == pa.PA_ERR_INVALID_ARG
    assert "2^31" in pa.pa_last_error()


def tables_call(f, n=1, old=4096, new=4096, free=4096, num_free=5, head=4096, head_out=4096, tables=4096, cu=4096,
                slots=4096, cap=5, handle=True):
    return lib().pa_build_tables(f.h if handle else None, n, old, new, free, num_free, head, head_out, tables, cu,
                                 slots, cap, None)


TABLES = [dict(handle=False), dict(n=-1), dict(n=8193), dict(num_free=-1), dict(cap=-1), dict(old=None),
          dict(new=None), dict(free=None), dict(head=None), dict(head_out=None), dict(tables=None), dict(cu=None),
          dict(slots=None), dict(old=4097), dict(slots=4098), dict(cu=4099), dict(head=4097)]


@pytest.mark.parametrize("bad", TABLES, ids=[str(b) for b in TABLES])
def test_tables_refusals(bad):
    assert tables_call(Fake(), **bad) == pa.PA_ERR_INVALID_ARG


APPEND = [dict(layer=2), dict(layer=-1), dict(T=-1), dict(slots=None), dict(k=None), dict(v=None), dict(k=4104),
          dict(v=4097), dict(slots=4097), dict(handle=False)]


@pytest.mark.parametrize("bad", APPEND, ids=[str(b) for b in APPEND])
def test_append_refusals(bad):
    f = Fake()
    a = dict(layer=0, T=3, slots=4096, k=4096, v=4096, handle=True) | bad
    assert lib().pa_append_kv_slots(f.h if a["handle"] else None, a["layer"], a["T"], a["slots"], a["k"], a["v"],
                                    None) == pa.PA_ERR_INVALID_ARG


def test_host_only_pools_refuse():
    f = Fake(host_only=True)
    assert attend(f) == pa.PA_ERR_INVALID_ARG
    assert attend(f, True) == pa.PA_ERR_INVALID_ARG
    assert tables_call(f) == pa.PA_ERR_INVALID_ARG
    assert lib().pa_append_kv_slots(f.h, 0, 3, 4096, 4096, 4096, None) == pa.PA_ERR_INVALID_ARG


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    p = pa.pa_pool_create(num_layers=1, num_kv_heads=2, block_size=16, num_blocks=8, max_seqs=2,
                          max_blocks_per_seq=4, host_only=True)
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.pa_prefill_attention(p, 0, [3], q, q, 0.1, seqs=[0])
    with pytest.raises(ValueError):
        pa.pa_tree_attention(p, 0, [3], torch.zeros(3, dtype=torch.int32), q, q, 0.1, seqs=[0])
    with pytest.raises(ValueError):
        pa.pa_append_kv_slots(p, 0, i, q, q)
    with pytest.raises(ValueError):
        pa.pa_build_tables(p, i, i, i, i[:1], i[:1], i.view(3, 1), i, i)
