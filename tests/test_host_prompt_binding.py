"""What the Python binding of the prompt-side calls refuses before it reaches the library.

No GPU: tensors live on the host and only say that they are on the pool's device, and the
library is a stand-in that fails if it is reached (or records the call)."""
import pytest
import torch

import pagedattention_decode_03_b200 as pa
from pagedattention_decode_03_b200 import binding


class OnDevice(torch.Tensor):
    """A host tensor that says it is on cuda:0."""

    def get_device(self):
        return 0


class Library:
    """Stands in for the library: notes the calls that reach it."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or pa.PA_OK


N, H, MBPS, T = 3, 2, 5, 7


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(binding, "lib", lambda: L)
    return L


def pool():
    return pa.Pool(handle=None, desc=None, num_layers=1, num_kv_heads=H, block_size=16, num_blocks=64, max_seqs=N,
                   max_blocks_per_seq=MBPS, kv_dtype="bf16", act_dtype="bf16", device=0)


def dev(shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


def attend_args(tree=False):
    a = dict(q_lens=[3, 0, 4], q=dev((T, 4 * H, 128), torch.bfloat16), out=dev((T, 4 * H, 128), torch.bfloat16),
             scale=0.1, kv_lens=[30, 2, 40], block_tables=dev((N, MBPS)), stream=0)
    if tree:
        a["tree_lens"], a["tree_mask"] = a.pop("q_lens"), dev((T,), torch.int64)
    return a


def attend(tree, **change):
    a = attend_args(tree) | change
    if not tree:
        return pa.pa_prefill_attention(pool(), 0, **a)
    return pa.pa_tree_attention(pool(), 0, **a)


@pytest.mark.parametrize("dtype", [torch.int64, torch.uint64])
def test_masks_of_64_bits_pass(library, dtype):
    attend(True, tree_mask=dev((T,), dtype))
    assert [c[0] for c in library.calls] == ["pa_tree_attention"]


@pytest.mark.parametrize("mask", [dev((T,), torch.complex64), dev((T,), torch.float64), dev((T,)),
                                  dev((T, 2)), dev((T + 1,), torch.int64), dev((2 * T,), torch.int64)[::2],
                                  torch.zeros(T, dtype=torch.int64)],
                         ids=["complex64", "float64", "int32", "pairs of int32", "long", "strided", "host"])
def test_other_masks_are_refused(library, mask):
    with pytest.raises(ValueError, match="tree_mask must"):
        attend(True, tree_mask=mask)
    assert not library.calls


# ---------------------------------------------------------------- build_tables
def tables(**change):
    a = dict(old_lens=dev((N,)), new_lens=dev((N,)), free_blocks=dev((9,)), free_head=dev((1,)),
             free_head_out=dev((1,)), block_tables=dev((N, MBPS)), cu_tokens=dev((N + 1,)), slots=dev((11,)), stream=0)
    pa.pa_build_tables(pool(), **(a | change))


def test_tables_pass(library):
    tables()
    tables(block_tables=dev((0, MBPS)), old_lens=dev((0,)), new_lens=dev((0,)), cu_tokens=dev((1,)), slots=dev((0,)))
    assert [c[0] for c in library.calls] == ["pa_build_tables"] * 2


@pytest.mark.parametrize("shape", [(MBPS, N), (N * MBPS,), (1, N, MBPS), (N, MBPS + 1)])
def test_tables_of_another_shape_are_refused(library, shape):
    """[max_blocks][n] holds as many entries, and its rows would be read as [n][max_blocks]."""
    with pytest.raises(ValueError, match="block_tables must"):
        tables(block_tables=dev(shape))
    assert not library.calls


NOT_I32 = {"host": lambda k: torch.zeros(k, dtype=torch.int32), "int64": lambda k: dev((k,), torch.int64),
           "strided": lambda k: dev((2 * k,))[::2], "long": lambda k: dev((k + 1,)), "short": lambda k: dev((k - 1,))}


@pytest.mark.parametrize("name,size,how", [(name, size, how) for name, size in
                                           (("new_lens", N), ("free_head", 1), ("free_head_out", 1), ("cu_tokens", N + 1))
                                           for how in NOT_I32 if size > 1 or how != "strided"])  # (one element is contiguous)
def test_other_lists_are_refused(library, name, size, how):
    with pytest.raises(ValueError, match=name + " must"):
        tables(**{name: NOT_I32[how](size)})
    assert not library.calls


@pytest.mark.parametrize("how", ["host", "int64", "strided"])
@pytest.mark.parametrize("name,size", [("old_lens", N), ("free_blocks", 9), ("slots", 11)])
def test_other_lists_of_any_length_are_refused(library, name, size, how):
    with pytest.raises(ValueError, match=name + " must"):
        tables(**{name: NOT_I32[how](size)})
    assert not library.calls


# ------------------------------------------------------------------ attention
NOT_ROWS = {"host": torch.zeros((T, 4 * H, 128), dtype=torch.bfloat16), "fp16": dev((T, 4 * H, 128), torch.float16),
            "rows": dev((T + 1, 4 * H, 128), torch.bfloat16), "head_dim": dev((T, 4 * H, 64), torch.bfloat16),
            "strided": dev((T, 4 * H, 256), torch.bfloat16)[..., :128],
            "transposed": dev((4 * H, T, 128), torch.bfloat16).transpose(0, 1)}


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("how", list(NOT_ROWS))
@pytest.mark.parametrize("name", ["q", "out"])
def test_other_rows_are_refused(library, tree, name, how):
    with pytest.raises(ValueError, match="(q|out) must"):
        attend(tree, **{name: NOT_ROWS[how]})
    assert not library.calls


@pytest.mark.parametrize("tree", [False, True])
def test_rows_of_another_number_of_heads_are_refused(library, tree):
    with pytest.raises(ValueError, match="out must have shape"):
        attend(tree, out=dev((T, 2 * H, 128), torch.bfloat16))
    with pytest.raises(ValueError, match="q must"):
        attend(tree, q=dev((T, 4 * H * 128), torch.bfloat16))
    assert not library.calls


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("bad", [torch.zeros((N, MBPS), dtype=torch.int32), dev((N, MBPS), torch.int64), dev((MBPS, N)),
                                 dev((N + 1, MBPS)), dev((MBPS, N)).t()], ids=["host", "int64", "transposed", "rows", "view"])
def test_attention_refuses_other_tables(library, tree, bad):
    with pytest.raises(ValueError, match="block_tables must"):
        attend(tree, block_tables=bad)
    assert not library.calls


@pytest.mark.parametrize("tree", [False, True])
def test_host_lists_of_another_length_are_refused(library, tree):
    with pytest.raises(ValueError, match="kv_lens and the query lengths"):
        attend(tree, kv_lens=[30, 2])
    with pytest.raises(ValueError, match="seqs and the query lengths"):
        attend(tree, kv_lens=None, block_tables=None, seqs=[0, 1, 2, 1])
    with pytest.raises(OverflowError):
        attend(tree, kv_lens=[30, 2, 2 ** 31])
    assert not library.calls


# --------------------------------------------------------------------- append
@pytest.mark.parametrize("name,bad", [("slots", torch.zeros(T, dtype=torch.int32)), ("slots", dev((T,), torch.int64)),
                                      ("slots", dev((T, 1))), ("slots", dev((2 * T,))[::2]), ("slots", dev((T - 1,))),
                                      ("k_new", dev((T, H, 128), torch.float16)), ("k_new", dev((T, 128 * H), torch.bfloat16)),
                                      ("v_new", torch.zeros((T, H, 128), dtype=torch.bfloat16)),
                                      ("v_new", dev((T, H, 256), torch.bfloat16)[..., ::2]),
                                      ("v_new", dev((T + 1, H, 128), torch.bfloat16))])
def test_append_refuses_other_tensors(library, name, bad):
    a = dict(slots=dev((T,)), k_new=dev((T, H, 128), torch.bfloat16), v_new=dev((T, H, 128), torch.bfloat16), stream=0)
    with pytest.raises(ValueError, match="(slots|k_new|v_new) must"):
        pa.pa_append_kv_slots(pool(), 0, **(a | {name: bad}))
    assert not library.calls
    pa.pa_append_kv_slots(pool(), 0, **a)
    assert [c[0] for c in library.calls] == ["pa_append_kv_slots"]
