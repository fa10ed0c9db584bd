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
