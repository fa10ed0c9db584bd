"""Cases of the prompt and tree attention that need their own data or sizes: scores that
rise along the cache, calls of more than 48 sequences.  Bounds: prompt_reference.py.
"""
import math

import pytest
import torch

import pagedattention_decode_03_b200 as pa
from prompt_reference import Setup, random_tree_mask

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)
KINDS = [("bf16", "bf16"), ("fp16", "fp16"), ("fp8_e4m3", "bf16"), ("fp8_e4m3", "fp16")]


def ramp_keys(s, lo, hi):
    """K rows of every sequence: a ramp along its positions, the same in every d, and noise."""
    for i, n in enumerate(s.lens):
        pos = torch.arange(n, device="cuda")
        blk = s.tables[i].long()[pos // s.B]
        r = torch.linspace(lo, hi, n, device="cuda")[:, None, None] + 0.1 * s.rand(n, s.H).float()
        x = r.to(torch.float8_e4m3fn).view(torch.uint8) if s.kv == "fp8_e4m3" else r.to(s.cache[0].dtype)
        s.cache[0][s.layer][blk, :, pos % s.B] = x


@pytest.mark.parametrize("kv,act", KINDS)
@pytest.mark.parametrize("lens,new", [([1700, 300], [1700, 300]), ([9000], [20]), ([2000] * 10, [600] * 10)],
                         ids=["whole", "split", "paired"])
@pytest.mark.parametrize("hi", [60.0, 8.0])
def test_every_tile_passes_the_maximum_before_it(kv, act, lens, new, hi):
    """Scores that rise along the cache, by tens or by a few units a tile of positions: the
    weights of a tile are made anew against its own maximum, tile after tile."""
    s = Setup(lens, H=4, kv=kv, act=act, seed=5)
    ramp_keys(s, -hi / 8, hi)
    scale = SCALE if kv != "fp8_e4m3" else SCALE / float(s.scale_k.max())
    q = s.rand(sum(new), 16).abs() * 0.5
    out = torch.full_like(q, float("nan"))
    pa.pa_prefill_attention(s.pool, 0, new, q, out, scale, kv_lens=lens, block_tables=s.tables)
    s.check(new, q, out, scale)
    few = [min(m, 50) for m in new]
    mask = random_tree_mask(few, torch.Generator().manual_seed(2))
    qt = q[:sum(few)].contiguous()
    out = torch.full_like(qt, float("nan"))
    pa.pa_tree_attention(s.pool, 0, few, mask, qt, out, scale, kv_lens=lens, block_tables=s.tables)
    s.check(few, qt, out, scale, mask=mask)
    assert pa.pa_check_device_errors(s.pool) == 0


# Calls of up to 48 sequences with query tokens, and of more, have launches of their own.
def both(s, new, hq):
    """The chunk and the tree attention of these query tokens, checked."""
    q = s.rand(sum(new), hq, 2.0)
    out = torch.full_like(q, float("nan"))
    own = dict(kv_lens=s.lens, block_tables=s.tables)
    pa.pa_prefill_attention(s.pool, s.layer, new, q, out, SCALE, **own)
    s.check(new, q, out, SCALE)
    mask = random_tree_mask(new, torch.Generator().manual_seed(len(new)))
    mask[::5] = 0
    out.fill_(float("nan"))
    pa.pa_tree_attention(s.pool, s.layer, new, mask, q, out, SCALE, **own)
    s.check(new, q, out, SCALE, mask=mask)
    assert pa.pa_check_device_errors(s.pool) == 0


def cycle(values, n):
    return [values[i % len(values)] for i in range(n)]


@pytest.mark.parametrize("kv,act", KINDS)
@pytest.mark.parametrize("n", [48, 49])
@pytest.mark.parametrize("B,G,H", [(16, 4, 2), (32, 8, 1), (16, 1, 3)])
def test_many_ragged_sequences(kv, act, n, B, G, H):
    new = cycle([1, 17, 40, 64, 5, 33], n) + [0, 0]
    past = cycle([0, 200, 15, 16, 400], n) + [0, 70]
    new.insert(7, 0)
    past.insert(7, 33)
    s = Setup([a + b for a, b in zip(past, new)], H=H, kv=kv, act=act, B=B, layers=2, layer=1, seed=n)
    both(s, new, H * G)


@pytest.mark.parametrize("kv,act", KINDS)
@pytest.mark.parametrize("n", [48, 49])
def test_many_sequences_of_paired_tiles(kv, act, n):
    """Two query tiles over the same KV tiles: 64 tokens of 8 heads are two pairs a sequence."""
    new = [64] * n
    s = Setup([64 + p for p in cycle([0, 130, 7, 300], n)], H=4, kv=kv, act=act, seed=n)
    both(s, new, 32)


@pytest.mark.parametrize("kv,act", KINDS)
@pytest.mark.parametrize("n", [48, 49, 60])
def test_many_sequences_with_split_positions(kv, act, n):
    """Fewer units than SMs, caches of one tile of positions to 70: the longer ones are
    computed in parts and joined, the others not."""
    new = cycle([16, 1, 9, 12], n)
    past = cycle([100, 3000, 40, 900, 9000, 0, 1500], n)
    s = Setup([a + b for a, b in zip(past, new)], H=1, kv=kv, act=act, seed=n)
    both(s, new, 8)


@pytest.mark.parametrize("kv,act", KINDS)
def test_sequences_of_two_launches(kv, act):
    """More than one launch holds (512), the second one's positions split."""
    new = [1] * 512 + [3, 0, 2]
    past = cycle([0, 5, 130], 512) + [5000, 10, 300]
    s = Setup([a + b for a, b in zip(past, new)], H=1, kv=kv, act=act, seed=1)
    both(s, new, 4)
