"""Cases of the prompt and tree attention that need their own data or sizes: scores that
rise along the cache or are very large, negative scales of K, calls of more than 48
sequences.  Bounds: prompt_reference.py.
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


@pytest.mark.parametrize("kv,act", KINDS)
@pytest.mark.parametrize("lens,new", [([1700, 300], [1700, 300]), ([9000], [20]), ([2000] * 10, [600] * 10)],
                         ids=["whole", "split", "paired"])
@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_as_large_as_the_types_allow(kv, act, lens, new, rising, sign):
    """Scores apart by far more than their rounding: each row's weight is all on one position,
    whose V row it is, or on positions of one score.  K rows are whole multiples of a step, alike
    in every d, so the products and their sums are exact; they rise along the cache, or stand
    in any order."""
    s = Setup(lens, H=4, kv=kv, act=act, seed=5)
    big_q, step = {"bf16": (2.0 ** 60, 2.0 ** 40), "fp16": (2.0 ** 15, 2.0 ** 5), "fp8_e4m3": (2.0 ** 15, 2.0)}[kv]
    if kv == "fp8_e4m3" and act == "bf16":
        big_q = 2.0 ** 80
    top = 15 if kv == "fp8_e4m3" else 127                 # multiples of the step that the type holds
    g = torch.Generator().manual_seed(1)
    want = []
    for i, (n, m) in enumerate(zip(lens, new)):
        level = torch.randint(0, top, (n,), generator=g)
        if rising:
            level = torch.arange(n) * top // n
        pos = torch.arange(n, device="cuda")
        x = (level.float() * step).cuda()[:, None, None].expand(n, 4, 128)
        x = x.to(torch.float8_e4m3fn).view(torch.uint8) if kv == "fp8_e4m3" else x.to(s.cache[0].dtype)
        s.cache[0][0][s.tables[i].long()[pos // s.B], :, pos % s.B] = x
        v = s.rows(1, i, n)                               # [n, H, D]
        level = level.cuda()
        for t in range(n - m, n):
            best = level[:t + 1] == level[:t + 1].max()
            want.append(torch.stack([v[:t + 1][best].mean(0), v[:t + 1][best].abs().mean(0)]))
    want, mean = torch.stack(want, 1)[:, :, :, None].expand(-1, -1, -1, 4, -1).reshape(2, sum(new), 16, 128)
    q = torch.full((sum(new), 16, 128), sign * big_q, dtype=want.dtype).to(s.rand(1, 1).dtype).cuda()
    out = torch.full_like(q, float("nan"))
    pa.pa_prefill_attention(s.pool, 0, new, q, out, sign * SCALE, kv_lens=lens, block_tables=s.tables)
    # as in prompt_reference.py: the ties' weights are 2^x for one x near 0, rounded to the
    # type, u times the mean of |v| under them (their sum is not rounded), and the exponential
    # a sixteenth of that; sums in fp32; the result's own rounding (fp16: subnormal steps)
    u = torch.finfo(out.dtype).eps / 2
    bound = u * (1 + 1 / 16) * mean + u * want.abs() + (2 * (max(lens) + 8) * 2.0 ** -24) * mean
    bound = bound + (2.0 ** -25 if act == "fp16" else 0)
    assert torch.isfinite(out).all()
    assert ((out.double() - want).abs() <= bound).all()
    assert pa.pa_check_device_errors(s.pool) == 0


@pytest.mark.parametrize("act", ["bf16", "fp16"])
@pytest.mark.parametrize("scale", [SCALE, -SCALE])
def test_negative_scales_of_k(act, scale):
    """FP8 codes may stand for numbers of the other sign in some heads."""
    lens, new = [300, 9000, 77], [300, 16, 9]
    s = Setup(lens, H=4, kv="fp8_e4m3", act=act, seed=4)
    sign = torch.tensor([1.0, -1.0, -1.0, 1.0], device="cuda")
    for t in (s.pool.scales[0], s.pool.scales[2]):
        t *= sign
    s.scale_k *= sign
    q = s.rand(sum(new), 16, 2.0)
    out = torch.full_like(q, float("nan"))
    pa.pa_prefill_attention(s.pool, 0, new, q, out, scale, kv_lens=lens, block_tables=s.tables)
    s.check(new, q, out, scale)
    few = [30, 16, 9]
    mask = random_tree_mask(few, torch.Generator().manual_seed(2))
    mask[::4] = 0
    qt = q[:sum(few)].contiguous()
    out = torch.full_like(qt, float("nan"))
    pa.pa_tree_attention(s.pool, 0, few, mask, qt, out, scale, kv_lens=lens, block_tables=s.tables)
    s.check(few, qt, out, scale, mask=mask)
    assert pa.pa_check_device_errors(s.pool) == 0
