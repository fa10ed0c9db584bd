"""Cases of the prompt and tree attention that need their own data or sizes: scores that
rise along the cache.  Bounds: prompt_reference.py.
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
