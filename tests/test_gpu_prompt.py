"""Attention of prompts, chunks and drafted trees over the paged cache, against the
same formulas in 64 bits (bounds derived in prompt_reference.py).

Slots past every length, and blocks that belong to nobody, hold NaN bytes.
"""
import math

import pytest
import torch

import pagedattention_decode_03_b200 as pa
from prompt_reference import DT, Setup, random_tree_mask

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)
KINDS = [("bf16", "bf16"), ("fp16", "fp16"), ("fp8_e4m3", "bf16"), ("fp8_e4m3", "fp16")]
# lengths around blocks, tiles of 128 positions and groups of 128 rows; empty ones between
PROMPTS = [1, 0, 15, 16, 17, 33, 127, 128, 129, 0, 255, 257, 300, 2]


def prefill(s, q_lens, hq, scale=SCALE, **kw):
    q = s.rand(sum(q_lens), hq, 2.0)
    out = torch.full_like(q, float("nan"))
    kw = kw or dict(kv_lens=s.lens, block_tables=s.tables)
    pa.pa_prefill_attention(s.pool, s.layer, q_lens, q, out, scale, **kw)
    return q, out


def tree(s, lens, mask, hq, scale=SCALE, **kw):
    q = s.rand(sum(lens), hq, 2.0)
    out = torch.full_like(q, float("nan"))
    kw = kw or dict(kv_lens=s.lens, block_tables=s.tables)
    pa.pa_tree_attention(s.pool, s.layer, lens, mask, q, out, scale, **kw)
    return q, out


@pytest.mark.parametrize("kv,act", KINDS)
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("B", [16, 32])
def test_whole_prompts(kv, act, G, B):
    s = Setup(PROMPTS, H=2, kv=kv, act=act, B=B, layers=2, layer=1, seed=G)
    q, out = prefill(s, PROMPTS, 2 * G)
    s.check(PROMPTS, q, out, SCALE)
    assert pa.pa_check_device_errors(s.pool) == 0


@pytest.mark.parametrize("kv,act", KINDS)
@pytest.mark.parametrize("G,H", [(1, 3), (2, 4), (4, 2), (8, 1)])
def test_chunks_behind_a_cached_prefix(kv, act, G, H):
    past = [1, 0, 100, 127, 128, 129, 700, 2000, 33, 4100, 16]
    new = [1, 1, 28, 1, 0, 300, 64, 3, 129, 17, 16]
    s = Setup([p + m for p, m in zip(past, new)], H=H, kv=kv, act=act, seed=G + H)
    q, out = prefill(s, new, H * G)
    s.check(new, q, out, SCALE)
    assert pa.pa_check_device_errors(s.pool) == 0


@pytest.mark.parametrize("kv,act", KINDS)
@pytest.mark.parametrize("lens,new,G,H", [([3000], [3000], 8, 1), ([2111, 1500, 1], [2111, 1500, 1], 4, 4),
                                          ([40000], [5], 8, 2), ([40000], [700], 4, 1), ([20001], [20], 1, 2),
                                          ([9000, 20, 30000, 129], [40, 20, 16, 129], 2, 2)])
def test_long_sequences(kv, act, lens, new, G, H):
    s = Setup(lens, H=H, kv=kv, act=act, seed=len(lens))
    q, out = prefill(s, new, H * G)
    s.check(new, q, out, SCALE)
    assert pa.pa_check_device_errors(s.pool) == 0


@pytest.mark.parametrize("kv,act", KINDS)
@pytest.mark.parametrize("B", [16, 32])
def test_paired_tiles_of_prompts_and_wide_trees(kv, act, B):
    """Enough query tiles for two to share each KV tile (a pair for every SM)."""
    past = [0, 5, 300, 128, 0, 77, 16, 1000] * 5
    new = [64, 64, 64, 63, 64, 64, 33, 64] * 5
    s = Setup([p + m for p, m in zip(past, new)], H=4, kv=kv, act=act, B=B, seed=11)
    mask = random_tree_mask(new, torch.Generator().manual_seed(3))
    mask[::5] = 0
    q, out = tree(s, new, mask, 32)
    s.check(new, q, out, SCALE, mask=mask)
    lens = [700, 0, 650, 1, 512, 800, 33, 640]
    s = Setup(lens, H=4, kv=kv, act=act, B=B, seed=12)
    q, out = prefill(s, lens, 16)
    s.check(lens, q, out, SCALE)
    assert pa.pa_check_device_errors(s.pool) == 0


def test_decode_and_prompt_attention_on_one_pool():
    """The single-query decode (stream-K split, fixed partitions) between prompt calls
    that split positions: they share the pool's workspace and counters."""
    s = Setup([], H=2, mbps=600, num_blocks=1300)
    p = pa.pa_pool_create(num_layers=1, num_kv_heads=2, block_size=16, num_blocks=1300, max_seqs=3,
                          max_blocks_per_seq=600, kv_dtype="bf16", k_cache=s.cache[0], v_cache=s.cache[1])
    lens = [9000, 700, 33]
    for i, n in enumerate(lens):
        pa.pa_alloc_blocks(p, i, n)
        pa.pa_append_kv(p, 0, [i] * n, list(range(n)), s.rand(n, 2), s.rand(n, 2))
    s.pool, s.lens = p, lens
    s.tables = torch.tensor([(pa.pa_get_seq(p, i)[1] + [0] * 600)[:600] for i in range(3)], device="cuda")
    for part in (0, 512, 0):
        q, out = prefill(s, [20, 20, 20], 16, seqs=[0, 1, 2])
        s.check([20, 20, 20], q, out, SCALE)
        q, dec = s.rand(3, 16, 2.0), torch.empty((3, 16, 128), dtype=torch.bfloat16, device="cuda")
        one = torch.empty_like(dec)
        pa.pa_decode_attention(p, 0, [0, 1, 2], q, dec, SCALE, part)
        pa.pa_prefill_attention(p, 0, [1, 1, 1], q, one, SCALE, seqs=[0, 1, 2])
        s.check([1, 1, 1], q, dec, SCALE)
        s.check([1, 1, 1], q, one, SCALE)
    assert pa.pa_check_device_errors(p) == 0


def test_two_pools_on_two_streams():
    """Calls of different pools may overlap on the GPU, captured ones too."""
    lens, new = [600, 12000, 64], [600, 16, 64]
    setups = [Setup(lens, H=2, kv=kv, seed=5) for kv in ("bf16", "fp8_e4m3")]
    streams = [torch.cuda.Stream() for _ in setups]
    qs = [s.rand(sum(new), 16, 2.0) for s in setups]
    outs = [torch.zeros_like(q) for q in qs]
    torch.cuda.synchronize()
    graphs = []
    for s, st, q, out in zip(setups, streams, qs, outs):
        with torch.cuda.stream(st):
            pa.pa_prefill_attention(s.pool, 0, new, q, out, SCALE, kv_lens=lens, block_tables=s.tables)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(3):
                pa.pa_prefill_attention(s.pool, 0, new, q, out, SCALE, kv_lens=lens, block_tables=s.tables)
        graphs.append(g)
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for s, q, out in zip(setups, qs, outs):
        s.check(new, q, out, SCALE)
        assert pa.pa_check_device_errors(s.pool) == 0


def test_more_sequences_than_one_launch_holds():
    lens = [(i * 37) % 90 for i in range(1100)]
    s = Setup(lens, H=1, seed=3)
    q, out = prefill(s, lens, 4)
    s.check(lens, q, out, SCALE)
    few = [min(x, 3) for x in lens]
    mask = random_tree_mask(few, torch.Generator().manual_seed(0))
    q, out = tree(s, few, mask, 4)
    s.check(few, q, out, SCALE, mask=mask)


@pytest.mark.parametrize("scale", [0.0, -SCALE, 1.0, 1e-6])
@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_scales(scale, kv):
    lens = [200, 31, 513]
    s = Setup(lens, H=2, kv=kv, seed=9)
    q, out = prefill(s, lens, 8, scale)
    s.check(lens, q, out, scale)


@pytest.mark.parametrize("scale", [-1e-8, 1e-8, -SCALE])
@pytest.mark.parametrize("kv,act", KINDS)
def test_rows_of_zeros_attend_evenly(kv, act, scale):
    """Padding rows: zero queries weigh all that they attend the same, for scales of
    both signs and so small that scale x 2^-126 is no number of fp32 any more."""
    lens, new = [200, 31, 513], [200, 9, 40]
    s = Setup(lens, H=2, kv=kv, act=act, seed=12)
    q = s.rand(sum(new), 8)
    q[::2] = 0
    out = torch.full_like(q, float("nan"))
    pa.pa_prefill_attention(s.pool, s.layer, new, q, out, scale, kv_lens=s.lens, block_tables=s.tables)
    s.check(new, q, out, scale)


def test_large_scores_do_not_overflow():
    """Scores of several thousand, rising and falling along the positions."""
    s = Setup([700], H=1, kv="bf16", seed=4)
    pos = torch.arange(700, device="cuda")
    rows = s.cache[0][0][s.tables[0].long()[pos // 16], :, pos % 16]
    ramp = torch.cat([torch.linspace(-30, 30, 350), torch.linspace(30, -30, 350)]).cuda()
    s.cache[0][0][s.tables[0].long()[pos // 16], :, pos % 16] = (rows.float() * 0.01 + ramp[:, None, None]).to(rows.dtype)
    q, out = prefill(s, [700], 4)
    s.check([700], q, out, SCALE)


@pytest.mark.parametrize("kv,act", KINDS)
@pytest.mark.parametrize("G,H", [(1, 4), (2, 2), (4, 2), (8, 2)])
@pytest.mark.parametrize("B", [16, 32])
def test_trees(kv, act, G, H, B):
    past = [0, 0, 1, 15, 16, 112, 127, 128, 500, 1000, 64, 7]
    new = [1, 64, 5, 1, 0, 16, 33, 64, 17, 40, 64, 9]
    s = Setup([p + m for p, m in zip(past, new)], H=H, kv=kv, act=act, B=B, seed=G * H)
    mask = random_tree_mask(new, torch.Generator().manual_seed(G))
    q, out = tree(s, new, mask, H * G)
    s.check(new, q, out, SCALE, mask=mask)
    assert pa.pa_check_device_errors(s.pool) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp16", "fp8_e4m3"])
@pytest.mark.parametrize("lens,new,G,H", [([33000], [12], 8, 2), ([5000, 130, 64], [64, 64, 64], 8, 1),
                                          ([20000, 19000], [64, 3], 1, 2)])
def test_trees_over_long_caches(kv, lens, new, G, H):
    s = Setup(lens, H=H, kv=kv, seed=2)
    mask = random_tree_mask(new, torch.Generator().manual_seed(8))
    q, out = tree(s, new, mask, H * G)
    s.check(new, q, out, SCALE, mask=mask)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_any_mask_and_rows_that_attend_nothing(kv):
    past, new = [0, 0, 300, 0], [64, 7, 64, 20]
    s = Setup([p + m for p, m in zip(past, new)], H=2, kv=kv, seed=6)
    g = torch.Generator().manual_seed(3)
    mask = torch.randint(-2 ** 63, 2 ** 63 - 1, (sum(new),), generator=g).cuda()   # bits past the drafts as well
    mask[::3] = 0
    mask[5], mask[70] = -1, -(2 ** 63)
    q, out = tree(s, new, mask, 16)
    inside = torch.cat([torch.full((m,), (1 << m) - 1 if m < 64 else -1) for m in new]).cuda()
    s.check(new, q, out, SCALE, mask=mask & inside)
    empty = (mask & inside) == 0
    empty[71:71 + 64] = False                       # the third sequence has a prefix
    assert empty.any() and (out[empty] == 0).all()


def test_drafts_in_a_chain_equal_a_causal_chunk():
    lens, new = [300, 77, 1000], [64, 9, 33]
    s = Setup(lens, H=2, seed=1)
    chain = torch.cat([(torch.ones(m, dtype=torch.int64) << torch.arange(m)) * 2 - 1 for m in new]).cuda()
    q, a = prefill(s, new, 8)
    b = torch.empty_like(a)
    pa.pa_tree_attention(s.pool, 0, new, chain, q, b, SCALE, kv_lens=s.lens, block_tables=s.tables)
    s.check(new, q, a, SCALE)
    s.check(new, q, b, SCALE)


def test_uint64_masks():
    s = Setup([64], H=1, seed=1)
    mask = random_tree_mask([64], torch.Generator().manual_seed(1))
    q, a = tree(s, [64], mask, 4)
    b = torch.empty_like(a)
    pa.pa_tree_attention(s.pool, 0, [64], mask.view(torch.uint64), q, b, SCALE, kv_lens=s.lens, block_tables=s.tables)
    assert torch.equal(a, b)


def test_the_pools_own_tables():
    """Sequences that the pool's block manager holds, forked ones and one named twice."""
    s = Setup([], H=2, mbps=40, num_blocks=200)
    p = pa.pa_pool_create(num_layers=1, num_kv_heads=2, block_size=16, num_blocks=200, max_seqs=6,
                          max_blocks_per_seq=40, kv_dtype="bf16", k_cache=s.cache[0], v_cache=s.cache[1],
                          free_order=torch.randperm(200, generator=torch.Generator().manual_seed(2)).numpy())
    lens = {0: 300, 3: 77, 5: 33}
    for i, n in lens.items():
        pa.pa_alloc_blocks(p, i, n)
        pa.pa_append_kv(p, 0, [i] * n, list(range(n)), s.rand(n, 2), s.rand(n, 2))
    pa.pa_fork_cow(p, 0, 1)
    pa.pa_alloc_blocks(p, 1, 304)                         # copies the shared tail block
    pa.pa_append_kv(p, 0, [1] * 4, list(range(300, 304)), s.rand(4, 2), s.rand(4, 2))
    seqs, new = [3, 0, 1, 5, 3], [77, 300, 10, 0, 4]
    s.pool, s.lens = p, [pa.pa_get_seq(p, i)[0] for i in seqs]
    s.tables = torch.tensor([(pa.pa_get_seq(p, i)[1] + [0] * 40)[:40] for i in seqs], device="cuda")
    q, out = prefill(s, new, 8, seqs=seqs)
    s.check(new, q, out, SCALE)
    new = [5, 6, 4, 1, 2]
    mask = random_tree_mask(new, torch.Generator().manual_seed(8))
    q, out = tree(s, new, mask, 8, seqs=seqs)
    s.check(new, q, out, SCALE, mask=mask)
    assert pa.pa_check_device_errors(p) == 0


def test_results_do_not_depend_on_placement_or_repetition():
    lens, new = [2000, 900, 5000], [300, 900, 40]
    outs = []
    for seed in (0, 1):
        s = Setup(lens, H=2, kv="bf16", seed=7)
        if seed:                                          # the same rows in other blocks
            nb = s.cache[0].shape[1]
            perm = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).cuda()
            for c in s.cache:
                c[:, perm] = c.clone()
            s.tables = torch.where(s.tables >= 0, perm[s.tables.long().clamp(min=0)].int(), s.tables)
        s.gen = torch.Generator(device="cuda").manual_seed(1)
        q, out = prefill(s, new, 16)
        again = torch.empty_like(out)
        pa.pa_prefill_attention(s.pool, 0, new, q, again, SCALE, kv_lens=s.lens, block_tables=s.tables)
        assert torch.equal(out, again)
        drafts = [40, 3, 64]
        mask = random_tree_mask(drafts, torch.Generator().manual_seed(1))
        _, t = tree(s, drafts, mask, 16)
        outs.append((out, t))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_rows_around_the_call_stay():
    """Padding rows of q / out before and behind the packed tokens."""
    lens = [130, 5]
    s = Setup(lens, H=1, seed=1)
    q = s.rand(200, 8)
    q[:20] = q[155:] = float("nan")
    out = torch.full_like(q, 7.0)
    pa.pa_prefill_attention(s.pool, 0, lens, q[20:155], out[20:155], SCALE, kv_lens=lens, block_tables=s.tables)
    s.check(lens, q[20:155], out[20:155], SCALE)
    assert (out[:20] == 7).all() and (out[155:] == 7).all()


@pytest.mark.parametrize("kv,act", KINDS)
@pytest.mark.parametrize("lens,new", [([300, 40], [300, 40]), ([9000], [20]), ([2000] * 10, [600] * 10)])
def test_a_nan_query_gives_a_nan_row_and_no_other(kv, act, lens, new):
    """Whole, split and paired tiles; an infinite query element gives no finite row either."""
    s = Setup(lens, H=4, kv=kv, act=act, seed=2)
    q = s.rand(sum(new), 16, 2.0)
    clean = q.clone()
    q[7, 3, 5] = float("nan")
    q[11, 9, 100] = float("inf")
    out = torch.zeros_like(q)
    pa.pa_prefill_attention(s.pool, 0, new, q, out, SCALE, kv_lens=lens, block_tables=s.tables)
    assert torch.isnan(out[7, 3]).all() and not torch.isfinite(out[11, 9]).any()
    ref = torch.zeros_like(q)
    pa.pa_prefill_attention(s.pool, 0, new, clean, ref, SCALE, kv_lens=lens, block_tables=s.tables)
    s.check(new, clean, ref, SCALE)
    out[7, 3], out[11, 9] = ref[7, 3], ref[11, 9]
    s.check(new, clean, out, SCALE)


@pytest.mark.parametrize("lens,new", [([130, 5], [130, 5]), ([9000], [20]), ([2000] * 10, [600] * 10)])
def test_queries_and_output_at_sixteen_byte_addresses(lens, new):
    """q and out need 16-byte alignment, not more (whole, split and paired tiles)."""
    s = Setup(lens, H=4, seed=1)
    rows = sum(new)
    q = torch.empty(rows * 16 * 128 + 8, dtype=DT["bf16"], device="cuda")[8:].view(rows, 16, 128)
    whole = torch.full((rows * 16 * 128 + 16,), 7.0, dtype=DT["bf16"], device="cuda")
    out = whole[8:-8].view(rows, 16, 128)
    assert q.data_ptr() % 32 == 16 and out.data_ptr() % 32 == 16
    q.copy_(s.rand(rows, 16, 2.0))
    pa.pa_prefill_attention(s.pool, 0, new, q, out, SCALE, kv_lens=lens, block_tables=s.tables)
    s.check(new, q, out, SCALE)
    assert (whole[:8] == 7).all() and (whole[-8:] == 7).all()


def test_other_stream_and_graph_replay():
    lens, new = [600, 9000, 64], [600, 16, 64]
    s = Setup(lens, H=2, seed=5)
    drafts = [30, 16, 64]
    mask = random_tree_mask(drafts, torch.Generator().manual_seed(1))
    q, qt = s.rand(sum(new), 16, 2.0), s.rand(sum(drafts), 16, 2.0)
    out, outt = torch.zeros_like(q), torch.zeros_like(qt)
    st = torch.cuda.Stream()

    def both():
        pa.pa_prefill_attention(s.pool, 0, new, q, out, SCALE, kv_lens=lens, block_tables=s.tables)
        pa.pa_tree_attention(s.pool, 0, drafts, mask, qt, outt, SCALE, kv_lens=lens, block_tables=s.tables)
        pa.pa_prefill_attention(s.pool, 0, new, q, out, SCALE, kv_lens=lens, block_tables=s.tables)

    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        both()
    st.synchronize()
    s.check(new, q, out, SCALE)
    s.check(drafts, qt, outt, SCALE, mask=mask)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        both()
    for k in range(3):
        q.copy_(s.rand(sum(new), 16, 2.0))
        qt.copy_(s.rand(sum(drafts), 16, 2.0))
        mask.copy_(random_tree_mask(drafts, torch.Generator().manual_seed(k + 5)))
        g.replay()
        torch.cuda.synchronize()
        s.check(new, q, out, SCALE)
        s.check(drafts, qt, outt, SCALE, mask=mask)
    assert pa.pa_check_device_errors(s.pool) == 0


def test_a_pools_first_call_may_be_captured():
    """Its counters are set when the call is captured, not at the first replay, and a
    replay does not clear an error that a call before it found."""
    lens, new = [600, 9000, 64], [600, 16, 64]
    s = Setup(lens, H=2, seed=6)
    s.pool.workspace.fill_(0xFF)
    q = s.rand(sum(new), 16, 2.0)
    out, eager = torch.zeros_like(q), torch.zeros_like(q)
    torch.cuda.synchronize()
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        pa.pa_prefill_attention(s.pool, 0, new, q, out, SCALE, kv_lens=lens, block_tables=s.tables)
    pa.pa_prefill_attention(s.pool, 0, new, q, eager, SCALE, kv_lens=lens, block_tables=s.tables)
    torch.cuda.synchronize()
    s.check(new, q, eager, SCALE)
    assert pa.pa_check_device_errors(s.pool) == 0
    bad = s.tables.clone()
    bad[0, 0] = -1                                        # block 0 is read instead
    pa.pa_prefill_attention(s.pool, 0, new, q, eager, SCALE, kv_lens=lens, block_tables=bad)
    torch.cuda.synchronize()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    s.check(new, q, out, SCALE)
    assert pa.pa_check_device_errors(s.pool) == pa.PA_DEVERR_BAD_BLOCK


def test_chained_calls_on_the_default_stream():
    """Launches may begin while the kernel before them runs: rows that one call writes
    and the next reads, with torch kernels between and around them, 40 times over."""
    H, G, n, B = 2, 8, 3, 16
    s = Setup([], H=H, mbps=20, num_blocks=60, seed=3)
    dev = dict(dtype=torch.int32, device="cuda")
    free = torch.randperm(60, generator=torch.Generator().manual_seed(4)).to(torch.int32).cuda()
    head, old, lens = torch.zeros(1, **dev), [0] * n, [260, 7, 33]
    cu, slots = torch.zeros(n + 1, **dev), torch.zeros(300, **dev)
    s.tables, s.lens = torch.zeros((n, 20), **dev), lens
    a, b = torch.tensor(old, **dev), torch.tensor(lens, **dev)
    drafts = [17, 7, 20]
    mask = random_tree_mask(drafts, torch.Generator().manual_seed(2))
    k, v, q = s.rand(300, H), s.rand(300, H), s.rand(300, H * G, 2.0)
    qt = q[:sum(drafts)].contiguous()
    results = []
    for i in range(40):
        s.tables.fill_(-1)
        head.zero_()
        slots.fill_(-1)
        for c in s.cache:
            c.view(torch.uint8).fill_(0xFF)
        out, outt = torch.full_like(q, float("nan")), torch.full_like(qt, float("nan"))
        pa.pa_build_tables(s.pool, a, b, free, head, head, s.tables, cu, slots)
        pa.pa_append_kv_slots(s.pool, 0, slots, k, v)
        pa.pa_prefill_attention(s.pool, 0, lens, q, out, SCALE, kv_lens=lens, block_tables=s.tables)
        pa.pa_tree_attention(s.pool, 0, drafts, mask, qt, outt, SCALE, kv_lens=lens, block_tables=s.tables)
        results.append((out, outt))
        qn = qt * 1.0                                     # a torch kernel right behind
        qt, _ = qn, results
    torch.cuda.synchronize()
    s.check(lens, q, results[0][0], SCALE)
    s.check(drafts, qt, results[0][1], SCALE, mask=mask)
    for out, outt in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(outt, results[0][1])
    assert pa.pa_check_device_errors(s.pool) == 0


def test_a_corrupt_table_entry_is_reported():
    for bad in (-1, 10 ** 6):
        s = Setup([300, 40], H=1, seed=5)
        s.tables[0, 3] = bad
        for c in s.cache:
            c[0][0] = 1.0                                 # block 0 is read instead
        q, out = prefill(s, [300, 40], 8)
        assert pa.pa_check_device_errors(s.pool) == pa.PA_DEVERR_BAD_BLOCK
        assert pa.pa_check_device_errors(s.pool) == 0
        mask = torch.ones(4, dtype=torch.int64, device="cuda")
        tree(s, [2, 2], mask, 8)
        assert pa.pa_check_device_errors(s.pool) == pa.PA_DEVERR_BAD_BLOCK


def test_caches_past_32_bits():
    """Blocks whose element offsets pass 2^31 and 2^32."""
    nb = (1 << 18) + 100
    s = Setup([], H=8, kv="fp8_e4m3", mbps=16, num_blocks=nb)
    lens = [200]
    ids = torch.tensor([nb - 1 - 7 * i for i in range(6)] + [nb // 2 + i for i in range(7)], dtype=torch.int32)
    s.tables = torch.zeros((1, 16), dtype=torch.int32)
    s.tables[0, :13] = ids
    s.tables, s.lens = s.tables.cuda(), lens
    pos = torch.arange(200, device="cuda")
    for c in s.cache:
        c[0][s.tables[0].long()[pos // 16], :, pos % 16] = torch.randint(0, 0x7F, (200, 8, 128), device="cuda").to(torch.uint8)
    q, out = prefill(s, lens, 64)
    s.check(lens, q, out, SCALE)
    mask = random_tree_mask([33], torch.Generator().manual_seed(1))
    q, out = tree(s, [33], mask, 64)
    s.check([33], q, out, SCALE, mask=mask)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_a_serving_step_from_lengths_to_drafts(kv):
    """Lengths on the GPU -> tables and slots -> append -> prompt attention -> one decode
    step through the device tables -> drafted tokens and their tree."""
    H, G, B, n = 2, 4, 16, 5
    s = Setup([], H=H, kv=kv, mbps=30, num_blocks=150, seed=1)
    dev = dict(dtype=torch.int32, device="cuda")
    free = torch.randperm(150, generator=torch.Generator().manual_seed(4)).to(torch.int32).cuda()
    head, tables = torch.zeros(1, **dev), torch.full((n, 30), -1, **dev)
    cu, slots = torch.zeros(n + 1, **dev), torch.zeros(1000, **dev)
    lens = [0] * n
    s.tables = tables
    for step, new in enumerate(([5, 200, 16, 129, 77], [1] * n, [8, 64, 1, 30, 17])):
        old, lens = lens, [a + m for a, m in zip(lens, new)]
        T = sum(new)
        pa.pa_build_tables(s.pool, torch.tensor(old, **dev), torch.tensor(lens, **dev), free, head, head, tables, cu,
                           slots)
        k, v = s.rand(1000, H), s.rand(1000, H)
        pa.pa_append_kv_slots(s.pool, 0, slots, k, v)     # the padded map: rows behind the tokens are skipped
        s.lens = lens
        if step == 0:
            q, out = prefill(s, new, H * G)
            s.check(new, q, out, SCALE)
            continue
        if step == 1:
            q, out = s.rand(n, H * G, 2.0), torch.empty((n, H * G, 128), dtype=DT[s.act], device="cuda")
            pa.pa_decode_attention_noalloc(s.pool.desc, 0, tables, lens, q, out, SCALE)
            assert pa.pa_noalloc_check_errors(0) == 0
            chunk = torch.empty_like(out)
            pa.pa_prefill_attention(s.pool, 0, new, q, chunk, SCALE, kv_lens=lens, block_tables=tables)
            s.check(new, q, chunk, SCALE)
            s.check(new, q, out, SCALE)
            continue
        mask = random_tree_mask(new, torch.Generator().manual_seed(5))
        q, out = tree(s, new, mask, H * G)
        s.check(new, q, out, SCALE, mask=mask)
        # stored rows are the appended ones
        if kv == "bf16":
            for i, m in enumerate(new):
                a = int(cu[i])
                assert torch.equal(s.rows(0, i, lens[i])[-m:], k[a:a + m].double())
    assert int(head) == sum(-(-x // B) for x in lens)
    assert pa.pa_check_device_errors(s.pool) == 0
