"""Order of the prompt-side calls: on the legacy default stream against blocking streams,
and of a pool's first call after what its stream was given before.

A launch that may begin while the kernel before it runs must still come after work that
other blocking streams were given before it, and that work must come after all of the
launch.  Buffers only change between valid values, so a missed order shows as a wrong
result.  References: the same calls with a synchronisation between them.
"""
import math

import pytest
import torch

import pagedattention_decode_03_b200 as pa
from prompt_reference import Setup, random_tree_mask, tables_reference

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)


@pytest.fixture
def blocking():
    """A stream that the legacy default stream waits for, and that waits for it."""
    import ctypes
    handle = ctypes.c_void_p()
    assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(handle))) == 0
    torch.cuda.synchronize()
    yield torch.cuda.ExternalStream(handle.value)
    torch.cuda.synchronize()
    assert int(torch.cuda.cudart().cudaStreamDestroy(handle.value)) == 0


@pytest.mark.parametrize("lens,new", [([130, 77], [130, 77]), ([9000], [20]), ([2000] * 10, [600] * 10)],
                         ids=["whole", "split", "paired"])
def test_attention_between_work_of_a_blocking_stream(blocking, lens, new):
    """Queries are replaced, and results copied away, by a blocking stream between calls."""
    s = Setup(lens, H=4, seed=3)
    qs = [s.rand(sum(new), 16, 2.0) for _ in range(4)]
    few = [min(m, 30) for m in new]
    mask = random_tree_mask(few, torch.Generator().manual_seed(2))
    own = dict(kv_lens=lens, block_tables=s.tables)

    def prefill(q, out):
        pa.pa_prefill_attention(s.pool, 0, new, q, out, SCALE, **own)

    def tree(q, out):
        pa.pa_tree_attention(s.pool, 0, few, mask, q, out, SCALE, **own)

    want = []
    for x in qs:
        a, b = torch.empty_like(x), torch.empty_like(x[:sum(few)])
        prefill(x, a)
        tree(x[:sum(few)], b)
        torch.cuda.synchronize()
        want.append((a, b))
    q = qs[0].clone()
    a, b = torch.empty_like(q), torch.empty_like(q[:sum(few)])
    got = [[torch.empty_like(x) for x in (a, b)] for _ in range(24)]
    torch.cuda.synchronize()
    for i in range(24):
        with torch.cuda.stream(blocking):
            torch.cuda._sleep(200000)                     # ~0.1 ms: a launch that did not wait would be done by then
            q.copy_(qs[i % 4])
        prefill(q, a)
        tree(q[:sum(few)], b)
        with torch.cuda.stream(blocking):
            got[i][0].copy_(a)
            got[i][1].copy_(b)
            a.zero_()
            b.zero_()
    torch.cuda.synchronize()
    for i in range(24):
        assert torch.equal(got[i][0], want[i % 4][0]) and torch.equal(got[i][1], want[i % 4][1]), i
    assert pa.pa_check_device_errors(s.pool) == 0


def test_large_tables_and_appends_between_work_of_a_blocking_stream(blocking):
    """Calls large enough to overlap on the default stream (many slots a thread; more than
    a thousand CTAs of rows): lengths, slots and rows are replaced and results copied away
    by a blocking stream."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B, H, n, mbps = 16, 8, 300, 260
    nb, T, cap = n * mbps, 20000, sms * 2048 + 37
    p = pa.pa_pool_create(num_layers=1, num_kv_heads=H, block_size=B, num_blocks=nb, max_seqs=n, max_blocks_per_seq=mbps)
    g = torch.Generator().manual_seed(1)
    dev = dict(dtype=torch.int32, device="cuda")
    free = torch.randperm(nb, generator=g).to(torch.int32).cuda()
    lens = [[int(x) for x in torch.randint(0, 1000, (n,), generator=g)] for _ in range(2)]
    new_of = [torch.tensor(x, **dev) for x in lens]
    rows = [torch.full((T, H, 128), 1.0 + i, dtype=torch.bfloat16, device="cuda") for i in range(2)]
    old, new = torch.zeros(n, **dev), torch.zeros(n, **dev)
    head, head_out, cu = torch.zeros(1, **dev), torch.zeros(1, **dev), torch.zeros(n + 1, **dev)
    tables, slots, x = torch.full((n, mbps), -1, **dev), torch.full((cap,), -1, **dev), rows[0].clone()
    got = []
    torch.cuda.synchronize()
    for i in range(12):
        with torch.cuda.stream(blocking):
            torch.cuda._sleep(200000)
            new.copy_(new_of[i % 2])
            x.copy_(rows[i % 2])
        pa.pa_build_tables(p, old, new, free, head, head_out, tables, cu, slots)
        pa.pa_append_kv_slots(p, 0, slots[:T], x, x)
        with torch.cuda.stream(blocking):
            got.append((slots.clone(), cu.clone(), head_out.clone(), p.k_cache.amax(), p.v_cache.amax()))
            slots.fill_(-1)
            p.k_cache.zero_()
            p.v_cache.zero_()
    torch.cuda.synchronize()
    assert pa.pa_check_device_errors(p) == 0
    want = [tables_reference([0] * n, x, free.tolist(), 0, [[-1] * mbps] * n, B, cap) for x in lens]
    for i, (sl, c, h, k, v) in enumerate(got):
        _, cu_w, slots_w, head_w = want[i % 2]
        assert c.tolist() == cu_w and h.tolist() == [head_w] and sl.tolist() == slots_w, i
        assert float(k) == float(v) == 1.0 + i % 2


# ---------------------------------------------------------- a pool's first call
LENS, NEW = [600, 9000, 64], [600, 16, 64]


def queue_fill(s, stream):
    """~50 ms of work and, behind it, bytes over the whole workspace, on `stream`."""
    with torch.cuda.stream(stream):
        for _ in range(5):
            torch.cuda._sleep(20_000_000)
        s.pool.workspace.fill_(0xFF)


def attend(s, q, out, tables=None):
    pa.pa_prefill_attention(s.pool, 0, NEW, q, out, SCALE, kv_lens=LENS, block_tables=s.tables if tables is None else tables)


@pytest.mark.parametrize("captured", [False, True])
def test_a_first_call_comes_after_what_writes_the_workspace(captured):
    """The workspace may still be written when the call is made (or captured): the call's
    own setting of it comes behind that."""
    s, warm = Setup(LENS, H=2, seed=6), Setup(LENS, H=2, seed=6)
    q = s.rand(sum(NEW), 16, 2.0)
    out = torch.full_like(q, float("nan"))
    attend(warm, q, out)                                  # kernels are loaded, which may wait for the device
    out.fill_(float("nan"))
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    queue_fill(s, st)
    with torch.cuda.stream(st):
        if captured:
            g.capture_begin()
            attend(s, q, out)
            attend(s, q, out)
            g.capture_end()
            assert not st.query()                         # what was queued before is still running
            g.replay()
            g.replay()
        else:
            attend(s, q, out)
            assert not st.query()
    torch.cuda.synchronize()
    s.check(NEW, q, out, SCALE)
    assert pa.pa_check_device_errors(s.pool) == 0


def test_captured_calls_only():
    """No call of the pool is ever made outside a capture: the state is set at the first
    replay of whichever graph comes first, once; errors collect over replays."""
    s = Setup(LENS, H=2, seed=7)
    s.pool.workspace.fill_(0xFF)
    q = s.rand(sum(NEW), 16, 2.0)
    bad = s.tables.clone()
    bad[0, 0] = -1                                        # block 0 is read instead
    outs = [torch.full_like(q, float("nan")) for _ in range(2)]
    st, graphs = torch.cuda.Stream(), [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    for g, out, tab in zip(graphs, outs, (s.tables, bad)):
        with torch.cuda.graph(g, stream=st):
            attend(s, q, out, tab)
            attend(s, q, out, tab)
    assert pa.pa_check_device_errors(s.pool) == 0         # nothing has run
    for k in (1, 0, 0):
        graphs[k].replay()
    torch.cuda.synchronize()
    assert pa.pa_check_device_errors(s.pool) == pa.PA_DEVERR_BAD_BLOCK
    assert pa.pa_check_device_errors(s.pool) == 0
    s.check(NEW, q, outs[0], SCALE)
    graphs[0].replay()
    attend(s, q, outs[1])
    torch.cuda.synchronize()
    s.check(NEW, q, outs[1], SCALE)
    assert pa.pa_check_device_errors(s.pool) == 0


def test_one_workspace_of_two_pools_in_turn():
    """A pool over the buffer of an earlier one sets it anew."""
    s = Setup(LENS, H=2, seed=8)
    q = s.rand(sum(NEW), 16, 2.0)
    out = torch.empty_like(q)
    bad = s.tables.clone()
    bad[0, 0] = -1
    attend(s, q, out, bad)                                # leaves an error behind
    torch.cuda.synchronize()
    first = s.pool
    s.pool = pa.pa_pool_create(num_layers=1, num_kv_heads=2, block_size=16, num_blocks=s.cache[0].shape[1],
                               max_seqs=len(LENS), max_blocks_per_seq=s.mbps, kv_dtype="bf16", k_cache=s.cache[0],
                               v_cache=s.cache[1], workspace=first.workspace)
    attend(s, q, out)
    torch.cuda.synchronize()
    s.check(NEW, q, out, SCALE)
    assert pa.pa_check_device_errors(s.pool) == 0
