"""Sizes at which building block tables changes its kernel or its launch.  Whole numbers:
every comparison is exact."""
import os
import random
import subprocess
import sys

import pytest
import torch

import pagedattention_decode_03_b200 as pa
from prompt_reference import tables_reference

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

# n requests of one token each through a slot map of `cap` entries, in a process whose first
# call this is: what an earlier call with more requests asked for must not be needed.
ONE_CALL = """
import sys
sys.path[:0] = [{root!r}]
import torch, pagedattention_decode_03_b200 as pa
n, cap = {n}, {cap}
i32 = lambda k, v=0: torch.full((k,), v, dtype=torch.int32, device="cuda")
p = pa.pa_pool_create(num_layers=1, num_kv_heads=1, block_size=16, num_blocks=n, max_seqs=n, max_blocks_per_seq=1)
free, cu, slots, head, tables = torch.randperm(n).to(torch.int32).cuda(), i32(n + 1), i32(cap, -9), i32(1), i32(n, -7).view(n, 1)
pa.pa_build_tables(p, i32(n), i32(n, 1), free, head, head, tables, cu, slots)
assert pa.pa_check_device_errors(p) == 0
assert torch.equal(cu.cpu(), torch.arange(n + 1, dtype=torch.int32)) and int(head) == n
assert torch.equal(tables[:, 0], free) and torch.equal(slots[:n], free * 16) and bool((slots[n:] == -1).all())
"""


@pytest.mark.parametrize("n", [4072, 4073, 4095, 4096, 8192])
@pytest.mark.parametrize("cap", [9001, 400001])
def test_the_first_call_of_a_process(n, cap):
    """Sums of many requests take more shared memory than a launch has unasked."""
    r = subprocess.run([sys.executable, "-c", ONE_CALL.format(root=os.path.dirname(HERE), n=n, cap=cap)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def requests(n, B, hi, total, seed):
    """n requests of up to `hi` new tokens (none for some), about `total` in all, with their
    tables so far, free ids and sizes."""
    r = random.Random(seed)
    old = [r.choice((0, r.randint(0, 40), 3 * B)) for _ in range(n)]
    new = [a + (0 if r.random() < 0.1 else r.randint(1, hi)) for a in old]
    scale = total / max(1, sum(new) - sum(old))
    new = [a + int((b - a) * min(1.0, scale)) for a, b in zip(old, new)]
    mbps = max(-(-b // B) for b in new) + 1
    nb = sum(-(-b // B) for b in new) + 5
    ids = list(range(nb))
    r.shuffle(ids)
    tables, at = [], 0
    for a in old:
        k = -(-a // B)
        tables.append(ids[at:at + k] + [-5] * (mbps - k))
        at += k
    return old, new, tables, ids[at:], mbps, nb


class Call:
    """One build of tables into a slot map of `cap` entries that starts `off` entries into a
    16-byte aligned buffer, the words around it watched."""

    def __init__(self, old, new, tables, free, mbps, nb, B, cap, off=0):
        n = len(old)
        self.pool = pa.pa_pool_create(num_layers=1, num_kv_heads=1, block_size=B, num_blocks=nb, max_seqs=n,
                                      max_blocks_per_seq=mbps)
        self.tables, self.head, self.cap = i32(tables).view(n, mbps), i32([2]), cap
        self.cu = torch.full((n + 1,), -9, dtype=torch.int32, device="cuda")
        self.whole = torch.full((cap + 8,), -9, dtype=torch.int32, device="cuda")
        self.slots = self.whole[off:off + cap]
        self.off = off
        self.args = (i32(old), i32(new), i32([0, 0] + free))

    def run(self, **kw):
        old, new, free = self.args
        pa.pa_build_tables(self.pool, old, new, free, self.head, self.head, self.tables, self.cu, self.slots, **kw)

    def check(self, want):
        tables, cu, slots, head = want
        assert self.head.tolist() == [head] and self.cu.tolist() == cu
        assert torch.equal(self.slots.cpu(), torch.tensor(slots, dtype=torch.int32))
        assert torch.equal(self.tables.cpu(), torch.tensor(tables, dtype=torch.int32))
        assert (self.whole[:self.off] == -9).all() and (self.whole[self.off + self.cap:] == -9).all()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("B", [16, 32])
@pytest.mark.parametrize("per_sm,extra,off", [(2048, 0, 0), (2048, 1, 0), (2048, 39, 1), (8192, 0, 0), (8192, 16, 3),
                                              (8192, 30001, 2)])
@pytest.mark.parametrize("n,hi", [(60, 30000), (8192, 170)])
def test_large_maps(B, per_sm, extra, off, n, hi):
    """Sixteen slots a thread (from 2,048 an SM on), and more than a round of the grid (8,192):
    few long and many short requests, maps filled, padded and at odd addresses."""
    cap = sms() * per_sm + extra
    old, new, tables, free, mbps, nb = requests(n, B, hi, cap - 1000 * (extra % 2), n + per_sm + extra)
    c = Call(old, new, tables, free, mbps, nb, B, cap, off)
    c.run()
    assert pa.pa_check_device_errors(c.pool) == 0
    c.check(tables_reference(old, new, [0, 0] + free, 2, tables, B, cap))


def test_large_maps_of_nothing_and_of_too_much():
    """No new token, too few ids, one token more than the map holds, and a bad id."""
    B, cap = 16, sms() * 2048 + 77
    old, new, tables, free, mbps, nb = requests(300, B, 4000, cap - 500, 1)
    need = sum(-(-b // B) - -(-a // B) for a, b in zip(old, new))
    total = sum(new) - sum(old)
    c = Call(old, old, tables, free, mbps, nb, B, cap)
    c.run()
    c.check((tables, [0] * 301, [-1] * cap, 2))
    assert pa.pa_check_device_errors(c.pool) == 0
    c = Call(old, new, tables, free[:need - 1], mbps, nb, B, cap)
    c.run()
    c.check((tables, [0] * 301, [-1] * cap, 2))
    assert pa.pa_check_device_errors(c.pool) == pa.PA_DEVERR_NO_BLOCKS
    more = list(new)
    more[7] += cap + 1 - total
    mb = max(mbps, -(-more[7] // B))
    wide = [t + [-5] * (mb - mbps) for t in tables]
    c = Call(old, more, wide, free + [1] * cap, mb, nb, B, cap)
    c.run()
    c.check((wide, [0] * 301, [-1] * cap, 2))
    assert pa.pa_check_device_errors(c.pool) == pa.PA_DEVERR_BAD_LEN
    ids = list(free)
    ids[5], ids[need - 2] = nb, -1
    c = Call(old, new, tables, ids, mbps, nb, B, cap)
    c.run()
    t, cu, slots, head = tables_reference(old, new, [0, 0] + ids, 2, tables, B, cap)
    c.check((t, cu, [x if 0 <= x < nb * B else -1 for x in slots], head))
    assert pa.pa_check_device_errors(c.pool) == pa.PA_DEVERR_BAD_BLOCK


def test_large_maps_on_another_stream_and_replayed():
    B, cap = 16, sms() * 2048 + 5
    old, new, tables, free, mbps, nb = requests(200, B, 4000, cap, 9)
    want = tables_reference(old, new, [0, 0] + free, 2, tables, B, cap)
    c = Call(old, new, tables, free, mbps, nb, B, cap)
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        c.run()
    st.synchronize()
    c.check(want)
    with torch.cuda.graph(g, stream=st):
        c.run()
    for _ in range(2):
        c.head.fill_(2)
        c.slots.fill_(-9)
        c.tables.copy_(i32(tables).view(200, mbps))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        c.check(want)
    assert pa.pa_check_device_errors(c.pool) == 0


@pytest.mark.parametrize("kv,act", [("bf16", "bf16"), ("fp16", "fp16"), ("fp8_e4m3", "bf16"), ("fp8_e4m3", "fp16")])
def test_large_appends_chained_with_their_tables(kv, act):
    """Calls that overlap on the default stream, chained, with torch kernels that write what
    they read and read what they write right before and behind them: the stored rows are
    those that pa_append_kv stores."""
    B, H, n, cap = 16, 8, 40, sms() * 2048 + 9
    T = 12001
    dt = torch.bfloat16 if act == "bf16" else torch.float16
    new = [300] * n
    new[-1] += T - 2 - sum(new)                           # two rows of the map stay free
    mbps = -(-max(new) // B)
    nb = sum(-(-x // B) for x in new) + 3
    g = torch.Generator(device="cuda").manual_seed(3)
    kw = {}
    if kv == "fp8_e4m3":
        sc = [torch.rand((1, H), generator=g, device="cuda") * 0.02 + 0.004 for _ in range(2)]
        kw = dict(k_scale=sc[0], v_scale=sc[1], k_inv_scale=1 / sc[0], v_inv_scale=1 / sc[1])
    order = torch.randperm(nb, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    p, ref = [pa.pa_pool_create(num_layers=1, num_kv_heads=H, block_size=B, num_blocks=nb, max_seqs=n, kv_dtype=kv,
                                act_dtype=act, max_blocks_per_seq=mbps, free_order=order.numpy(), **kw) for _ in range(2)]
    rows = [(torch.randn((T, H, 128), generator=g, device="cuda") * 2).to(dt) for _ in range(2)]
    pa.pa_alloc_blocks_n(ref, list(range(n)), new)
    pa.pa_append_kv(ref, 0, [i for i in range(n) for _ in range(new[i])], [t for x in new for t in range(x)],
                    rows[0][:T - 2].contiguous(), rows[1][:T - 2].contiguous())
    zero, lens, free = i32([0] * n), i32(new), order.cuda()
    old, want = zero.clone(), lens.clone()
    head, cu, slots, tables = i32([0]), i32([0] * (n + 1)), i32([-1] * cap), torch.full((n, mbps), -1, dtype=torch.int32, device="cuda")
    x = [torch.empty_like(r) for r in rows]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        want.copy_(zero)
        for c in (p.k_cache, p.v_cache):
            c.view(torch.uint8).zero_()
        head.zero_()
        for a, b in zip(x, rows):
            a.copy_(b)
        want.copy_(lens)                                  # right before the call that reads it
        pa.pa_build_tables(p, old, want, free, head, head, tables, cu, slots)
        pa.pa_append_kv_slots(p, 0, slots[:T], x[0], x[1])
        got.append([c.clone() for c in (p.k_cache, p.v_cache)])
        for a in x:
            a.zero_()
    torch.cuda.synchronize()
    for k, v in got:
        assert torch.equal(k.view(torch.uint8), ref.k_cache.view(torch.uint8))
        assert torch.equal(v.view(torch.uint8), ref.v_cache.view(torch.uint8))
    assert pa.pa_check_device_errors(p) == 0


def test_lengths_near_32_bits_leave_their_request_alone():
    """A length within 255 of 2^31 cannot be rounded up to blocks in 32 bits."""
    B, mbps = 16, 1 << 27
    p = pa.pa_pool_create(num_layers=1, num_kv_heads=1, block_size=B, num_blocks=64, max_seqs=1, max_blocks_per_seq=mbps,
                          min_partition_tokens=1 << 24)
    tables = torch.full((1, mbps), 7, dtype=torch.int32, device="cuda")
    free, head, cu, slots = i32(list(range(64))), i32([5]), i32([-9, -9]), i32([-9] * 40)
    for old, new, ok in ((2 ** 31 - 20, 2 ** 31 - 1, False), (2 ** 31 - 270, 2 ** 31 - 255, False),
                         (2 ** 31 - 280, 2 ** 31 - 256, True)):
        pa.pa_build_tables(p, i32([old]), i32([new]), free, head, head, tables, cu, slots)
        assert pa.pa_check_device_errors(p) == (0 if ok else pa.PA_DEVERR_BAD_LEN)
        if not ok:
            assert cu.tolist() == [0, 0] and slots.tolist() == [-1] * 40 and head.tolist() == [5]
            assert int((tables != 7).sum()) == 0
    a, b = 2 ** 31 - 280, 2 ** 31 - 256                    # 2^31 - 272 begins a fresh block
    assert cu.tolist() == [0, b - a] and head.tolist() == [6] and int((tables != 7).sum()) == 1
    assert int(tables[0, (b - 1) // B]) == 5
    assert slots.tolist() == [(7 if t < 2 ** 31 - 272 else 5) * B + t % B for t in range(a, b)] + [-1] * 16
