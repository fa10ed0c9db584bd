"""Block tables and slot maps built on the GPU, and the append that reads them.

Whole numbers and stored bits: every comparison is exact.  References: plain
integer arithmetic, and pa_append_kv for the stored rows.
"""
import random

import numpy as np
import pytest
import torch

import pagedattention_decode_03_b200 as pa
from prompt_reference import DT, tables_reference

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool_of(n, mbps, nb, B=16, **kw):
    return pa.pa_pool_create(num_layers=kw.pop("layers", 1), num_kv_heads=kw.pop("H", 1), block_size=B,
                             num_blocks=nb, max_seqs=max(n, 1), max_blocks_per_seq=mbps, **kw)


def case(n, B, old_hi, new_hi, seed):
    r = random.Random(seed)
    old = [r.choice((0, r.randint(0, old_hi), B * r.randint(0, old_hi // B))) for _ in range(n)]
    new = [a + r.choice((0, 1, r.randint(0, new_hi))) for a in old]
    mbps = max([-(-b // B) for b in new] + [1]) + r.randrange(3)
    nb = sum(-(-b // B) for b in new) + 9
    ids = list(range(nb))
    r.shuffle(ids)
    tables, at = [], 0
    for a in old:
        k = -(-a // B)
        tables.append(ids[at:at + k] + [-5] * (mbps - k))
        at += k
    return old, new, tables, ids[at:], mbps, nb


class Run:
    def __init__(self, old, new, tables, free, mbps, nb, B, cap, head=0):
        self.pool = pool_of(len(old), mbps, nb, B)
        self.old, self.new, self.free, self.head = i32(old), i32(new), i32(free), i32([head])
        self.tables = i32(tables).view(len(old), mbps)
        self.cu = torch.full((len(old) + 1,), -9, dtype=torch.int32, device="cuda")
        self.slots = torch.full((cap,), -9, dtype=torch.int32, device="cuda")
        self.head_out = self.head

    def call(self, **kw):
        pa.pa_build_tables(self.pool, self.old, self.new, self.free, self.head, self.head_out, self.tables,
                           self.cu, self.slots, **kw)

    def check(self, want):
        tables, cu, slots, head = want
        assert self.cu.tolist() == cu
        assert self.slots.tolist() == slots
        assert self.tables.tolist() == tables
        assert self.head_out.tolist() == [head]


@pytest.mark.parametrize("n,old_hi,new_hi", [(0, 1, 1), (1, 0, 1), (1, 100, 5000), (3, 40, 17), (64, 4000, 1),
                                             (513, 63, 300), (700, 0, 33), (8192, 30, 20)])
@pytest.mark.parametrize("B", [16, 32])
@pytest.mark.parametrize("pad", [0, 37])
def test_tables_slots_and_head(n, old_hi, new_hi, B, pad):
    old, new, tables, free, mbps, nb = case(n, B, old_hi, new_hi, n * 7 + B + pad)
    cap = sum(new) - sum(old) + pad
    head = 3
    want = tables_reference(old, new, free, head, tables, B, cap)
    r = Run(old, new, tables, free, mbps, nb, B, cap, head)
    r.head_out = i32([-1])
    r.call()
    r.check(want)
    assert r.head.tolist() == [head]
    # the same inputs again (fresh entries are rewritten alike), the head in place
    r.head_out = r.head
    r.call()
    r.check(want)
    assert pa.pa_check_device_errors(r.pool) == 0


def test_steps_chain_through_the_head():
    """Three steps, each from the lengths the one before reached, head in place."""
    B, n, r = 16, 40, random.Random(5)
    lens = [[0] * n]
    for hi in (200, 1, 33):
        lens.append([a + r.randint(0, hi) for a in lens[-1]])
    mbps, nb = 20, n * 20
    free = list(range(nb))
    r.shuffle(free)
    run = Run(lens[0], lens[1], [[-1] * mbps] * n, free, mbps, nb, B, 200 * n)
    tables, head = [[-1] * mbps] * n, 0
    for a, b in zip(lens, lens[1:]):
        run.old.copy_(i32(a))
        run.new.copy_(i32(b))
        run.call()
        want = tables_reference(a, b, free, head, tables, B, 200 * n)
        run.check(want)
        tables, head = want[0], want[3]
    assert pa.pa_check_device_errors(run.pool) == 0


def test_slots_at_odd_addresses_and_neighbours_untouched():
    old, new, tables, free, mbps, nb = case(30, 16, 50, 90, 3)
    total = sum(new) - sum(old)
    r = Run(old, new, tables, free, mbps, nb, 16, total)
    whole = torch.full((total + 9,), -9, dtype=torch.int32, device="cuda")
    r.slots = whole[3:3 + total]
    r.call()
    r.check(tables_reference(old, new, free, 0, tables, 16, total))
    assert (whole[:3] == -9).all() and (whole[3 + total:] == -9).all()


def test_nothing_is_taken_when_ids_or_slots_run_out():
    old, new, tables, free, mbps, nb = case(9, 16, 50, 400, 11)
    need = sum(-(-b // 16) - -(-a // 16) for a, b in zip(old, new))
    total = sum(new) - sum(old)
    for bits, cap, ids, head in ((pa.PA_DEVERR_NO_BLOCKS, total, free[:need - 1], 0),
                                 (pa.PA_DEVERR_NO_BLOCKS, total, free[:need], 1),
                                 (pa.PA_DEVERR_NO_BLOCKS, total, free, -1),
                                 (pa.PA_DEVERR_NO_BLOCKS, total, free[:need], need + 1),
                                 (pa.PA_DEVERR_BAD_LEN, total - 1, free, 0)):
        r = Run(old, new, tables, ids, mbps, nb, 16, cap, head)
        r.call()
        r.check((tables, [0] * 10, [-1] * cap, head))
        assert pa.pa_check_device_errors(r.pool) == bits
    # exactly enough is enough, and the pool is usable after an error
    r = Run(old, new, tables, free[:need], mbps, nb, 16, total)
    r.call()
    r.check(tables_reference(old, new, free, 0, tables, 16, total))
    assert pa.pa_check_device_errors(r.pool) == 0


def test_a_bad_length_leaves_its_request_alone():
    B, mbps = 16, 8
    old, new = [5, 20, 0, -3, 7], [40, 19, 8 * B + 1, 4, 2 ** 31 - 1]
    tables = [[i * 8 + k for k in range(mbps)] for i in range(5)]
    free = list(range(40, 60))
    r = Run(old, new, tables, free, mbps, 64, B, 50)
    r.call()
    keep = [0, 0, 0, 0]
    want = tables_reference([5] + keep, [40] + keep, free, 0, tables, B, 50)
    r.check(want)
    assert pa.pa_check_device_errors(r.pool) == pa.PA_DEVERR_BAD_LEN


def test_a_bad_id_gives_no_slot():
    r = Run([0, 4], [40, 18], [[-1] * 4, [2, -1, -1, -1]], [7, 99, 5, -4, 1], 4, 10, 16, 54)
    r.call()
    tables, cu, slots, head = tables_reference([0, 4], [40, 18], [7, 99, 5, -4, 1], 0, [[-1] * 4, [2, -1, -1, -1]],
                                               16, 54)
    slots = [-1 if s < 0 or s >= 160 else s for s in slots]
    r.check((tables, cu, slots, head))
    assert pa.pa_check_device_errors(r.pool) == pa.PA_DEVERR_BAD_BLOCK


def test_captured_and_replayed_with_other_lengths():
    old, new, tables, free, mbps, nb = case(50, 16, 60, 0, 21)
    cap = 50 * 40
    mbps, nb = mbps + 4, nb + 400
    tables = [t + [-5] * (mbps - len(t)) for t in tables]
    free = free + list(range(nb - 400, nb))
    r = Run(old, old, tables, free, mbps, nb, 16, cap)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        r.call()
    s.synchronize()
    r.check(tables_reference(old, old, free, 0, tables, 16, cap))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        r.call()
    head, rnd = 0, random.Random(1)
    for _ in range(3):
        new = [a + rnd.randint(0, 30) for a in old]
        new = [min(b, mbps * 16) for b in new]
        r.old.copy_(i32(old))
        r.new.copy_(i32(new))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = tables_reference(old, new, free, head, tables, 16, cap)
        r.check(want)
        tables, old, head = want[0], new, want[3]
    assert pa.pa_check_device_errors(r.pool) == 0


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("kv,act", [("bf16", "bf16"), ("fp16", "fp16"), ("fp8_e4m3", "bf16"), ("fp8_e4m3", "fp16")])
@pytest.mark.parametrize("B", [16, 32])
@pytest.mark.parametrize("T,H", [(1, 1), (7, 3), (64, 8), (301, 2)])
def test_append_by_slots_stores_what_append_stores(kv, act, B, T, H):
    layers, nb = 2, T // B + 3
    g = torch.Generator(device="cuda").manual_seed(T * H)
    kw = {}
    if kv == "fp8_e4m3":
        sc = [torch.rand((layers, H), generator=g, device="cuda") * 0.02 + 0.004 for _ in range(2)]
        kw = dict(k_scale=sc[0], v_scale=sc[1], k_inv_scale=1 / sc[0], v_inv_scale=1 / sc[1])
    pools = [pool_of(1, nb, nb, B, layers=layers, H=H, kv_dtype=kv, act_dtype=act,
                     free_order=np.random.default_rng(T).permutation(nb), **kw) for _ in range(2)]
    k, v = [(torch.randn((T, H, 128), generator=g, device="cuda") * 2).to(DT[act]) for _ in range(2)]
    pa.pa_alloc_blocks(pools[0], 0, T)
    pa.pa_append_kv(pools[0], 1, [0] * T, list(range(T)), k, v)
    _, table = pa.pa_get_seq(pools[0], 0)
    order = torch.randperm(T, generator=g, device="cuda")
    slots = i32([table[t // B] * B + t % B for t in range(T)])[order].contiguous()
    pa.pa_append_kv_slots(pools[1], 1, slots, k[order].contiguous(), v[order].contiguous())
    for a, b in ((pools[0].k_cache, pools[1].k_cache), (pools[0].v_cache, pools[1].v_cache)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert pa.pa_check_device_errors(pools[1]) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_append_skips_slots_that_are_none(kv):
    H, nb, B = 2, 4, 16
    one = torch.ones((1, H), device="cuda")
    kw = dict(k_scale=one, v_scale=one, k_inv_scale=one, v_inv_scale=one) if kv == "fp8_e4m3" else {}
    p = pool_of(1, nb, nb, B, H=H, kv_dtype=kv, **kw)
    x = torch.ones((6, H, 128), dtype=torch.bfloat16, device="cuda")
    pa.pa_append_kv_slots(p, 0, i32([-1, 3, -1, -1, 63, -1]), x, x)
    for c in (p.k_cache, p.v_cache):
        hit = (c.view(torch.uint8).view(nb, H, B, -1) != 0).any(-1).permute(0, 2, 1).reshape(nb * B, H)
        assert hit.any(1).nonzero().flatten().tolist() == [3, 63] and hit[[3, 63]].all()
    assert pa.pa_check_device_errors(p) == 0
    before = p.k_cache.clone()
    pa.pa_append_kv_slots(p, 0, i32([64, -2, -1, 2 ** 31 - 1, -2 ** 31, -1]), x * 3, x * 3)
    assert torch.equal(before.view(torch.uint8), p.k_cache.view(torch.uint8))
    assert pa.pa_check_device_errors(p) == pa.PA_DEVERR_BAD_BLOCK
    pa.pa_append_kv_slots(p, 0, i32([]), x[:0], x[:0])
    assert pa.pa_check_device_errors(p) == 0


def test_append_past_32_bits():
    """Element offsets beyond 2^31 (an FP8 cache of 2^25 rows)."""
    H, B, nb = 8, 16, 1 << 18
    one = torch.ones((1, H), device="cuda")
    p = pool_of(1, 8, nb, B, H=H, kv_dtype="fp8_e4m3", k_scale=one, v_scale=one, k_inv_scale=one, v_inv_scale=one)
    x = torch.full((2, H, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    pa.pa_append_kv_slots(p, 0, i32([nb * B - 1, nb * B // 2 + 5]), x, -x)
    assert pa.pa_check_device_errors(p) == 0
    for c, val in ((p.k_cache, 2.0), (p.v_cache, -2.0)):
        f = c.view(torch.float8_e4m3fn)
        assert (f[0, nb - 1, :, B - 1].float() == val).all() and (f[0, nb // 2, :, 5].float() == val).all()
        assert int((c[0, -1] != 0).sum()) == H * 128 and int((c[0, nb // 2] != 0).sum()) == H * 128
