"""Cases of the prompt-side and drafted-token operators over the paged cache.

Four operators, one after the other what a serving step does with them:

* ``tables``   block tables and the slot map of the new tokens, built on the GPU from request lengths;
* ``append``   K/V rows written into the cache through a slot map (FP8 caches quantise);
* ``prefill``  causal attention of whole prompts, or chunks of them, over the paged cache;
* ``tree``     attention of a tree of drafted tokens over the paged cache.

``own`` selects who computes: elementary torch operations in 32 bits, or the library's entry points.
"""
import math
import random

import torch

own = False

D = 128                      # head_dim of every pool
SCALE = 1.0 / math.sqrt(D)
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------------------------- cases
def _attn(op, name, hq, hkv, act, kv, block, n, past, new, lens=0):
    c = {"op": op, "hq": hq, "hkv": hkv, "act": act, "kv": kv, "block": block, "n": n,
         "past_lo": past[0], "past_hi": past[1], "new_lo": new[0], "new_hi": new[1], "lens": lens}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a decode step of 64 sequences, lengths kept on the device: the smallest call, latency only
        {"name": "tables decode step", "op": "tables", "n": 64, "block": 16, "mbps": 260, "old_lo": 128,
         "old_hi": 4095, "new_lo": 1, "new_hi": 1, "pad": 0, "lens": 1},
        # admission of a large batch of prompts, the slot map padded to a fixed capacity
        {"name": "tables prompts", "op": "tables", "n": 509, "block": 16, "mbps": 260, "old_lo": 0,
         "old_hi": 63, "new_lo": 1, "new_hi": 4033, "pad": 1000, "lens": 2},
        # one decode step's rows of the 8B-class layer
        {"name": "append decode step", "op": "append", "hkv": 8, "act": "bf16", "kv": "bf16", "block": 16, "T": 64},
        # the prompts of one prefill step into an FP8 cache
        {"name": "append prompts fp8", "op": "append", "hkv": 8, "act": "bf16", "kv": "fp8", "block": 16, "T": 32749},
        # the smallest pool's four prompts: few tiles, latency
        dict(_attn("prefill", "prefill tiny", 8, 2, "bf16", "bf16", 16, 4, (0, 0), (16, 825)), new="825,200,103,16"),
        # a ragged batch of prompts, 8B-class layer
        _attn("prefill", "prefill ragged", 32, 8, "bf16", "bf16", 16, 16, (0, 0), (128, 4096), 3),
        # chunks of prompts behind a cached prefix in a long FP8 cache
        _attn("prefill", "prefill chunks fp8", 64, 8, "bf16", "fp8", 16, 8, (2000, 16000), (100, 700), 4),
        # two long prompts, 70B-class layer: the largest call
        dict(_attn("prefill", "prefill long", 64, 8, "bf16", "bf16", 16, 2, (0, 0), (7003, 9001)), new="9001,7003"),
        # one sequence of the worked example with eight drafted tokens
        _attn("tree", "tree one", 8, 2, "bf16", "bf16", 16, 1, (825, 825), (8, 8), 5),
        # 47 sequences of the 70B-class layer with small trees
        _attn("tree", "tree batch", 64, 8, "bf16", "bf16", 16, 47, (809, 841), (5, 16), 6),
        # long FP8 caches, one per sequence, larger trees
        _attn("tree", "tree long fp8", 64, 8, "bf16", "fp8", 16, 8, (30000, 32768), (20, 33), 7),
        # every query head with its own KV head, fp16, blocks of 32 tokens, the widest trees
        _attn("tree", "tree mha fp16", 32, 32, "fp16", "fp16", 32, 17, (1900, 2050), (40, 64), 8),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = {"prefill": 2.1e12, "tree": 2.3e9}
    while True:
        op = rng.choice(("tables", "append", "prefill", "tree"))
        block = rng.choice((16, 32))
        if op == "tables":
            n = _logint(rng, 1, 509)
            old, new = _logint(rng, 1, 4000), _logint(rng, 1, 4033)
            return {"op": op, "n": n, "block": block, "mbps": -(-(old + new) // block) + rng.randrange(4),
                    "old_lo": 0, "old_hi": old, "new_lo": rng.choice((0, 1)), "new_hi": new,
                    "pad": rng.choice((0, rng.randrange(300))), "lens": rng.randrange(1 << 20)}
        act = rng.choice(("bf16", "fp16"))
        kv = rng.choice((act, act, "fp8"))
        if op == "append":
            return {"op": op, "hkv": rng.choice((1, 2, 4, 8, 16)), "act": act, "kv": kv, "block": block,
                    "T": _logint(rng, 1, 16001)}
        g = rng.choice((1, 2, 4, 8))
        hkv = rng.choice((1, 2, 4, 8, 32 // g))
        n = _logint(rng, 1, 47)
        if op == "tree":
            m = _logint(rng, 1, 64)
            past = _logint(rng, 1, 32768)
            c = _attn(op, None, g * hkv, hkv, act, kv, block, n, (past // rng.choice((1, 2, 5)), past),
                      (max(1, m // 2), m), rng.randrange(1 << 20))
        else:
            m = _logint(rng, 1, 9001)
            past = rng.choice((0, 0, _logint(rng, 1, 16000)))
            c = _attn(op, None, g * hkv, hkv, act, kv, block, n, (past // 2, past),
                      (max(1, m // rng.choice((1, 3, 20))), m), rng.randrange(1 << 20))
        w = work(c)
        if (op == "tree" and w["bytes"] < top[op]) or (op == "prefill" and w["flops"] < top[op]):
            return c


def _span(case, lo, hi, salt):
    """The lengths of a case: they belong to it and not to the seed."""
    r = random.Random(case.get("lens", 0) * 7 + salt)
    return [r.randint(case[lo], case[hi]) for _ in range(case["n"])]


def _lens(case):
    """(cached tokens, new tokens) of each sequence."""
    if case["op"] == "tables":
        return _span(case, "old_lo", "old_hi", 1), _span(case, "new_lo", "new_hi", 2)
    if "new" in case:
        new = [int(x) for x in case["new"].split(",")]
        return [0] * len(new), new
    return _span(case, "past_lo", "past_hi", 1), _span(case, "new_lo", "new_hi", 2)


def _pairs(case):
    """(query, key) pairs that one query head works on; a drafted token counts its whole tree."""
    past, new = _lens(case)
    if case["op"] == "tree":
        return sum(m * (p + m) for p, m in zip(past, new))
    return sum(m * p + m * (m + 1) // 2 for p, m in zip(past, new))


def _kv_bytes(case):
    return 1 if case["kv"] == "fp8" else 2


def work(case):
    op = case["op"]
    if op == "tables":
        past, new = _lens(case)
        B = case["block"]
        need = sum(-(-(p + m) // B) - -(-p // B) for p, m in zip(past, new))
        tails = sum(1 for p, m in zip(past, new) if p % B and m)
        return {"bytes": 4 * (2 * case["n"] + 2 * need + tails + case["n"] + 1 + sum(new) + case["pad"] + 2), "flops": 0}
    if op == "append":
        row = 2 * case["hkv"] * D
        return {"bytes": case["T"] * (4 + row * (2 + _kv_bytes(case))), "flops": 0}
    past, new = _lens(case)
    cached = sum(past) + sum(new)
    rows = sum(new) * case["hq"] * D * 2 * 2
    extra = 8 * sum(new) if op == "tree" else 0
    return {"bytes": rows + 2 * cached * case["hkv"] * D * _kv_bytes(case) + 4 * (cached // case["block"]) + extra,
            "flops": 4 * D * case["hq"] * _pairs(case)}


# --------------------------------------------------------------------------------------------- inputs
def _rand(g, shape, dtype, mul=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * mul).to(dtype)


def _cache(case, g, num_blocks):
    """A filled cache [1][blocks][H][B][D], its scales (FP8) and a pool over it for the library's calls."""
    shape = (1, num_blocks, case["hkv"], case["block"], D)
    s = {}
    if case["kv"] == "fp8":
        s["scale"] = [torch.rand((1, case["hkv"]), generator=g, device="cuda") * 0.004 + 0.008 for _ in range(2)]
        s["inv"] = [1.0 / x for x in s["scale"]]
        cache = [(_rand(g, shape, torch.float32) / x.view(1, 1, -1, 1, 1)).clamp_(-448, 448).to(torch.float8_e4m3fn)
                 for x in s["scale"]]
    else:
        cache = [_rand(g, shape, DT[case["act"]]) for _ in range(2)]
    s["k"], s["v"] = cache
    return s


def _pool(case, s, num_blocks, seqs, mbps):
    import pagedattention_decode_03_b200 as pa
    fp8 = case["kv"] == "fp8"
    kw = {}
    if fp8:
        kw = {"k_scale": s["scale"][0], "v_scale": s["scale"][1], "k_inv_scale": s["inv"][0], "v_inv_scale": s["inv"][1]}
    k, v = (s["k"].view(torch.uint8), s["v"].view(torch.uint8)) if fp8 else (s["k"], s["v"])
    return pa.pa_pool_create(num_layers=1, num_kv_heads=case["hkv"], block_size=case["block"], num_blocks=num_blocks,
                             max_seqs=seqs, max_blocks_per_seq=mbps, kv_dtype="fp8_e4m3" if fp8 else case["act"],
                             act_dtype=case["act"], k_cache=k, v_cache=v, **kw)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B = case["op"], case["block"]
    s = {"case": case}
    if op == "append":
        T = case["T"]
        nb = -(-T // B) * 5 // 4 + 2
        s.update(_cache(case, g, nb))
        s["slots"] = torch.randperm(nb * B, generator=g, device="cuda")[:T].to(torch.int32)
        s["new"] = [_rand(g, (T, case["hkv"], D), DT[case["act"]], 1.5) for _ in range(2)]
        if own:
            s["pool"] = _pool(case, s, nb, 1, nb)
        return s
    past, new = _lens(case)
    n = len(new)
    have, want = [-(-p // B) for p in past], [-(-(p + m) // B) for p, m in zip(past, new)]
    if op == "tables":
        mbps, total = case["mbps"], sum(want)
        nb = total * 5 // 4 + 8
        ids = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        s["tables"] = torch.full((n, mbps), -1, dtype=torch.int32, device="cuda")
        held = torch.arange(mbps, device="cuda")[None, :] < torch.tensor(have, device="cuda")[:, None]
        s["tables"][held] = ids[:sum(have)]
        s["free"] = ids[sum(have):].contiguous()
        s["head"] = torch.randint(0, 8, (1,), generator=g, device="cuda", dtype=torch.int32)
        s["head_out"] = torch.zeros_like(s["head"])
        s["old"] = torch.tensor(past, dtype=torch.int32, device="cuda")
        s["lens"] = torch.tensor([p + m for p, m in zip(past, new)], dtype=torch.int32, device="cuda")
        s["cu"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
        s["slots"] = torch.zeros(sum(new) + case["pad"], dtype=torch.int32, device="cuda")
        if own:
            import pagedattention_decode_03_b200 as pa
            s["pool"] = pa.pa_pool_create(num_layers=1, num_kv_heads=1, block_size=B, num_blocks=nb, max_seqs=n,
                                          max_blocks_per_seq=mbps, kv_dtype="bf16")
        return s
    mbps = max(want)
    nb = sum(want) * 5 // 4 + 1
    s.update(_cache(case, g, nb))
    ids = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    s["tables"] = torch.zeros((n, mbps), dtype=torch.int32, device="cuda")
    held = torch.arange(mbps, device="cuda")[None, :] < torch.tensor(want, device="cuda")[:, None]
    s["tables"][held] = ids[:sum(want)]
    s["q"] = _rand(g, (sum(new), case["hq"], D), DT[case["act"]], 2.0)
    s["out"] = torch.empty_like(s["q"])
    s["new"], s["kv_lens"] = new, [p + m for p, m in zip(past, new)]
    if op == "tree":
        # parents: token i hangs under an earlier token or under the prefix; a token sees itself and its ancestors
        m = max(new)
        seen = torch.zeros((n, m), dtype=torch.int64, device="cuda")
        for i in range(m):
            up = (torch.rand(n, generator=g, device="cuda") * (i + 1)).long().clamp_(max=i) - 1
            above = torch.where(up >= 0, seen.gather(1, up.clamp(min=0)[:, None])[:, 0], 0)
            seen[:, i] = above | (torch.ones_like(above) << i)
        count = torch.tensor(new, device="cuda")
        inside = torch.arange(m, device="cuda")[None, :] < count[:, None]
        s["mask"] = seen[inside].contiguous()
        s["count"], s["past"] = count, torch.tensor(past, device="cuda")
    if own:
        s["pool"] = _pool(case, s, nb, n, mbps)
    return s


# ------------------------------------------------------------------------------------------ plain forms
def _tables_plain(s):
    B, tables = s["case"]["block"], s["tables"]
    old, new = s["old"].long(), s["lens"].long()
    have, want = (old + B - 1) // B, (new + B - 1) // B
    need = want - have
    take = need.cumsum(0) - need
    at = torch.arange(tables.shape[1], device=tables.device)[None, :]
    fresh = (at >= have[:, None]) & (at < want[:, None])
    pick = (s["head"].long() + take[:, None] + at - have[:, None]).clamp(0, s["free"].numel() - 1)
    tables.copy_(torch.where(fresh, s["free"][pick], tables))
    cu = torch.zeros_like(s["cu"], dtype=torch.int64)
    cu[1:] = (new - old).cumsum(0)
    t = torch.arange(s["slots"].numel(), device=tables.device)
    i = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=old.numel() - 1)
    pos = (old[i] + t - cu[i]).clamp(max=tables.shape[1] * B - 1)
    slot = tables[i, pos // B].long() * B + pos % B
    s["slots"].copy_(torch.where(t < cu[-1], slot, -1))
    s["cu"].copy_(cu)
    s["head_out"].copy_(s["head"] + need.sum())
    return tables, s["cu"], s["slots"], s["head_out"]


def _append_plain(s):
    B = s["case"]["block"]
    slots = s["slots"].long()
    for c, x, k in zip((s["k"], s["v"]), s["new"], range(2)):
        if s["case"]["kv"] == "fp8":
            x = (x.float() * s["inv"][k][0][None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            c = c.view(torch.uint8)
        c[0][slots // B, :, slots % B] = x
    return s["k"], s["v"]


def _softmax_av(x, v):
    """exp(x - max) v / sum over the last axis; rows with nothing left give zero."""
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total == 0, torch.ones_like(total), total)


def _rows(s, name, blocks):
    """Cache rows of the given blocks in 32 bits: [..., H, tokens, D]."""
    x = s[name][0][blocks].float()                   # [..., nb, H, B, D]
    x = x.transpose(-4, -3).flatten(-3, -2)          # [..., H, nb * B, D]
    if "scale" in s:
        x = x * s["scale"][0 if name == "k" else 1][0][:, None, None]
    return x


def _prefill_plain(s):
    case, out = s["case"], s["out"]
    H, G, B, base = case["hkv"], case["hq"] // case["hkv"], case["block"], 0
    for i, (m, L) in enumerate(zip(s["new"], s["kv_lens"])):   # sequences differ in both lengths
        blocks = s["tables"][i, :-(-L // B)].long()
        k, v = _rows(s, "k", blocks)[:, :L], _rows(s, "v", blocks)[:, :L]
        step = max(1, (1 << 28) // (case["hq"] * L))
        for a in range(0, m, step):                            # a block of query rows at a time: the scores are large
            b = min(m, a + step)
            q = s["q"][base + a:base + b].float().view(b - a, H, G, D).permute(1, 2, 0, 3)
            x = (q @ k.transpose(-1, -2)[:, None]) * SCALE
            pos = torch.arange(L - m + a, L - m + b, device=x.device)
            x = x.masked_fill(torch.arange(L, device=x.device)[None, :] > pos[:, None], -math.inf)
            o = _softmax_av(x, v[:, None])
            out[base + a:base + b] = o.permute(2, 0, 1, 3).reshape(b - a, H * G, D).to(out.dtype)
        base += m
    return out


def _tree_plain(s):
    case = s["case"]
    H, G, n, m, L = case["hkv"], case["hq"] // case["hkv"], len(s["new"]), max(s["new"]), max(s["kv_lens"])
    dev = s["q"].device
    inside = torch.arange(m, device=dev)[None, :] < s["count"][:, None]
    start = (s["count"].cumsum(0) - s["count"])[:, None] + torch.arange(m, device=dev)[None, :]
    start = start.clamp(max=s["q"].shape[0] - 1)
    q = s["q"][start].float().view(n, m, H, G, D).permute(0, 2, 3, 1, 4).reshape(n, H, G * m, D)
    k, v = _rows(s, "k", s["tables"].long())[:, :, :L], _rows(s, "v", s["tables"].long())[:, :, :L]
    x = (q @ k.transpose(-1, -2)) * SCALE
    at = torch.arange(L, device=dev)[None, None, :] - s["past"][:, None, None]
    bit = (s["mask"][start][:, :, None] >> at.clamp(0, 63)) & 1
    ok = (at < 0) | ((at < s["count"][:, None, None]) & (bit == 1))                  # [n, m, L]
    x = x.view(n, H, G, m, L).masked_fill(~ok[:, None, None], -math.inf).view(n, H, G * m, L)
    o = _softmax_av(x, v).view(n, H, G, m, D).permute(0, 3, 1, 2, 4).reshape(n, m, H * G, D)
    rows = torch.where(inside, start, s["q"].shape[0]).flatten()
    whole = torch.empty((s["q"].shape[0] + 1, H * G, D), dtype=s["out"].dtype, device=dev)
    whole[rows] = o.flatten(0, 1).to(whole.dtype)
    s["out"].copy_(whole[:-1])
    return s["out"]


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"tables": _tables_plain, "append": _append_plain, "prefill": _prefill_plain, "tree": _tree_plain}[op](s)
    import pagedattention_decode_03_b200 as pa
    if op == "tables":
        pa.pa_build_tables(s["pool"], s["old"], s["lens"], s["free"], s["head"], s["head_out"], s["tables"], s["cu"],
                           s["slots"])
        return s["tables"], s["cu"], s["slots"], s["head_out"]
    if op == "append":
        pa.pa_append_kv_slots(s["pool"], 0, s["slots"], s["new"][0], s["new"][1])
        return s["k"], s["v"]
    if op == "prefill":
        pa.pa_prefill_attention(s["pool"], 0, s["new"], s["q"], s["out"], SCALE, kv_lens=s["kv_lens"],
                                block_tables=s["tables"])
    else:
        pa.pa_tree_attention(s["pool"], 0, s["new"], s["mask"], s["q"], s["out"], SCALE, kv_lens=s["kv_lens"],
                             block_tables=s["tables"])
    return s["out"]


# ------------------------------------------------------------------------------------- values in 64 bits
def exact(case, seed):
    """The operators' definitions, sequence by sequence and head by head, in 64 bits."""
    s = prepare(case, seed)
    B, op = case["block"], case["op"]
    if op == "tables":
        return None                                      # whole numbers only
    if op == "append":
        got = []
        for k, name in enumerate(("k", "v")):
            c = s[name][0].double()
            x = s["new"][k].double()
            if case["kv"] == "fp8":
                x = (x * s["inv"][k][0].double().view(1, -1, 1)).clamp(-448.0, 448.0)
            where = s["slots"].long()
            flat = c.permute(0, 2, 1, 3).reshape(-1, case["hkv"], D)      # one row a slot
            flat[where] = x
            got.append(flat.view(-1, B, case["hkv"], D).permute(0, 2, 1, 3)[None].contiguous())
        return tuple(got)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    G, base = case["hq"] // case["hkv"], 0
    masks = s["mask"].tolist() if op == "tree" else None
    for i, (m, L) in enumerate(zip(s["new"], s["kv_lens"])):
        slot = torch.arange(L, device="cuda")
        blk = s["tables"][i].long()[slot // B]
        allowed = None
        if op == "tree":
            rows = [[True] * (L - m) + [bool(masks[base + r] >> j & 1) for j in range(m)] for r in range(m)]
            allowed = torch.tensor(rows, device="cuda")
        for h in range(case["hkv"]):
            k, v = s["k"][0][blk, h, slot % B].double(), s["v"][0][blk, h, slot % B].double()
            if case["kv"] == "fp8":
                k, v = k * s["scale"][0][0, h].double(), v * s["scale"][1][0, h].double()
            for a in range(0, m, 1024):
                b = min(m, a + 1024)
                end = L - m + b if op == "prefill" else L
                q = s["q"][base + a:base + b, h * G:(h + 1) * G].double()
                x = torch.einsum("tgd,pd->gtp", q, k[:end]) / math.sqrt(D)
                if op == "prefill":
                    seen = slot[:end].view(1, -1) <= (L - m + torch.arange(a, b, device="cuda")).view(-1, 1)
                else:
                    seen = allowed[a:b]
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                w = torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
                out[base + a:base + b, h * G:(h + 1) * G] = torch.einsum("gtp,pd->tgd", w, v[:end])
        base += m
    return out
