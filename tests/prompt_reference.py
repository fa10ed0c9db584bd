"""Plain references of the prompt-side operators, and the bound their results keep.

Attention is computed in 64 bits from the stored cache values.  The bound on an
output element is a sum over what the kernels round, with u = eps / 2 of the
activation type and A = sum p |v| / sum p, the mean of |v| under the weights:

* the weights enter the second product rounded to the activation type: u A
  (plus, for fp16, weights under 2^-14 of the row's reference are subnormal and
  carry an absolute error of 2^-25 each at most: 2^-25 x sum |v| / sum p);
* an FP8 cache's products run on fp16 operands (codes are exact in fp16) with
  weights up to 2^15, 2^12 at the row's reference or more: subnormal weights are
  off by half of 2^-24 there, 2^-37 of the reference, which is not above the
  row's maximum: 2^-37 x sum |v| / sum p with p relative to the maximum;
* the exponential itself is held to a sixteenth of that: u A / 16;
* scores are fp32 sums of 128 products; with the scale they are off by at most
  e = 130 x 2^-24 x scale x max sum |q_d k_d|, which moves every weight, and
  their sum, by a factor 1 +- e: 2 e A;
* weights and products are summed in fp32 over L positions: 2 (L + 8) 2^-24 A;
* the result is rounded to the activation type: u |o|.
"""
import math

import numpy as np
import torch

import pagedattention_decode_03_b200 as pa

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
D = 128


def tables_reference(old, new, free, head, tables, B, cap):
    """(tables, cu, slots, head) after extending `old` to `new`; python integers."""
    tables = [list(r) for r in tables]
    cu, slots = [0], []
    for i, (a, b) in enumerate(zip(old, new)):
        for k in range(-(-a // B), -(-b // B)):
            tables[i][k] = free[head]
            head += 1
        slots += [tables[i][p // B] * B + p % B for p in range(a, b)]
        cu.append(cu[-1] + b - a)
    return tables, cu, slots + [-1] * (cap - len(slots)), head


class Setup:
    """A filled cache with random placement, a pool over it and block tables.

    Slots past each length (and blocks of nobody) hold NaN bytes."""

    def __init__(self, lens, *, H, kv="bf16", act=None, B=16, layers=1, layer=0, seed=0, extra=3, mbps=None,
                 num_blocks=None):
        act = act or ("bf16" if kv == "fp8_e4m3" else kv)
        self.lens, self.H, self.kv, self.act, self.B, self.layer = list(lens), H, kv, act, B, layer
        g = torch.Generator().manual_seed(seed)
        need = [-(-x // B) for x in lens]
        nb = num_blocks or sum(need) + extra
        self.mbps = mbps or max(need + [1]) + 1
        elem = torch.uint8 if kv == "fp8_e4m3" else DT[act]
        kw = {}
        self.scale_k = self.scale_v = None
        if kv == "fp8_e4m3":
            ks, vs = [torch.rand((layers, H), generator=g) * 0.01 + 0.005 for _ in range(2)]
            self.scale_k, self.scale_v = ks[layer].double().cuda(), vs[layer].double().cuda()
            kw = dict(k_scale=ks.cuda(), v_scale=vs.cuda(), k_inv_scale=(1 / ks).cuda(), v_inv_scale=(1 / vs).cuda())
        self.cache = [torch.empty((layers, nb, H, B, D), dtype=elem, device="cuda") for _ in range(2)]
        for c in self.cache:
            c.view(torch.uint8).fill_(0xFF)
        self.pool = pa.pa_pool_create(num_layers=layers, num_kv_heads=H, block_size=B, num_blocks=nb,
                                      max_seqs=max(len(lens), 1), max_blocks_per_seq=self.mbps, kv_dtype=kv,
                                      act_dtype=act, k_cache=self.cache[0], v_cache=self.cache[1], **kw)
        ids = torch.randperm(nb, generator=g).to(torch.int32)
        self.tables = torch.full((len(lens), self.mbps), -7, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.tables[i, :n] = ids[at:at + n]
            at += n
        self.free = ids[at:]
        self.tables = self.tables.cuda()
        g2 = torch.Generator(device="cuda").manual_seed(seed + 1)
        for i, n in enumerate(lens):
            pos = torch.arange(n, device="cuda")
            blk = self.tables[i].long()[pos // B]
            for c in self.cache:
                if kv == "fp8_e4m3":
                    x = torch.randint(0, 0x7F, (n, H, D), generator=g2, device="cuda", dtype=torch.uint8)
                    x |= torch.randint(0, 2, (n, H, D), generator=g2, device="cuda", dtype=torch.uint8) << 7
                else:
                    x = torch.randn((n, H, D), generator=g2, device="cuda").to(elem)
                c[layer][blk, :, pos % B] = x
        self.gen = g2

    def rand(self, rows, heads, mul=1.0):
        return (torch.randn((rows, heads, D), generator=self.gen, device="cuda") * mul).to(DT[self.act])

    def rows(self, which, i, n):
        """The first n cached rows of sequence i in 64 bits: [n, H, D]."""
        pos = torch.arange(n, device="cuda")
        x = self.cache[which][self.layer][self.tables[i].long()[pos // self.B], :, pos % self.B]
        if self.kv == "fp8_e4m3":
            x = x.view(torch.float8_e4m3fn).double()
            return x * (self.scale_k if which == 0 else self.scale_v)[None, :, None]
        return x.double()

    def check(self, q_lens, q, out, scale, mask=None, kv_lens=None, what="attention"):
        """Every output element within the bound of the module's head comment."""
        kv_lens = kv_lens or self.lens
        u = torch.finfo(DT[self.act]).eps / 2
        G, base, worst = q.shape[1] // self.H, 0, 0.0
        for i, (m, L) in enumerate(zip(q_lens, kv_lens)):
            if m == 0:
                continue
            k, v = self.rows(0, i, L), self.rows(1, i, L)
            pos = torch.arange(L, device="cuda")
            for a in range(0, m, 512):
                b = min(m, a + 512)
                t = torch.arange(a, b, device="cuda")[:, None]
                if mask is None:
                    seen = pos[None, :] <= L - m + t
                else:
                    bits = (mask[base + a:base + b, None] >> (pos[None, :] - (L - m)).clamp(0, 63)) & 1
                    seen = (pos[None, :] < L - m) | (bits == 1)
                for h in range(self.H):
                    qq = q[base + a:base + b, h * G:(h + 1) * G].double()
                    x = torch.einsum("tgd,pd->gtp", qq, k[:, h]) * scale
                    e = torch.einsum("tgd,pd->gtp", qq.abs(), k[:, h].abs()).amax(-1) * abs(scale) * 130 * 2.0 ** -24
                    x = x.masked_fill(~seen, -math.inf)
                    top = x.amax(-1, keepdim=True).clamp(min=-1e300)
                    w = torch.exp(x - top)
                    s = w.sum(-1, keepdim=True)
                    one = torch.where(s == 0, torch.ones_like(s), s)
                    ref = (w @ v[:, h]) / one
                    A = (w @ v[:, h].abs()) / one
                    bound = u * (1 + 1 / 16) * A + (2 * e[..., None] + 2 * (L + 8) * 2.0 ** -24) * A + u * ref.abs()
                    if self.act == "fp16":
                        bound = bound + 2.0 ** -25 * (seen.double() @ v[:, h].abs())[None] / one + 2.0 ** -25
                    if self.kv == "fp8_e4m3":
                        bound = bound + 2.0 ** -37 * (seen.double() @ v[:, h].abs())[None] / one
                    got = out[base + a:base + b, h * G:(h + 1) * G].double().permute(1, 0, 2)
                    assert torch.isfinite(got).all(), (what, i, a, h)
                    ratio = (got - ref).abs() / bound.clamp(min=1e-300)
                    ratio = torch.where((got == ref), torch.zeros_like(ratio), ratio)
                    worst = max(worst, float(ratio.max()))
                    assert worst <= 1.0, (what, "sequence", i, "head", h, "rows from", a, "error / bound", worst)
            base += m
        return worst


def random_tree_mask(lens, gen):
    """Ancestors-and-self bits of random trees, packed (int64)."""
    words = []
    for m in lens:
        seen = []
        for i in range(m):
            up = int(torch.randint(-1, i, (1,), generator=gen)) if i else -1
            seen.append((seen[up] if up >= 0 else 0) | 1 << i)
        words += seen
    return torch.from_numpy(np.array(words, np.uint64).view(np.int64)).cuda()
