"""Shared helpers for the paged-cache tests: a cache built on the CPU and the
operators' definitions in 64 bits (no code in common with the library).

Tolerances, element by element, from the roundings the kernel makes:
  * the output is rounded to bf16: at most 2^-8 of the value (half a step);
  * each weight is rounded to bf16 (2^-8 of it) or, over an e4m3 cache, to f16
    (2^-11): the output moves by at most that times A = sum w |v| / sum w;
  * fp32 arithmetic: a score of d <= 192 products with sum |q k| scale <= 32
    is off by at most 192 * 32 * 2^-24 < 2^-11 in the worst case, and a weight
    by as much of itself (times ln 2 in the log2 domain); the sums of up to
    2^13 terms in a warp's share add less than 2^-11 of A (worst case 2^13 *
    2^-24).  Numerator and denominator both: 4 * 2^-11 = 2^-9 of A in all.
  lse: the score error and the sum's, 2^-10, and 2^-22 of the value for its
  own rounding and that of log2.
"""
import math

import torch

OUT_STEP, FP32_SLACK = 2.0 ** -8, 2.0 ** -9
P_STEP = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -11}
LSE_ABS, LSE_REL = 2.0 ** -10, 2.0 ** -22


class Cache:
    """A paged cache with random contents whose pages lie in a random order;
    rows that belong to no key hold `waste`."""

    def __init__(self, lens, hkv, dqk, page, dtype="bf16", seed=0, waste=float("nan"), spare=2, interleaved=False, per_head=True):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.dqk, self.page, self.dtype = list(lens), hkv, dqk, page, dtype
        need = [-(-n // page) for n in self.lens]
        self.pages = sum(need) + spare
        width = max(max(need), 1) + 1
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((len(self.lens), width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cols = {"k": dqk, "v": 128}
        self.descale, self.store = {}, {}
        used = torch.zeros(self.pages, page, dtype=torch.bool)
        for b, n in enumerate(self.lens):
            pos = torch.arange(n)
            used[self.table[b, pos // page].long(), pos % page] = True
        for x in "kv":
            t = torch.randn((self.pages, page, hkv, self.cols[x]), generator=g)
            if dtype == "e4m3":
                ds = 0.01 * torch.exp(torch.randn((hkv if per_head else 1,), generator=g))
                t = (t / ds[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
                self.descale[x] = ds
                if waste is not None:
                    t.view(torch.uint8)[~used] = 0x7F  # e4m3 NaN
            else:
                t = t.to(torch.bfloat16)
                if waste is not None:
                    t[~used] = waste
            self.store[x] = t
        self.interleaved = interleaved

    def cuda(self):
        """The arguments of attn_decode / kv_append after q (or k, v)."""
        k, v = self.store["k"].cuda(), self.store["v"].cuda()
        if self.interleaved:  # keys and values of a page side by side in one allocation
            both = torch.cat([k.flatten(1), v.flatten(1)], dim=1)
            n = k[0].numel()
            k, v = both[:, :n].view(k.shape), both[:, n:].view(v.shape)
        ds = {x + "_descale": self.descale[x].cuda() for x in self.descale}
        return dict(k_cache=k, v_cache=v, block_table=self.table.cuda(),
                    cache_seqlens=torch.tensor(self.lens, dtype=torch.int32).cuda(), **ds)

    def rows(self, x, b, n=None):
        """Keys or values of sequence b in order, 64 bits, and which of them are on a page of the cache."""
        n = self.lens[b] if n is None else n
        pos = torch.arange(n)
        pg = self.table[b, pos // self.page].long()
        ok = (pg >= 0) & (pg < self.pages)
        t = self.store[x][pg.clamp(0, self.pages - 1), pos % self.page].double()
        return (t * self.descale[x].double()[:, None] if self.descale else t), ok


def decode_ref(cache, q, scale=None):
    """(out, lse, A) in 64 bits; q (B, Hq, d)."""
    B, hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros((B, hq, 128), dtype=torch.float64)
    mass = torch.zeros((B, hq, 128), dtype=torch.float64)
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64)
    group = hq // cache.hkv
    for b in range(B):
        k, ok = cache.rows("k", b)
        v, _ = cache.rows("v", b)
        k, v = k[ok], v[ok]
        if k.shape[0] == 0:
            continue
        x = torch.einsum("gjd,ngd->gjn", q[b].double().view(cache.hkv, group, d), k) * scale
        lse[b] = torch.logsumexp(x, dim=-1).flatten()
        w = torch.softmax(x, dim=-1)
        out[b] = torch.einsum("gjn,ngd->gjd", w, v).flatten(0, 1)
        mass[b] = torch.einsum("gjn,ngd->gjd", w, v.abs()).flatten(0, 1)
    return out, lse, mass


def check_decode(cache, q, out, lse, scale=None):
    ro, rl, mass = decode_ref(cache, q, scale)
    o, l = out.double().cpu(), lse.double().cpu()
    assert torch.isfinite(o).all(), "non-finite output"
    assert torch.equal(torch.isinf(l), torch.isinf(rl)), "empty rows differ"
    tol = OUT_STEP * ro.abs() + (P_STEP[cache.dtype] + FP32_SLACK) * mass
    worst = ((o - ro).abs() / tol.clamp(min=1e-30)).max().item() if o.numel() else 0.0
    assert worst <= 1.0, "output off by %.3g of its tolerance" % worst
    fin = ~torch.isinf(rl)
    dl = ((l - rl).abs() / (LSE_ABS + LSE_REL * rl.abs()))[fin]
    assert not fin.any() or dl.max().item() <= 1.0, "lse off by %.3g of its tolerance" % dl.max().item()
    return worst
