"""The serving operators at the largest batch (65535 sequences) and head count
(4096) that they accept, against the definition in 64 bits on the GPU.

Tolerances as in paged_cases, with the weights' own rounding: bf16 outputs
2^-8 of the value; A = sum w |v| / sum w times 2^-9 for fp32 and, packed prompts
and e4m3 caches, 2^-8 and 2^-11 for the weights; lse 2^-10."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _zq():
    import bf16_causal_prefill_02_b200 as zq

    return zq


def _rnd(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def _attend(q, k, v, seen, scale):
    """q (..., R, d), k and v (..., S, .), seen (..., R, S): out, lse, A in 64 bits; rows that see nothing get 0 and -inf."""
    x = (q.double() @ k.double().transpose(-1, -2)) * scale
    x = x.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, dim=-1)
    w = torch.exp(x - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[..., None])
    return w @ v.double(), lse, w @ v.double().abs()


def _check(out, lse, want, p_step):
    ro, rl, mass = want
    assert torch.isfinite(out).all() and torch.equal(lse.isinf(), rl.isinf())
    assert ((out.double() - ro).abs() <= 2.0 ** -8 * ro.abs() + (p_step + 2.0 ** -9) * mass).all()
    fin = ~rl.isinf()
    assert ((lse.double() - rl)[fin].abs() <= 2.0 ** -10 + 2.0 ** -22 * rl[fin].abs()).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("room", [32, 2048])
def test_decode_of_65535_sequences(dtype, room):
    B, page, hq = 65535, 16, 2
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(-1, 21, (B,), generator=g).to(torch.int32)
    table = torch.full((B, room // page), -1, dtype=torch.int32)
    pages = 4 * B // 3  # (some pages serve two sequences)
    table[:, :2] = torch.randint(0, pages, (B, 2), generator=g)
    t = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
    k, v, q = _rnd(pages, page, 1, 128, seed=2, dtype=t), _rnd(pages, page, 1, 128, seed=3, dtype=t), _rnd(B, hq, 128, seed=4)
    table, lens = table.cuda(), lens.cuda()
    out, lse = _zq().attn_decode(q, k, v, table, lens)
    for b0 in range(0, B, 8192):
        b = slice(b0, b0 + 8192)
        at = table[b, :2].long()
        kk, vv = (x.view(torch.uint8)[at].view(t).flatten(1, 2)[:, :, 0] for x in (k, v))
        seen = torch.arange(32, device="cuda")[None, None, :] < lens[b, None, None]
        _check(out[b], lse[b], _attend(q[b], kk, vv, seen.expand(-1, hq, -1), 128 ** -0.5), 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hkv,lens,room", [(1, [40, 3], 64), (1, [40, 700], 65536), (4096, [40, 3], 64), (4096, [33, 0, 100], 65536)])
def test_append_and_decode_of_4096_heads(dtype, hkv, lens, room):
    zq = _zq()
    hq, page, B = 4096, 16, len(lens)
    n = [-(-(x + 1) // page) for x in lens]
    t = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
    table = torch.full((B, room // page), -1, dtype=torch.int32)
    for b in range(B):
        table[b, :n[b]] = torch.arange(sum(n[:b]), sum(n[:b + 1]))
    table = table.cuda()
    k, v, q = _rnd(sum(n), page, hkv, 128, seed=5, dtype=t), _rnd(sum(n), page, hkv, 128, seed=6, dtype=t), _rnd(B, hq, 128, seed=7)
    kn, vn = _rnd(B, hkv, 128, seed=8), _rnd(B, hkv, 128, seed=9)
    have = torch.tensor(lens, dtype=torch.int32, device="cuda")
    zq.kv_append(kn, vn, k, v, table, have)
    out, lse = zq.attn_decode(q, k, v, table, have + 1)
    for b in range(B):
        kk, vv = (x[sum(n[:b]):sum(n[:b + 1])].flatten(0, 1)[:lens[b] + 1].transpose(0, 1) for x in (k, v))  # (hkv, keys, 128)
        assert torch.equal(kk[:, -1].float(), kn[b].to(t).float()) and torch.equal(vv[:, -1].float(), vn[b].to(t).float())
        qq = q[b].view(hkv, hq // hkv, 128)
        want = _attend(qq, kk, vv, torch.ones((1, 1, 1), dtype=torch.bool, device="cuda"), 128 ** -0.5)
        _check(out[b].view(hkv, -1, 128), lse[b].view(hkv, -1), want, 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11)


def test_packed_prompts_of_65535_sequences():
    B, hq, hkv = 65535, 2, 1
    g = torch.Generator().manual_seed(10)
    lq, lk = torch.randint(0, 4, (B,), generator=g), torch.randint(0, 5, (B,), generator=g)
    cq, ck = (torch.cat([torch.zeros(1, dtype=torch.int64), x.cumsum(0)]).cuda() for x in (lq, lk))
    q, k, v = _rnd(int(cq[-1]), hq, 128, seed=11), _rnd(int(ck[-1]), hkv, 128, seed=12), _rnd(int(ck[-1]), hkv, 128, seed=13)
    out, lse = _zq().attn_varlen(q, k, v, cq.to(torch.int32), ck.to(torch.int32))
    lq, lk, own = lq.cuda(), lk.cuda(), torch.repeat_interleave(torch.arange(B, device="cuda"), lq.cuda())
    i = torch.arange(q.shape[0], device="cuda") - cq[own]
    j = torch.arange(4, device="cuda")
    seen = j[None, :] <= torch.minimum(i + lk[own] - lq[own], lk[own] - 1)[:, None]
    at = (ck[own][:, None] + j).clamp(max=k.shape[0] - 1)
    want = _attend(q, k[at, 0], v[at, 0], seen[:, None, :].expand(-1, hq, -1), 128 ** -0.5)
    _check(out, lse.t(), want, 2.0 ** -8)


@pytest.mark.parametrize("hkv", [1, 4096])
def test_packed_prompts_of_4096_heads(hkv):
    hq, lens = 4096, [130, 1, 20]
    cu = torch.tensor([0, 130, 131, 151], dtype=torch.int32, device="cuda")
    q, k, v = _rnd(151, hq, 128, seed=14), _rnd(151, hkv, 128, seed=15), _rnd(151, hkv, 128, seed=16)
    out, lse = _zq().attn_varlen(q, k, v, cu, cu)
    at = 0
    for n in lens:
        r = slice(at, at + n)
        seen = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
        for h in range(0, hq, 512):
            hh, kh = slice(h, h + 512), slice(h, h + 512) if hkv == hq else slice(0, 1)
            want = _attend(q[r, hh].transpose(0, 1), k[r, kh].transpose(0, 1), v[r, kh].transpose(0, 1), seen, 128 ** -0.5)
            _check(out[r, hh].transpose(0, 1), lse[hh, r], want, 2.0 ** -8)
        at += n
