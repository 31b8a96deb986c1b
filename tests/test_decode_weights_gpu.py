"""GPU tests of the weights' precision in the paged decode, against closed forms
or the definition in 64 bits."""
import math

import pytest
import torch

from paged_cases import decode_ref

pytestmark = pytest.mark.gpu


def _zq():
    import bf16_causal_prefill_02_b200 as zq

    return zq


OCTAVES = [12.0, 19.3, 23.4, 25.6]  # how far the first key lies above all others, for the heads of a group


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_many_keys_far_below_one(dtype):
    """One key far above 10^5 others that share a warp (148 sequences of 8
    heads over the same pages, so that each warp's share is about one of
    them).  The first key's value is 0, so the output is the others' alone,
    and nothing hides what their small weights lose.

    Tolerance, as in paged_cases: 2^-8 of the value for its rounding and 2^-9 of
    A = sum w |v| / sum w for fp32; a weight's own rounding, bf16 twice (2^-16 of
    it) or f16 (2^-11), and, f16 being subnormal below 2^-14, half of 2^-24
    where the largest weight is 2^11 or more: 2^-36 of the largest weight."""
    zq = _zq()
    n, page, B, hkv, group = 100000, 128, 148, 8, len(OCTAVES)
    pages = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    k = rnd(pages, page, hkv, 128)
    k[..., 0] = 0.0          # channel 0 is the only one that queries look at
    k[0, 0, :, 0] = 4.0
    v = 1.0 + 0.25 * rnd(pages, page, hkv, 128)
    v[0, 0] = 0.0
    ds = {}
    if dtype == "e4m3":
        k, v = k.mul(2.0).to(torch.float8_e4m3fn), v.mul(64.0).to(torch.float8_e4m3fn)
        ds = dict(k_descale=torch.tensor([0.5], device="cuda"), v_descale=torch.tensor([1 / 64], device="cuda"))
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    q = rnd(B, hkv, group, 128)
    q[..., 1:] = 0.0
    q[..., 0] = torch.tensor(OCTAVES, device="cuda") * math.log(2.0) / 4.0
    q = q.to(torch.bfloat16).view(B, hkv * group, 128)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, pages).contiguous()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    out, lse = zq.attn_decode(q, k, v, table, lens, softmax_scale=1.0, **ds)
    vd = v.view(-1, hkv, 128)[1:n].double() * (1 / 64 if dtype == "e4m3" else 1.0)
    w = torch.exp(-4.0 * q[0, :, 0].double())  # of the others, the first key's being 1
    total = 1.0 + (n - 1) * w
    scale = (w / total).view(hkv, group, 1)
    want = scale * vd.sum(0)[:, None]
    mass, each = scale * vd.abs().sum(0)[:, None], vd.abs().sum(0)[:, None] / total.view(hkv, group, 1)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -9 + (2.0 ** -16 if dtype == "bf16" else 2.0 ** -11)) * mass
    if dtype == "e4m3":
        tol = tol + 2.0 ** -36 * each
    off = (out.double().view(B, hkv, group, 128) - want).abs() / tol
    assert off.max().item() <= 1.0, off.amax(dim=(0, 1, 3)).tolist()
    assert (lse.double() - torch.log(total) - 4.0 * q[0, :, 0].double()).abs().max().item() <= 2.0 ** -10


@pytest.mark.parametrize("n", [2, 16, 33, 200])
@pytest.mark.parametrize("room", [512, 65536])
def test_bf16_weights_keep_two_roundings(n, room):
    """Weights over a bf16 cache enter as the sum of two bf16 values.  The
    values are such that the output nearly cancels (the heaviest key against
    all others), so its own rounding hides nothing.

    Queries are +-1 and keys multiples of 1/8, so q . k is exact in fp32.  A
    score s of up to 4 octaves carries the scale's rounding and its own, 2^-24 of
    it each, and s minus the reference, up to 8 octaves, is rounded once more:
    3 * 2^-21 octaves in all, times ln 2, and ex2.approx 2^-22: a weight is off
    by less than 2^-19 of itself.  Its two roundings to bf16 leave 2^-16 of it,
    and the sums of n terms are off by n steps of 2^-23 at most.  Numerator and
    denominator: (2^-16 + 2 (2^-19 + n 2^-23)) A, and the output's own 2^-8."""
    zq = _zq()
    hq, hkv, page = 8, 2, 16
    g = torch.Generator().manual_seed(n)
    q = torch.randint(0, 2, (1, hq, 128), generator=g).mul(2.0).sub(1.0).to(torch.bfloat16)
    pages = -(-n // page)
    k = (torch.randint(-8, 9, (pages, page, hkv, 128), generator=g) / 8.0).to(torch.bfloat16)
    v = torch.randint(0, 2, (pages, page, hkv, 128), generator=g).mul(2.0).sub(1.0)
    scale = 2.0 / 3.0 / math.sqrt(128)
    x = torch.einsum("gjd,ngd->gjn", q[0].double().view(hkv, hq // hkv, 128), k.view(-1, hkv, 128)[:n].double()) * scale
    assert x.abs().max().item() * 1.4427 <= 4.0
    # one head of each group cancels: its heaviest key takes minus the others' sum over its weight
    w = torch.softmax(x[:, 0], dim=-1)
    vf = v.view(-1, hkv, 128)
    for h in range(hkv):
        top = int(w[h].argmax())
        rest = (w[h, :, None] * vf[:n, h].double()).sum(0) - w[h, top] * vf[top, h].double()
        vf[top, h] = (-rest / w[h, top]).float()
    v = v.to(torch.bfloat16)

    class Flat:
        pass

    c = Flat()
    c.hkv, c.lens = hkv, [n]
    c.rows = lambda name, b: ((k if name == "k" else v).view(-1, hkv, 128)[:n].double(), torch.ones(n, dtype=torch.bool))
    ro, rl, mass = decode_ref(c, q, scale)
    table = torch.full((1, room // page), -1, dtype=torch.int32)
    table[0, :pages] = torch.arange(pages, dtype=torch.int32)
    out, lse = zq.attn_decode(q.cuda(), k.cuda(), v.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), softmax_scale=scale)
    tol = 2.0 ** -8 * ro.abs() + (2.0 ** -16 + 2 * (2.0 ** -19 + n * 2.0 ** -23)) * mass
    cancel = slice(0, None, hq // hkv)
    assert (ro.abs() / mass)[0, cancel].median().item() <= 2.0 ** -7  # (so the first term is small there)
    off = (out.double().cpu() - ro).abs() / tol
    assert off.max().item() <= 1.0, off.max().item()
    assert ((lse.double().cpu() - rl).abs() <= 2.0 ** -18 + n * 2.0 ** -23 + 2.0 ** -22 * rl.abs()).all()
