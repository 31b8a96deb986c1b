"""FP8 attention where a scale is 0, as the quantiser gives for a head whose
values are all 0, or where the product of the scales vanishes in 32 bits: every
score is 0, so a row's output is the mean of its visible values and its lse the
logarithm of their number.

Tolerance: the weights of a row are all 2^T exactly, so the output is off by its
rounding to bf16 (2^-8 of the value) and by the fp32 sums of n <= 1024 terms
(n 2^-24 <= 2^-14 of the mean of |v|).  lse: the sum is exact, log2 of a
value below 2^19 is off by 2 units in the last place at most (2^-18), and the
product with ln 2 rounds once more: 2^-17."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _zq():
    import bf16_causal_prefill_02_b200 as zq

    return zq


def _codes(n, h, d, seed):
    return torch.randn((n, h, d), generator=torch.Generator().manual_seed(seed)).mul(40).to(torch.float8_e4m3fn)


def _check_means(out, lse, v, sq, sk, causal):
    """out (Sq, 128), lse (Sq) of one head over the values v (Sk, 128)."""
    seen = [min(sk, max(0, i + sk - sq + 1)) if causal else sk for i in range(sq)]
    sums, mass = v.double().cumsum(0), v.double().abs().cumsum(0)
    for i, n in enumerate(seen):
        if n == 0:
            assert (out[i] == 0).all() and math.isinf(lse[i])
            continue
        want = sums[n - 1] / n
        assert ((out[i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -14 * mass[n - 1] / n).all(), i
        assert abs(float(lse[i]) - math.log(n)) <= 2.0 ** -17, (i, float(lse[i]), math.log(n))


LENS = [(200, 200), (130, 400), (300, 150), (1, 1)]


@pytest.mark.parametrize("mode", ["exact", "leanp"])
@pytest.mark.parametrize("dqk", [128, 192])
@pytest.mark.parametrize("block_scale,T,causal", [(True, 8, True), (False, 8, True), (True, 3, False)])
def test_packed_prompts_with_a_zero_head(mode, dqk, block_scale, T, causal):
    zq = _zq()
    hq, hkv = 4, 2
    tq, tk = sum(a for a, _ in LENS), sum(b for _, b in LENS)
    q, k, v = _codes(tq, hq, dqk, 1), _codes(tk, hkv, dqk, 2), _codes(tk, hkv, 128, 3)
    cu = [torch.tensor([0] + [sum(n[i] for n in LENS[:b + 1]) for b in range(len(LENS))], dtype=torch.int32) for i in range(2)]
    ds = {x: (0.01 + 0.01 * torch.rand((len(LENS), hkv), generator=torch.Generator().manual_seed(4 + i))) for i, x in enumerate("qkv")}
    a = dict(causal=causal, softmax_mode=zq.ZQ_SOFTMAX_EXACT if mode == "exact" else zq.ZQ_SOFTMAX_LEANP, block_scale=block_scale, headroom_T=T)

    def call():
        return zq.attn_varlen(q.cuda(), k.cuda(), v.cuda(), cu[0].cuda(), cu[1].cuda(), **{x + "_descale": ds[x].cuda() for x in ds}, **a)

    before = call()
    zero = {(0, 1): "k", (1, 0): "q", (2, 1): "qk", (3, 0): "tiny"}  # (sequence, kv head)
    for (b, g), what in zero.items():
        rows = {"q": slice(int(cu[0][b]), int(cu[0][b + 1])), "k": slice(int(cu[1][b]), int(cu[1][b + 1]))}
        for x in "qk":
            if what == "tiny":
                ds[x][b, g] = 1e-30  # the product is 0 in 32 bits; codes as they are
            elif x in what:
                ds[x][b, g] = 0.0
                (q[rows["q"], 2 * g:2 * g + 2] if x == "q" else k[rows["k"], g])[:] = 0.0
    out, lse = (t.cpu() for t in call())
    for b, (sq, sk) in enumerate(LENS):
        rq, rk = slice(int(cu[0][b]), int(cu[0][b + 1])), slice(int(cu[1][b]), int(cu[1][b + 1]))
        for h in range(hq):
            if (b, h // 2) in zero:
                _check_means(out[rq, h], lse[h, rq], v[rk, h // 2].float() * ds["v"][b, h // 2], sq, sk, causal)
            else:  # the others are what they were
                assert torch.equal(out[rq, h], before[0].cpu()[rq, h]) and torch.equal(lse[h, rq], before[1].cpu()[h, rq])


@pytest.mark.parametrize("mode", ["exact", "leanp"])
def test_packed_prompts_quantised_with_a_head_of_zeros(mode):
    # the quantiser's own scale of 0
    zq = _zq()
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn((1, 500, h, 128), generator=g).cuda() for h in (4, 2, 2))
    k[:, :, 1] = 0.0
    (cq, dq), (ck, dk), (cv, dv) = (zq.quantize_fp8_grouped(x, heads_per_scale=n) for x, n in ((q, 2), (k, 1), (v, 1)))
    assert float(dk[0, 1]) == 0.0
    cu = torch.tensor([0, 500], dtype=torch.int32, device="cuda")
    out, lse = zq.attn_varlen(cq[0], ck[0], cv[0], cu, cu, q_descale=dq, k_descale=dk, v_descale=dv,
                              softmax_mode=zq.ZQ_SOFTMAX_EXACT if mode == "exact" else zq.ZQ_SOFTMAX_LEANP)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    for h in (2, 3):
        _check_means(out[:, h].cpu(), lse[h].cpu(), (cv[0, :, 1].float() * dv[0, 1]).cpu(), 500, 500, True)


@pytest.mark.parametrize("mode", ["exact", "leanp"])
@pytest.mark.parametrize("dqk", [128, 192])
@pytest.mark.parametrize("sq,sk,causal", [(200, 200, True), (130, 400, True), (300, 150, True), (77, 200, False)])
def test_fixed_batch_with_a_zero_head(mode, dqk, sq, sk, causal):
    zq = _zq()
    q, k, v = _codes(2 * sq, 4, dqk, 11).view(2, sq, 4, dqk), _codes(2 * sk, 2, dqk, 12).view(2, sk, 2, dqk), _codes(2 * sk, 2, 128, 13).view(2, sk, 2, 128)
    ds = {x: torch.full((2, 2), 0.02) for x in "qkv"}
    ds["k"][0, 1], k[0, :, 1] = 0.0, 0.0
    ds["q"][1, 0], ds["k"][1, 0] = 1e-30, 1e-30  # the product is 0 in 32 bits
    out, lse = zq.attn_fwd(q.cuda(), k.cuda(), v.cuda(), causal=causal, softmax_mode=zq.ZQ_SOFTMAX_EXACT if mode == "exact" else zq.ZQ_SOFTMAX_LEANP,
                           **{x + "_descale": ds[x].cuda() for x in ds})
    for b, g in ((0, 1), (1, 0)):
        for h in (2 * g, 2 * g + 1):
            _check_means(out[b, :, h].cpu(), lse[b, h].cpu(), v[b, :, g].float() * ds["v"][b, g], sq, sk, causal)
    assert torch.isfinite(out).all()
