"""GPU tests of attention over packed prompts, against the oracle on every
sequence of its own, with the tolerances of the fixed-batch kernel (attn_cases)
taken over the pack; FP8 sequences are quantised one by one, so that the pack
runs with one scale per (sequence, kv head).

Rounding flips (FP8): a row counts as a flip where a score lands on the other
side of an e4m3 boundary than the emulation's.  fp32 scores are off by about
1e-6 in the log2 domain and the boundaries lie at least 1/16 apart, so a key
flips with a probability of about 3e-5, and a row, of which some tens of keys
carry weight, of about 1e-3: the share that attn_cases allows.  A pack of few
rows may have a flip all the same: the count is Poisson with a mean of at most
m = 1e-3 rows, so it is held to m + 4 sqrt(m) + 3."""
import math

import numpy as np
import pytest
import torch

import oracle
import workloads
from attn_cases import (CODE_STEP, ELEM_ABS, ELEM_ULPS, LSE_FLIP_BOUND, LSE_FLIP_FRAC, TOL_LSE_BF16, TOL_LSE_FP8, TOL_R1, TOL_R1_MAXABS_BF16,
                        TOL_R2, Case, bf16_ulp)
from paged_cases import Cache, check_decode

pytestmark = pytest.mark.gpu


def _zq():
    import bf16_causal_prefill_02_b200 as zq

    return zq


class Pack:
    """Sequences of (Sq, Sk) rows, packed; `front` and `back` rows belong to none."""

    def __init__(self, lens, hq, hkv, dqk, dtype="bf16", causal=True, seed=0, front=0, back=0, block_scale=True, T=8, std=1.0):
        self.lens, self.hq, self.hkv, self.dqk, self.dtype, self.causal = lens, hq, hkv, dqk, dtype, causal
        self.block_scale, self.T, self.front, self.back = block_scale, T, front, back
        self.cases = [None if not sq or not sk else
                      Case(1, sq, sk, hq, hkv, dqk, 128, dtype=dtype, causal=causal, seed=seed + i, std=std, block_scale=block_scale, T=T,
                           per_kv_descale=dtype != "bf16") for i, (sq, sk) in enumerate(lens)]

    def _rows(self, x):
        heads, d = (self.hq, self.dqk) if x == "q" else (self.hkv, self.dqk if x == "k" else 128)
        fp8 = self.dtype != "bf16"
        t = torch.uint8 if fp8 else torch.bfloat16
        none = lambda n: torch.full((n, heads, d), 0x7F if fp8 else float("nan"), dtype=t)  # noqa: E731
        parts = [none(self.front)]
        for c, (sq, sk) in zip(self.cases, self.lens):
            n = sq if x == "q" else sk
            parts.append(none(n) if c is None else torch.from_numpy(getattr(c, "c" + x))[0] if fp8 else getattr(c, x + "b")[0])
        return torch.cat(parts + [none(self.back)]).contiguous()

    def cu(self, i):
        return torch.tensor(np.cumsum([self.front] + [n[i] for n in self.lens]), dtype=torch.int32)

    def args(self):
        a = dict(zip("qkv", (self._rows(x).cuda() for x in "qkv")))
        a.update(cu_seqlens_q=self.cu(0).cuda(), cu_seqlens_k=self.cu(1).cuda(), causal=self.causal)
        if self.dtype != "bf16":
            zq = _zq()
            for x in "qkv":
                a[x + "_descale"] = torch.from_numpy(np.stack([
                    np.ones(self.hkv, dtype=np.float32) if c is None else np.asarray(getattr(c, "ds" + x), dtype=np.float32).reshape(-1)
                    for c in self.cases])).cuda()
            a.update(softmax_mode=zq.ZQ_SOFTMAX_EXACT if self.dtype == "exact" else zq.ZQ_SOFTMAX_LEANP,
                     block_scale=self.block_scale, headroom_T=self.T)
        return a

    def check(self, out, lse, rows=None, gate_r1=True, only=None):
        """The pack's outputs, or those of the sequences `only`, against the oracle."""
        got, want1, want2, hard, at = [], [], [], [], self.cu(0)
        for b, c in enumerate(self.cases):
            if only is not None and b not in only:
                continue
            o, l = out[at[b]:at[b + 1]], lse[:, at[b]:at[b + 1]]
            if c is None:
                assert (o == 0).all() and torch.isneginf(l).all()
                continue
            r = np.arange(self.hq * c.Sq) if rows is None or c.Sq <= 256 else workloads.sample_rows(1, self.hq, c.Sq, every=rows).numpy()
            got.append(c.gather(o[None], l[None], r))
            want1.append(c.r1(r))
            want2.append(c.r2(r) if c.fp8 else want1[-1])
            hard.append(np.full(len(r), CODE_STEP[c.dtype] * 2.0 * np.abs(c.vd).max() if c.fp8 else np.inf))
        if not got:
            return
        (o, l), (r1o, r1l), (r2o, r2l) = ([np.concatenate(x) for x in zip(*y)] for y in (got, want1, want2))
        assert np.all(np.isfinite(o)), "non-finite output"
        empty = np.isneginf(r1l)
        assert np.array_equal(np.isneginf(l), empty) and np.all(o[empty] == 0)
        r1, dl = oracle.rel_rmse(o, r1o), np.abs(np.where(empty, 0.0, l) - np.where(empty, 0.0, r2l))
        assert not gate_r1 or r1 <= TOL_R1[self.dtype], r1
        if self.dtype == "bf16":
            assert dl.max() <= TOL_LSE_BF16, dl.max()
            assert not gate_r1 or np.abs(o - r1o).max() <= TOL_R1_MAXABS_BF16, np.abs(o - r1o).max()
            return
        assert oracle.rel_rmse(o, r2o) <= TOL_R2, oracle.rel_rmse(o, r2o)
        assert dl.max() <= LSE_FLIP_BOUND[self.dtype], dl.max()
        diff = np.abs(o - r2o)
        over = (diff / (ELEM_ULPS * bf16_ulp(r2o) + ELEM_ABS * np.abs(r2o).max())).max(axis=1) > 1.0
        flips, m = int(np.sum((dl > TOL_LSE_FP8) | over)), LSE_FLIP_FRAC * len(l)
        assert flips <= m + 4 * math.sqrt(m) + 3, (flips, len(l))
        assert np.all(diff.max(axis=1) <= np.concatenate(hard))


EDGE = [(1, 1), (0, 5), (127, 127), (128, 128), (129, 129), (3, 0), (2, 300), (300, 2), (0, 0), (257, 400), (1, 129), (64, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "exact", "leanp"])
@pytest.mark.parametrize("hq,hkv,dqk", [(4, 2, 128), (2, 2, 192), (5, 1, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_edge_lengths(dtype, hq, hkv, dqk, causal):
    p = Pack(EDGE, hq, hkv, dqk, dtype, causal, seed=1)
    out, lse = _zq().attn_varlen(**p.args())
    p.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "exact", "leanp"])
def test_rows_of_no_sequence_stay_and_do_not_matter(dtype):
    # NaN before, behind, and in a sequence without queries between two others
    p = Pack([(70, 70), (0, 40), (200, 131), (5, 77)], 4, 2, 128, dtype, seed=40, front=9, back=200)
    a = p.args()
    total = a["q"].shape[0]
    out = torch.full((total, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, total), 3.0, device="cuda")
    o, l = _zq().attn_varlen(out=out, lse=lse, **a)
    assert o is out and l is lse
    p.check(out, lse)
    last = int(p.cu(0)[-1])
    assert (out[:9] == 3).all() and (out[last:] == 3).all() and (lse[:, :9] == 3).all() and (lse[:, last:] == 3).all()


@pytest.mark.parametrize("dtype", ["bf16", "leanp"])
def test_a_sequence_of_nan_spoils_no_other(dtype):
    p = Pack([(130, 130), (100, 100), (260, 260)], 4, 2, 128, dtype, seed=50)
    a = p.args()
    for x in "qkv":
        a[x][130:230] = float("nan") if dtype == "bf16" else 0x7F
    a["v"][130:135] = float("inf") if dtype == "bf16" else 0x7F
    out, lse = _zq().attn_varlen(**a)
    p.check(out, lse, only=(0, 2))


@pytest.mark.parametrize("dtype", ["bf16", "leanp"])
@pytest.mark.parametrize("n", [300, 777])
def test_many_short_sequences(dtype, n):
    # more sequences than prefix slots, and CTAs that cross many of them
    lens = [((13 * i) % 29, (13 * i) % 29 + (7 * i) % 3) for i in range(n)]
    p = Pack(lens, 2, 1, 128, dtype, seed=60)
    out, lse = _zq().attn_varlen(**p.args())
    p.check(out, lse)


@pytest.mark.parametrize("dtype,hq,hkv,dqk", [("bf16", 8, 2, 128), ("leanp", 8, 2, 128), ("bf16", 4, 4, 192), ("exact", 4, 4, 192)])
def test_long_and_short_together(dtype, hq, hkv, dqk):
    p = Pack([(37, 37), (5000, 5000), (1000, 7000), (128, 128), (513, 513)], hq, hkv, dqk, dtype, seed=70)
    out, lse = _zq().attn_varlen(**p.args())
    p.check(out, lse, rows=97)


@pytest.mark.parametrize("dtype", ["exact", "leanp"])
@pytest.mark.parametrize("T,block_scale", [(0, True), (4, False), (8, False)])
def test_fp8_options(dtype, T, block_scale):
    p = Pack([(200, 200), (77, 300)], 2, 2, 128, dtype, seed=80, T=T, block_scale=block_scale)
    out, lse = _zq().attn_varlen(**p.args())
    p.check(out, lse, gate_r1=False)


@pytest.mark.parametrize("dtype", ["bf16", "exact", "leanp"])
def test_growing_logits_move_the_reference(dtype):
    p = Pack([(400, 400), (300, 600)], 2, 1, 128, dtype, seed=90, std=3.0)
    out, lse = _zq().attn_varlen(**p.args())
    p.check(out, lse, gate_r1=False)


@pytest.mark.parametrize("dtype", ["exact", "leanp"])
@pytest.mark.parametrize("dqk", [128, 192])
def test_fp8_agrees_with_the_fixed_batch_kernel(dtype, dqk):
    # the same P but for keys next to a rounding border (another order of the
    # scale's factors, a closer exp2): a row differs by at most one code step
    zq = _zq()
    c = Case(2, 700, 700, 4, 2, dqk, 128, dtype=dtype, seed=7)
    o, l = c.run_gpu()
    q, k, v = (torch.from_numpy(x).cuda().flatten(0, 1) for x in (c.cq, c.ck, c.cv))
    ds = {n: torch.tensor([float(x)], device="cuda") for n, x in zip(("q_descale", "k_descale", "v_descale"), (c.dsq, c.dsk, c.dsv))}
    cu = torch.tensor([0, 700, 1400], dtype=torch.int32, device="cuda")
    mode = zq.ZQ_SOFTMAX_EXACT if dtype == "exact" else zq.ZQ_SOFTMAX_LEANP
    ov, lv = zq.attn_varlen(q, k, v, cu, cu, softmax_mode=mode, **ds)
    assert (lv.view(4, 2, 700).transpose(0, 1) - l).abs().max().item() <= LSE_FLIP_BOUND[dtype]
    assert (ov.view(2, 700, 4, 128).float() - o.float()).abs().max().item() <= CODE_STEP[dtype] * 2 * np.abs(c.vd).max()
    assert (ov.view(2, 700, 4, 128) != o).any(dim=-1).float().mean().item() <= 0.05


@pytest.mark.parametrize("lo,hi", [(-0.5, 0.5), (-100.0, 0.0)])
def test_degree_5_exp2(lo, hi):
    # fitted bound 2.33e-7 in fp32 Horner, one further rounding for the fused steps' order and the reference's own
    zq = _zq()
    x = torch.linspace(lo, hi, 100001, device="cuda")
    y = torch.empty_like(x)
    assert zq.zq_debug_exp2(x.data_ptr(), y.data_ptr(), x.numel(), 5, torch.cuda.current_stream().cuda_stream) == zq.ZQ_OK
    rel = (y.double() / torch.exp2(x.double()) - 1).abs().max().item()
    assert rel <= 2.33e-7 + 2.0 ** -23, rel


# At least 4 x 148 units of 256 rows and 256 rows a sequence: two query tiles
# per CTA (BF16, d = 128), here with both tiles, one, and none of a pair in use.
MANY = [(1, 1), (700, 700), (0, 5), (257, 257), (256, 256), (128, 128), (900, 1400), (385, 60), (3, 0), (1500, 1501), (641, 641)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv", [(48, 6), (32, 32), (40, 8)])
def test_two_tiles_per_cta(hq, hkv, causal):
    p = Pack(MANY, hq, hkv, 128, "bf16", causal, seed=200, front=3, back=130)
    a = p.args()
    assert a["q"].shape[0] >= 256 * len(MANY) and (a["q"].shape[0] + 255 * len(MANY)) // 256 * hq >= 4 * 148
    out = torch.full((a["q"].shape[0], hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    _, lse = _zq().attn_varlen(out=out, **a)
    p.check(out, lse, rows=61 if causal else 131)
    last = int(p.cu(0)[-1])
    assert (out[:3] == 3).all() and (out[last:] == 3).all()
    again, lse2 = _zq().attn_varlen(**a)
    assert torch.equal(again[3:last], out[3:last]) and torch.equal(lse2[:, 3:last], lse[:, 3:last])


def test_two_tiles_per_cta_beside_a_sequence_of_nan():
    p = Pack([(300, 300), (333, 333), (800, 800), (700, 700)], 64, 8, 128, "bf16", seed=220)
    a = p.args()
    assert (a["q"].shape[0] + 255 * 4) // 256 * 64 >= 4 * 148
    for x in "qkv":
        a[x][300:633] = float("nan")
    out, lse = _zq().attn_varlen(**a)
    p.check(out, lse, rows=61, only=(0, 2, 3))


def test_two_tiles_per_cta_over_many_sequences():
    # more sequences than prefix slots, many units per CTA, launches one behind the other
    p = Pack([(256 + i % 3, 256 + i % 5) for i in range(300)], 8, 2, 128, "bf16", seed=230)
    a = p.args()
    assert (a["q"].shape[0] + 255 * 300) // 256 * 8 >= 4 * 148
    first = _zq().attn_varlen(**a)
    p.check(*first, only=(0, 1, 149, 150, 298, 299))
    for got in [_zq().attn_varlen(**a) for _ in range(40)]:
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("dtype", ["bf16", "leanp"])
def test_rows_behind_the_last_sequence_cost_nothing_but_time(dtype):
    # a buffer of 20000 rows of which 300 are in use: the grid is a bound on the buffer
    p = Pack([(100, 100), (200, 200)], 8, 2, 128, dtype, seed=240, back=19700)
    out, lse = _zq().attn_varlen(**p.args())
    p.check(out, lse)


@pytest.mark.parametrize("hq", [64, 2])
def test_rows_past_32_bits(hq):
    # the last rows of a query tensor of more than 2^31 elements (both kernels: two tiles per CTA with 64 heads)
    p = Pack([(300, 300)], hq, 2, 128, "bf16", seed=250)
    a = p.args()
    rows = 2 ** 31 // (64 * 128) + 500
    big = torch.empty((rows, hq, 128), dtype=torch.bfloat16, device="cuda")
    big[rows - 300:] = a["q"]
    out = torch.empty_like(big)
    cu = torch.tensor([rows - 300, rows], dtype=torch.int32, device="cuda")
    _, lse = _zq().attn_varlen(big, a["k"], a["v"], cu, a["cu_seqlens_k"], out=out)
    p.check(out[rows - 300:], lse[:, rows - 300:])


def test_no_keys_and_no_queries():
    zq = _zq()
    z = lambda n, h: torch.zeros((n, h, 128), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = zq.attn_varlen(z(5, 4), z(0, 2), z(0, 2), cu(0, 2, 5), cu(0, 0, 0))
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = zq.attn_varlen(z(0, 4), z(5, 2), z(5, 2), cu(0, 0, 0), cu(0, 2, 5))
    torch.cuda.synchronize()
    assert out.shape == (0, 4, 128) and lse.shape == (4, 0)


def test_offsets_outside_the_tensors_are_clamped():
    p = Pack([(100, 100)], 4, 2, 128, "bf16", seed=95)
    a = p.args()
    a["cu_seqlens_q"] = torch.tensor([-5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    a["cu_seqlens_k"] = torch.tensor([-(2 ** 31), 101], dtype=torch.int32, device="cuda")
    out, lse = _zq().attn_varlen(**a)
    p.check(out, lse)
    # descending offsets: nothing is promised but that nothing outside is touched
    a["cu_seqlens_q"] = torch.tensor([90, 10], dtype=torch.int32, device="cuda")
    sentinel = torch.full((100, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    out, _ = _zq().attn_varlen(out=sentinel, **a)
    assert (out == 5).all()


def test_flash_style_entry():
    p = Pack([(33, 33), (200, 200)], 4, 2, 128, "bf16", seed=96)
    a = p.args()
    out, lse, none = _zq().flash_attn_varlen_func(a["q"], a["k"], a["v"], a["cu_seqlens_q"], a["cu_seqlens_k"], 200, 200,
                                                  return_attn_probs=True)
    p.check(out, lse)
    assert none is None
    assert torch.equal(_zq().flash_attn_varlen_func(a["q"], a["k"], a["v"], a["cu_seqlens_q"], a["cu_seqlens_k"]), out)


@pytest.mark.parametrize("dtype", ["bf16", "leanp"])
def test_repeats_bit_for_bit_and_status_stays_clear(dtype):
    p = Pack([(700, 700), (1, 900), (129, 129), (0, 3), (450, 450)], 8, 2, 128, dtype, seed=97)
    a = p.args()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = _zq().attn_varlen(status=status, **a)
    for _ in range(100):
        again = _zq().attn_varlen(status=status, **a)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert int(status.item()) == 0


def test_two_streams_at_once():
    packs = [Pack([(500 + 9 * i, 500 + 9 * i), (60, 60)], 8, 2, 128, "bf16", seed=100 + i) for i in range(2)]
    args, streams = [p.args() for p in packs], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [(i, _zq().attn_varlen(stream=streams[i] if r % 2 else streams[i].cuda_stream, **args[i])) for r in range(10) for i in range(2)]
    torch.cuda.synchronize()
    for i, (o, l) in got[:2] + got[-2:]:
        packs[i].check(o, l)
    for i, (o, l) in got:
        assert torch.equal(o, got[i][1][0]) and torch.equal(l, got[i][1][1])


def test_captured_call_follows_its_offsets():
    p = Pack([(200, 200), (100, 100), (300, 300)], 4, 2, 128, "bf16", seed=110)
    a = p.args()
    a["cu_seqlens_q"], a["cu_seqlens_k"] = (torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(2))
    _zq().attn_varlen(**a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = _zq().attn_varlen(**a)
    for i, x in enumerate("qk"):
        a["cu_seqlens_" + x].copy_(p.cu(i))
    graph.replay()
    torch.cuda.synchronize()
    p.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prompts_then_tokens(dtype):
    # what a server does: attend over the packed prompts, keep their keys and
    # values in pages, then append and attend for each further token
    zq = _zq()
    lens, hq, hkv = [150, 1, 64], 8, 2
    g = torch.Generator().manual_seed(120)
    rnd = lambda n, h: torch.randn((n, h, 128), generator=g).to(torch.bfloat16)  # noqa: E731
    T = sum(lens)
    q, k, v = rnd(T, hq), rnd(T, hkv), rnd(T, hkv)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).cuda()
    out, lse = zq.attn_varlen(q.cuda(), k.cuda(), v.cuda(), cu, cu)
    cache = Cache([n + 5 for n in lens], hkv, 128, 16, dtype, seed=121)
    a = cache.cuda()
    have = torch.zeros(3, dtype=torch.int32).cuda()
    a["cache_seqlens"] = have
    zq.kv_append(k.cuda(), v.cuda(), cu_seqlens=cu, **a)
    have += torch.tensor(lens, dtype=torch.int32).cuda()

    def mirror():
        cache.store = {x: a[x + "_cache"].cpu() for x in "kv"}
        cache.lens = have.tolist()

    # the last prompt row attends over the whole cache
    last = torch.tensor(np.cumsum(lens) - 1)
    o, l = zq.attn_decode(q[last].cuda(), **a)
    mirror()
    check_decode(cache, q[last], o, l)
    if dtype == "bf16":  # the same numbers by both ways: two roundings to bf16 and two of the weights
        d = (o.float() - out[last.cuda()].float()).abs()
        assert (d <= 2 * (2.0 ** -8 + 2.0 ** -9) * v.abs().max().item()).all()
        assert (l - lse.t()[last.cuda()]).abs().max().item() <= 2 * 2.0 ** -10
    for _ in range(5):
        qn, kn, vn = rnd(3, hq), rnd(3, hkv), rnd(3, hkv)
        zq.kv_append(kn.cuda(), vn.cuda(), **a)
        have += 1
        o, l = zq.attn_decode(qn.cuda(), **a)
        mirror()
        check_decode(cache, qn, o, l)
    assert math.isfinite(float(o.float().sum()))
