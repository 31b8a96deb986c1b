"""GPU tests of the paged-cache operators against their definitions in 64 bits."""
import pytest
import torch

from paged_cases import Cache, check_decode

pytestmark = pytest.mark.gpu

EDGE = [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 1000]


def _q(b, hq, d, seed=1, std=1.0):
    return (torch.randn((b, hq, d), generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16)


def _zq():
    import bf16_causal_prefill_02_b200 as zq

    return zq


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hkv,dqk,page,interleaved", [(8, 128, 16, False), (1, 192, 64, True), (5, 128, 1, False), (2, 192, 256, False)])
@pytest.mark.parametrize("new", [None, [3, 0, 1, 40, 257, 0, 2]])
def test_append_writes_every_token_and_nothing_else(dtype, hkv, dqk, page, interleaved, new):
    zq = _zq()
    have = [0, 5, 63, 64, 1, 9, 300]
    cnt = [1] * len(have) if new is None else new
    c = Cache([a + b for a, b in zip(have, cnt)], hkv, dqk, page, dtype, seed=3, interleaved=interleaved)
    T = sum(cnt)
    g = torch.Generator().manual_seed(4)
    wide = torch.randn((T, hkv * (dqk + 128)), generator=g).to(torch.bfloat16) * 3  # k and v as columns of one projection
    wide[0, 0], wide[0, 1], wide[-1, -1] = float("nan"), float("inf"), 1e30
    kv = {"k": wide[:, :hkv * dqk].view(T, hkv, dqk), "v": wide[:, hkv * dqk:].view(T, hkv, 128)}
    want = {x: c.store[x].clone() for x in "kv"}
    at = 0
    for b, n in enumerate(cnt):
        pos = torch.arange(have[b], have[b] + n)
        pg = c.table[b, pos // page].long()
        for x in "kv":
            r = kv[x][at:at + n]
            if dtype == "e4m3":
                # one rounding to e4m3 of the fp32 product with the reciprocal; NaN stays NaN
                inv = (1.0 / c.descale[x])[:, None]
                r = (r.float() * inv).clamp(-448, 448).to(torch.float8_e4m3fn)
                want[x].view(torch.uint8)[pg, pos % page] = r.view(torch.uint8)
            else:
                want[x][pg, pos % page] = r
        at += n
    a = c.cuda()
    a["cache_seqlens"] = torch.tensor(have, dtype=torch.int32).cuda()
    cu = None if new is None else torch.tensor([0] + list(torch.tensor(cnt).cumsum(0)), dtype=torch.int32).cuda()
    w = wide.cuda()
    gk, gv = zq.kv_append(w[:, :hkv * dqk].unflatten(1, (hkv, dqk)), w[:, hkv * dqk:].unflatten(1, (hkv, 128)), cu_seqlens=cu, **a)
    for x, got in (("k", gk), ("v", gv)):
        bits = torch.uint8 if dtype == "e4m3" else torch.int16
        eq = got.cpu().contiguous().view(bits) == want[x].contiguous().view(bits)
        if dtype == "e4m3":  # the sign of a NaN code is free
            eq |= got.cpu().float().isnan() & want[x].float().isnan()
        assert eq.all(), (x, int((~eq).sum()))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_append_drops_tokens_that_have_no_place(dtype):
    zq = _zq()
    c = Cache([16, 32, 16, 5], 2, 128, 16, dtype, seed=5, waste=None)
    a = c.cuda()
    width = c.table.shape[1]
    # past the table, on a page that is none (-1 and too large), a negative length
    a["cache_seqlens"] = torch.tensor([16 * width, 32, 0, -3], dtype=torch.int32).cuda()
    a["block_table"][2, 0] = c.pages
    before = {x: a[x + "_cache"].clone() for x in "kv"}
    k, v = torch.ones((9, 2, 128), dtype=torch.bfloat16).cuda(), torch.ones((9, 2, 128), dtype=torch.bfloat16).cuda()
    # tokens 0 and 8 are no sequence's
    zq.kv_append(k, v, cu_seqlens=torch.tensor([1, 2, 4, 6, 8], dtype=torch.int32).cuda(), **a)
    torch.cuda.synchronize()
    for x in "kv":
        assert torch.equal(a[x + "_cache"].view(torch.uint8), before[x].view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("cu", [[0, 9, 1, 9], [9, 0, 0, 0], [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 9], [5, -7, 3, 2 ** 31 - 1]])
def test_append_offsets_that_do_not_ascend_stay_in_the_pages(dtype, cu):
    """Tokens may go to places of the three sequences or be dropped; all other
    pages keep their bits.  The table is a view whose neighbouring columns name
    such a page, so a position before or behind a sequence's entries shows."""
    zq = _zq()
    c = Cache([16, 16, 16], 2, 128, 16, dtype, seed=6)
    a = c.cuda()
    used = set(a["block_table"].flatten().tolist())
    others = torch.tensor([p for p in range(c.pages) if p not in used])
    wide = torch.full((3, 4 + a["block_table"].shape[1] + 4), int(others[0]), dtype=torch.int32).cuda()
    wide[:, 4:-4] = a["block_table"]
    a["block_table"] = wide[:, 4:-4]
    a["cache_seqlens"] = torch.zeros(3, dtype=torch.int32).cuda()
    before = {x: a[x + "_cache"].clone() for x in "kv"}
    k, v = (torch.full((9, 2, 128), 7.0, dtype=torch.bfloat16).cuda() for _ in "kv")
    zq.kv_append(k, v, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), **a)
    torch.cuda.synchronize()
    for x in "kv":
        got, was = a[x + "_cache"].cpu().view(torch.uint8), before[x].cpu().view(torch.uint8)
        assert torch.equal(got[others], was[others])


def test_append_of_nothing_and_zero_scale():
    zq = _zq()
    c = Cache([4], 2, 128, 16, "e4m3", seed=6, waste=None)
    a = c.cuda()
    k = torch.zeros((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    zq.kv_append(k, k, cu_seqlens=torch.tensor([0, 0], dtype=torch.int32).cuda(), **a)
    a["k_descale"].zero_()
    one = torch.ones((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    zq.kv_append(one, one, **a)
    torch.cuda.synchronize()
    assert (a["k_cache"].view(torch.uint8)[c.table[0, 0], 4] == 0).all()


# ------------------------------------------------------------------- decode
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,dqk", [(8, 2, 128), (2, 2, 192), (5, 1, 128), (16, 1, 192), (40, 2, 128)])
@pytest.mark.parametrize("page", [1, 16, 128])
def test_decode_edge_lengths(dtype, hq, hkv, dqk, page):
    c = Cache(EDGE, hkv, dqk, page, dtype, seed=7)
    q = _q(len(EDGE), hq, dqk)
    out, lse = _zq().attn_decode(q.cuda(), **c.cuda())
    check_decode(c, q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [[1], [64], [20000], [5000, 3, 9000], [300] * 70])
def test_decode_splits_and_joins(dtype, lens):
    c = Cache(lens, 2, 128, 64, dtype, seed=8)
    q = _q(len(lens), 8, 128)
    out, lse = _zq().attn_decode(q.cuda(), **c.cuda())
    check_decode(c, q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,dqk,page", [(8, 2, 128, 16), (40, 2, 128, 64), (16, 16, 192, 1), (6, 3, 192, 16)])
def test_decode_tiny_tables(dtype, hq, hkv, dqk, page):
    # 64 keys: some warps of a block get none
    lens = [0, 1, 15, 16, 17, 31, 33, 48, 0, 47]
    c = Cache(lens, hkv, dqk, page, dtype, seed=18)
    assert (c.table.shape[1] - (page > 1)) * page <= 64  # (the table has a column to spare)
    a = c.cuda()
    a["block_table"] = a["block_table"][:, :max(1, 64 // page)].contiguous()
    q = _q(len(lens), hq, dqk)
    out, lse = _zq().attn_decode(q.cuda(), **a)
    check_decode(c, q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,dqk,page,n", [(8, 2, 128, 16, 40), (8, 2, 128, 64, 300), (40, 2, 128, 64, 20), (24, 2, 192, 16, 150), (3, 3, 192, 1, 200), (16, 1, 128, 64, 600)])
def test_decode_small_tables_are_one_launch(dtype, hq, hkv, dqk, page, n):
    # room for 512 keys: a block or two for each (sequence, head tile), e4m3 a warp each from 592 of them on
    lens = [(89 * i) % 497 if i % 7 else 0 for i in range(n - 1)] + [511 if page == 1 else 496]
    c = Cache(lens, hkv, dqk, page, dtype, seed=28)
    assert c.table.shape[1] * page in (512, 576)
    a = c.cuda()
    a["block_table"] = a["block_table"][:, :512 // page]  # (the table has a column to spare)
    a["block_table"][3, 1] = -1
    c.table[3, 1] = -1
    q = _q(n, hq, dqk)
    out, lse = _zq().attn_decode(q.cuda(), **a)
    check_decode(c, q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,dqk,room,n", [(8, 2, 128, 256, 300), (16, 1, 128, 128, 700), (12, 4, 192, 64, 90)])
def test_decode_tables_taken_by_a_warp(dtype, hq, hkv, dqk, room, n):
    lens = [(37 * i) % (room - 15) if i % 5 else 0 for i in range(n - 1)] + [room - 16]
    c = Cache(lens, hkv, dqk, 16, dtype, seed=48)
    assert c.table.shape[1] * 16 == room
    q = _q(n, hq, dqk)
    out, lse = _zq().attn_decode(q.cuda(), **c.cuda())
    check_decode(c, q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,dqk,room,n", [(8, 2, 128, 256, 9), (8, 2, 128, 1024, 60), (40, 2, 128, 2048, 5), (16, 1, 192, 4096, 3),
                                               (6, 3, 192, 2048, 12), (8, 1, 128, 4096, 37), (4, 1, 128, 8192, 2)])
def test_decode_tables_shared_by_a_cluster(dtype, hq, hkv, dqk, room, n):
    # 2, 4 and 8 blocks a (sequence, head tile); 4096 bf16 and 8192 e4m3 keys are the most
    lens = [[room - 32, 0, 1, 33, room // 2 + 5, 700 % room, 129, 16][i % 8] for i in range(n)]
    c = Cache(lens, hkv, dqk, 32, dtype, seed=38)
    assert c.table.shape[1] * 32 == room
    c.table[0, 2] = -1
    q = _q(n, hq, dqk)
    out, lse = _zq().attn_decode(q.cuda(), **c.cuda())
    check_decode(c, q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,hq,hkv", [([300] * 200, 8, 2), ([600 + 37 * (i % 9) for i in range(40)], 32, 8), ([5000] + [20] * 150, 16, 4)])
def test_decode_joins_by_entry(dtype, lens, hq, hkv):
    # more than 592 (sequence, head) rows: the join goes over the warps' cuts
    assert len(lens) * hq > 4 * 148
    c = Cache(lens, hkv, 128, 32, dtype, seed=19)
    q = _q(len(lens), hq, 128)
    out, lse = _zq().attn_decode(q.cuda(), **c.cuda())
    check_decode(c, q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_more_sequences_than_threads(dtype):
    lens = [(7 * i) % 41 for i in range(777)]
    c = Cache(lens, 1, 128, 16, dtype, seed=9)
    q = _q(len(lens), 3, 128)
    out, lse = _zq().attn_decode(q.cuda(), **c.cuda())
    check_decode(c, q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_layouts_scale_and_given_buffers(dtype):
    zq = _zq()
    c = Cache([700, 33], 4, 192, 32, dtype, seed=10, interleaved=True, per_head=False)
    wide = _q(2, 12, 192)
    q = wide[:, 4:8]  # query columns of a fused projection
    o = torch.full((2, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    e = torch.full((2, 4), 7.0, device="cuda")
    w = torch.full((zq.zq_decode_workspace_bytes(),), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = zq.attn_decode(wide.cuda()[:, 4:8], out=o, lse=e, workspace=w, softmax_scale=0.2, **c.cuda())
    assert out is o and lse is e
    check_decode(c, q, out, lse, scale=0.2)
    out, lse = zq.attn_decode(wide.cuda()[:, 4:8], return_lse=False, **c.cuda())
    assert lse is None


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_skips_keys_whose_page_is_none(dtype):
    c = Cache([100, 64, 20], 2, 128, 16, dtype, seed=11)
    c.table[0, 2], c.table[0, 4] = -1, c.pages
    c.table[1, :] = -7  # nothing left of this sequence
    q = _q(3, 8, 128)
    out, lse = _zq().attn_decode(q.cuda(), **c.cuda())
    check_decode(c, q, out, lse)
    assert torch.isinf(lse[1]).all() and (out[1] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_lengths_outside_the_table_are_clamped(dtype):
    c = Cache([48, 32], 2, 128, 16, dtype, seed=12)
    a = c.cuda()
    a["block_table"] = a["block_table"][:, :3].contiguous()
    a["cache_seqlens"] = torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32).cuda()
    c.lens = [48, 0]
    q = _q(2, 8, 128)
    out, lse = _zq().attn_decode(q.cuda(), **a)
    check_decode(c, q, out, lse)


def test_decode_e4m3_takes_queries_of_any_size():
    # the power of two that brings each row of queries into f16's range
    c = Cache([500, 3], 2, 128, 16, "e4m3", seed=13)
    q = _q(2, 8, 128)
    size = torch.tensor([1e-30, 1e-6, 1.0, 3.0, 1e5, 1e20, 0.0, 7e-41])
    q = (q.float() * size[None, :, None]).to(torch.bfloat16)
    for h, s in enumerate([1e30, 1e6, 1.0, 0.3, 1e-5, 1e-20, 1.0, 1e38]):
        out, lse = _zq().attn_decode(q.cuda(), softmax_scale=0.1 * s, **c.cuda())
        from paged_cases import decode_ref

        ro, rl, mass = decode_ref(c, q, 0.1 * s)
        tol = 2.0 ** -8 * ro.abs() + (2.0 ** -11 + 2.0 ** -9) * mass
        assert ((out.double().cpu() - ro).abs() <= tol)[:, h].all(), h
        assert ((lse.double().cpu() - rl).abs() <= 2.0 ** -10 + 2.0 ** -22 * rl.abs())[:, h].all(), h


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_offsets_past_32_bits(dtype):
    # pages at the end of caches of more than 2^31 elements
    zq = _zq()
    c = Cache([100, 37], 8, 128, 64, dtype, seed=21, waste=None)
    pages = 33000
    assert pages * 64 * 8 * 128 > 2 ** 31
    a = c.cuda()
    for x in "kv":
        big = torch.empty((pages, 64, 8, 128), dtype=a[x + "_cache"].dtype, device="cuda")
        big[pages - c.pages:].view(torch.uint8).copy_(a[x + "_cache"].view(torch.uint8))
        a[x + "_cache"] = big
    a["block_table"] += (a["block_table"] >= 0).int() * (pages - c.pages)
    q = _q(2, 32, 128)
    out, lse = zq.attn_decode(q.cuda(), **a)
    check_decode(c, q, out, lse)
    kn, vn = (torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16) for i in (3, 4))
    lens = a.pop("cache_seqlens")
    zq.kv_append(kn.cuda(), vn.cuda(), cache_seqlens=lens - 1, **a)
    out, lse = zq.attn_decode(q.cuda(), cache_seqlens=lens, **a)
    c.store = {x: a[x + "_cache"][pages - c.pages:].cpu() for x in "kv"}
    for b in range(2):  # the last key is the new one
        n = c.lens[b] - 1
        got = c.rows("k", b)[0][n] / (c.descale["k"].double()[:, None] if dtype == "e4m3" else 1.0)
        want = kn[b] if dtype == "bf16" else (kn[b].float() * (1.0 / c.descale["k"])[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert (got - want.double()).abs().max().item() <= 1e-9 * 448
    check_decode(c, q, out, lse)


def test_decode_nan_and_infinity_in_visible_keys_show():
    c = Cache([40, 40], 1, 128, 16, "bf16", seed=14)
    c.store["k"][c.table[0, 1].long(), 3, 0, 5] = float("nan")
    q = _q(2, 4, 128)
    out, lse = _zq().attn_decode(q.cuda(), **c.cuda())
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert torch.isfinite(out[1]).all()


def test_decode_repeats_bit_for_bit():
    c = Cache([9000, 1, 4000, 0, 77], 2, 128, 64, "bf16", seed=15)
    a, q = c.cuda(), _q(5, 8, 128).cuda()
    first = _zq().attn_decode(q, **a)
    for _ in range(50):
        again = _zq().attn_decode(q, **a)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_decode_two_streams_each_with_its_workspace():
    zq = _zq()
    cs = [Cache([9000 + 100 * i, 5, 300], 2, 128, 64, "bf16", seed=20 + i) for i in range(2)]
    args, qs = [c.cuda() for c in cs], [_q(3, 8, 128, seed=i) for i in range(2)]
    qd = [q.cuda() for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for r in range(20):
        for i in range(2):
            got.append((i, zq.attn_decode(qd[i], stream=streams[i] if r % 2 else streams[i].cuda_stream, **args[i])))
    torch.cuda.synchronize()
    for i, (o, l) in got:
        check_decode(cs[i], qs[i], o, l)


def test_captured_behind_a_memset_a_copy_and_another_stream():
    # what stands before a launch in the graph is no kernel, or comes from two streams
    zq = _zq()
    c = Cache([70, 300], 2, 128, 16, "bf16", seed=17)
    a, q = c.cuda(), _q(2, 8, 128)
    qd, src = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda"), q.cuda()
    out, lse = torch.empty((2, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 8), device="cuda")
    w = torch.empty(zq.zq_decode_workspace_bytes(), dtype=torch.uint8, device="cuda")
    kn, vn = (torch.randn((2, 2, 128), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16) for i in (1, 2))
    kd, vd = kn.cuda(), vn.cuda()
    have = torch.tensor([69, 299], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    lens = a.pop("cache_seqlens")

    def step():
        out.zero_()
        lse.fill_(5.0)
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            zq.kv_append(kd, vd, cache_seqlens=have, **a)
        qd.copy_(src)
        main.wait_stream(side)
        zq.attn_decode(qd, cache_seqlens=lens, out=out, lse=lse, workspace=w, **a)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out.zero_()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for b, pos in ((0, 69), (1, 299)):
        pg = c.table[b, pos // 16].long()
        c.store["k"][pg, pos % 16], c.store["v"][pg, pos % 16] = kn[b], vn[b]
    check_decode(c, q, out, lse)


def test_captured_step_follows_the_cache_as_it_grows():
    # append then decode in one graph, replayed while the host advances the lengths
    zq = _zq()
    c = Cache([40, 200], 2, 128, 16, "bf16", seed=16, waste=None)
    start = [3, 150]
    a = c.cuda()
    lens = torch.tensor(start, dtype=torch.int32).cuda()
    q, k, v = (torch.zeros((2, h, 128), dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))
    w = torch.empty(zq.zq_decode_workspace_bytes(), dtype=torch.uint8, device="cuda")
    a.pop("cache_seqlens")

    def step():
        zq.kv_append(k, v, cache_seqlens=lens, **a)
        lens.add_(1)
        return zq.attn_decode(q, cache_seqlens=lens, workspace=w, **a)

    step()
    lens.copy_(torch.tensor(start, dtype=torch.int32))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    lens.copy_(torch.tensor(start, dtype=torch.int32))
    for i in range(30):
        qn, kn, vn = _q(2, 8, 128, seed=100 + i), _q(2, 2, 128, seed=200 + i), _q(2, 2, 128, seed=300 + i)
        for dst, src in ((q, qn), (k, kn), (v, vn)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(2):
            pos = start[b] + i
            pg = c.table[b, pos // 16].long()
            c.store["k"][pg, pos % 16], c.store["v"][pg, pos % 16] = kn[b], vn[b]
        c.lens = [n + i + 1 for n in start]
        check_decode(c, qn, out, lse)
