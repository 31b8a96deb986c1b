"""The paged decode's forms (one launch, or a line of keys joined by (sequence,
head tile) or by the warps' cuts), each over the lengths, heads and pages where
it can go wrong.

Which form ran is read from the workspace: it starts with one record of 16 bytes
for each cut, {sequence, head tile, parts, first part}.  One launch leaves it as
it was; a join by (sequence, head tile) writes a record for each of those, one
by cuts a record for each warp of the grid."""
import pytest
import torch

from paged_cases import Cache, check_decode

pytestmark = pytest.mark.gpu

EDGE = [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 1000]
ROOM = 65536  # keys that the widened tables have room for: too many for one launch


def _run(c, q, room=ROOM):
    """attn_decode over c with its table widened to `room` keys: (out, lse, records written, parts to join)."""
    import bf16_causal_prefill_02_b200 as zq

    a = c.cuda()
    if room:
        wide = torch.full((len(c.lens), room // c.page), -1, dtype=torch.int32)
        wide[:, :c.table.shape[1]] = c.table
        a["block_table"] = wide.cuda()
    w = torch.full((zq.zq_decode_workspace_bytes(),), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = zq.attn_decode(q.cuda(), workspace=w, **a)
    cut = w[:1280 * 16].view(torch.int32).view(1280, 4).cpu()
    return out, lse, int((cut != -1).any(dim=1).sum()), int(cut[:, 2].clamp(min=0).sum())


def _q(b, hq, d, seed=1):
    return torch.randn((b, hq, d), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def _expect(b, hq, hkv):
    """Records of the line: (sequence, head tile) pairs where the join goes by those, else None (one per warp)."""
    group = hq // hkv
    items = b * hkv * -(-group // 16)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return items if items * min(group, 16) <= 4 * sms else None


def _check(c, q, hq, **kw):
    out, lse, records, parts = _run(c, q, **kw)
    items = _expect(len(c.lens), hq, c.hkv)
    if items is None:
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert records == min(2 * sms, 320) * 4
    else:
        assert records == items
    assert parts > 0
    check_decode(c, q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,dqk", [(8, 2, 128), (2, 2, 192), (5, 1, 128), (16, 1, 192), (40, 2, 128), (40, 2, 192), (12, 1, 128)])
@pytest.mark.parametrize("page", [1, 8, 16, 128])
def test_line_edge_lengths(dtype, hq, hkv, dqk, page):
    c = Cache(EDGE, hkv, dqk, page, dtype, seed=7)
    c.table[10, 2] = -1
    _check(c, _q(len(EDGE), hq, dqk), hq)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,dqk", [(3, 1, 128), (24, 1, 192)])
def test_line_more_sequences_than_threads(dtype, hq, hkv, dqk):
    lens = [(7 * i) % 41 for i in range(777)]
    c = Cache(lens, hkv, dqk, 16, dtype, seed=9)
    _check(c, _q(len(lens), hq, dqk), hq)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,hq,hkv,dqk", [([300] * 200, 8, 2, 128), ([600 + 37 * (i % 9) for i in range(40)], 32, 8, 128),
                                            ([5000] + [20] * 150, 16, 4, 128), ([3000, 1, 0, 900] * 12, 32, 2, 192)])
def test_line_joins_by_entry(dtype, lens, hq, hkv, dqk):
    c = Cache(lens, hkv, dqk, 32, dtype, seed=19)
    assert _expect(len(lens), hq, hkv) is None
    _check(c, _q(len(lens), hq, dqk), hq)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,hq,hkv,dqk", [([20000], 8, 2, 128), ([9000, 3], 16, 1, 192), ([4000, 0, 77], 40, 2, 128)])
def test_line_joins_by_item(dtype, lens, hq, hkv, dqk):
    c = Cache(lens, hkv, dqk, 64, dtype, seed=29)
    assert _expect(len(lens), hq, hkv) is not None
    _check(c, _q(len(lens), hq, dqk), hq)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,hq,hkv,room", [([200], 8, 2, 256), ([64, 0, 480], 16, 1, 512), ([100] * 9, 8, 2, 128), ([31] * 700, 4, 1, 64)])
def test_small_tables_leave_the_workspace_alone(dtype, lens, hq, hkv, room):
    c = Cache(lens, hkv, 128, 16, dtype, seed=39)
    q = _q(len(lens), hq, 128)
    out, lse, records, _ = _run(c, q, room=room)
    assert records == 0
    check_decode(c, q, out, lse)
