"""A step of a padded batch: slots whose length is below 0 take no token and get
0 and -inf, whatever their table says; the others are as in a batch of their own."""
import pytest
import torch

from paged_cases import Cache, check_decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("room", [128, 65536])
def test_step_with_empty_slots(dtype, packed, room):
    import bf16_causal_prefill_02_b200 as zq

    have = [40, -1, 0, -2 ** 31, 77, -7]
    c = Cache([max(n, 0) + 1 for n in have], 2, 128, 16, dtype, seed=61)
    a = c.cuda()
    table = torch.full((len(have), room // 16), -1, dtype=torch.int32)
    table[:, :c.table.shape[1]] = c.table
    a["block_table"] = table.cuda()
    lens = torch.tensor(have, dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(62)
    q, k, v = (torch.randn((len(have), h, 128), generator=g).to(torch.bfloat16) for h in (8, 2, 2))
    a.pop("cache_seqlens")
    before = {x: a[x + "_cache"].clone().view(torch.uint8) for x in "kv"}
    cu = torch.arange(len(have) + 1, dtype=torch.int32, device="cuda") if packed else None
    zq.kv_append(k.cuda(), v.cuda(), cache_seqlens=lens, cu_seqlens=cu, **a)
    for x in "kv":
        same = (a[x + "_cache"].view(torch.uint8) == before[x]).cpu().flatten(2).all(dim=2)
        changed = {(int(c.table[b, have[b] // 16]), have[b] % 16) for b in (0, 2, 4)}
        assert {(int(p), int(r)) for p, r in (~same).nonzero()} == changed
    c.store = {x: a[x + "_cache"].cpu() for x in "kv"}
    lens = torch.where(lens < 0, lens, lens + 1)
    out, lse = zq.attn_decode(q.cuda(), cache_seqlens=lens, **a)
    c.lens = [max(n, 0) for n in lens.tolist()]
    check_decode(c, q, out, lse)
    empty = torch.tensor([1, 3, 5])
    assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
