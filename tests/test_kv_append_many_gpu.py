"""The paged append over many sequences: the search for a token's sequence has
one level below 32 offsets, two below 1024, then three and four."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [30, 31, 32, 33, 63, 1022, 1023, 1024, 1057, 5000, 33000, 65535])
@pytest.mark.parametrize("shape", ["mixed", "sparse", "ones"])
def test_every_token_finds_its_sequence(B, shape):
    import bf16_causal_prefill_02_b200 as zq

    g = torch.Generator().manual_seed(B)
    page = 4
    cnt = {"mixed": torch.randint(0, 4, (B,), generator=g), "ones": torch.ones(B, dtype=torch.int64),
           "sparse": (torch.rand(B, generator=g) < 0.03).long() * 3}[shape]
    cnt[-1] = 2
    first = 5  # tokens before the first offset, and three behind the last, belong to none
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), cnt.cumsum(0)]) + first
    T = int(cu[-1]) + 3
    have = torch.randint(0, 3, (B,), generator=g)
    width = 2  # up to 3 keys there and 3 more
    table = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width)
    # a token's number in its first channels, exact in bf16 as two bytes and a rest
    x = torch.zeros((T, 1, 128))
    t = torch.arange(T)
    x[:, 0, 0], x[:, 0, 1], x[:, 0, 127] = t % 256, t // 256 % 256, t // 65536 + 1
    x = x.to(torch.bfloat16)
    ends = torch.tensor([0, 1, 127])
    want = torch.zeros((B * width, page, 3), dtype=torch.bfloat16)
    owner = torch.repeat_interleave(torch.arange(B), cnt)
    tok = torch.arange(first, int(cu[-1]))
    pos = have[owner] + tok - cu[owner]
    want[table[owner, pos // page].long(), pos % page] = x[tok, 0][:, ends]
    kc, vc = (torch.zeros((B * width, page, 1, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    zq.kv_append(x.cuda(), x.cuda(), kc, vc, table.cuda(), have.to(torch.int32).cuda(), cu_seqlens=cu.to(torch.int32).cuda())
    for c in (kc, vc):
        assert torch.equal(c[:, :, 0, ends.cuda()].cpu(), want)
        assert int((c != 0).sum()) == int((want != 0).sum())
