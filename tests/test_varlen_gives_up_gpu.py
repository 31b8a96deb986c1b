"""The packed kernels' way out when a wait runs into its limit.  The debug entry
keeps the matrix issuers from learning that P is written; every wait then runs
out, the kernel reports through the status word and returns, and the next call is
as always."""
import time

import pytest
import torch

from test_varlen_gpu import MANY, Pack

pytestmark = pytest.mark.gpu

# units of one tile and of many (more key tiles than stages), rows without keys
LENS = [(700, 700), (1, 1), (40, 900), (3, 0), (128, 128), (300, 200)] * 4
CASES = [(LENS, 12, 4, 128, "bf16"), (LENS, 12, 4, 192, "bf16"), (LENS, 12, 4, 128, "leanp"), (LENS, 12, 4, 192, "exact"), (MANY, 48, 6, 128, "bf16")]


@pytest.mark.parametrize("lens,hq,hkv,dqk,dtype", CASES)
def test_withheld_work_ends_with_a_status(lens, hq, hkv, dqk, dtype):
    import bf16_causal_prefill_02_b200 as zq

    p = Pack(lens, hq, hkv, dqk, dtype, seed=300)
    a = p.args()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = zq.attn_varlen(status=status, **a)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    t = time.monotonic()
    zq.attn_varlen(status=status, debug_flags=1, **a)
    torch.cuda.synchronize()
    assert int(status.item()) == zq.ZQ_ERR_TIMEOUT
    assert time.monotonic() - t < 20.0  # a few tenths of a second for each wave of CTAs
    status.zero_()
    again = zq.attn_varlen(status=status, **a)
    assert int(status.item()) == 0
    assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    p.check(*again, rows=131)


def test_without_a_status_word():
    import bf16_causal_prefill_02_b200 as zq

    p = Pack([(200, 200)], 4, 2, 128, "bf16", seed=301)
    zq.attn_varlen(debug_flags=1, **p.args())
    torch.cuda.synchronize()
    p.check(*zq.attn_varlen(**p.args()))
