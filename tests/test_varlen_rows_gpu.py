"""Packed prompts in tensors of more than 2^31 elements, in the kernel with one
query tile per CTA (FP8 and 192-wide heads never take the other)."""
import pytest
import torch

from test_varlen_gpu import Pack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,hq,hkv,dqk", [("leanp", 16, 2, 128), ("bf16", 12, 3, 192)])
def test_rows_past_32_bits_one_tile_per_cta(dtype, hq, hkv, dqk):
    import bf16_causal_prefill_02_b200 as zq

    p = Pack([(300, 300), (70, 131)], hq, hkv, dqk, dtype, seed=251)
    a = p.args()
    n = 370
    rows = 2 ** 31 // (hq * 128) + 500
    assert (rows - n) * hq * 128 > 2 ** 31 and (rows - n) * hq * dqk > 2 ** 31  # first rows in use, of out and of q
    q = torch.empty((rows, hq, dqk), dtype=a["q"].dtype, device="cuda")
    q[rows - n:] = a["q"]
    out = torch.empty((rows, hq, 128), dtype=torch.bfloat16, device="cuda")
    out[:rows - n] = 3.0
    a.update(q=q, cu_seqlens_q=torch.tensor([rows - n, rows - 70, rows], dtype=torch.int32, device="cuda"))
    _, lse = zq.attn_varlen(out=out, **a)
    p.check(out[rows - n:], lse[:, rows - n:])
    assert (out[:rows - n] == 3.0).all()
