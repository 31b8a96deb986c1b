"""Refusals of the serving operators that keep a kernel from addresses it may
not read, on a host without a GPU: no call here has valid arguments."""
import pytest

import bf16_causal_prefill_02_b200 as zq
from test_paged_boundary import A, _cache


@pytest.mark.parametrize("B,hkv,hq,width,page", [(65535, 4096, 4096, 1 << 14, 1 << 16), (65535, 1, 4096, 1 << 30, 1), (4096, 8, 4096, 1 << 15, 1 << 15)])
def test_decode_refuses_lines_past_63_bits(B, hkv, hq, width, page):
    # more key tiles, times pieces of the line, than 63 bits hold
    c = _cache(B=B, Hkv=hkv, table_width=width, page_size=page)
    assert B * hq * width * page > 1 << 53
    assert zq.zq_attn_decode(c, A, 0, hq, 0.0, A, A, A, None) == zq.ZQ_ERR_SHAPE


def test_lines_that_are_accepted_fit_63_bits():
    # the largest line that passes: 16-key tiles, 5 further places for each (sequence, head), 1280 pieces
    keys_and_heads, pairs = 1 << 53, 65535 * 4096
    assert (keys_and_heads // 16 + 5 * pairs) * 1280 < 2 ** 63
