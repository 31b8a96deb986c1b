"""Refusals of the serving operators that keep a kernel from addresses it may
not read, on a host without a GPU: no call here has valid arguments."""
import pytest

import bf16_causal_prefill_02_b200 as zq
from test_paged_boundary import A, _cache, _varlen


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


@pytest.mark.parametrize("off", [1, 2])
@pytest.mark.parametrize("kw", ["block_table", "cache_seqlens", "k_descale", "v_descale"])
def test_words_of_a_cache_must_be_aligned(kw, off):
    c = _cache(dtype=1, **{kw: A + off})
    assert zq.zq_kv_append(c, A, A, 0, 0, A, 5, None) == zq.ZQ_ERR_ALIGN
    assert zq.zq_attn_decode(c, A, 0, 4, 0.0, A, A, A, None) == zq.ZQ_ERR_ALIGN


def test_offsets_of_tokens_must_be_aligned():
    assert zq.zq_kv_append(_cache(), A, A, 0, 0, A + 2, 5, None) == zq.ZQ_ERR_ALIGN


@pytest.mark.parametrize("kw", ["cu_seqlens_q", "cu_seqlens_k", "status", "q_descale", "k_descale", "v_descale"])
def test_words_of_a_pack_must_be_aligned(kw):
    assert zq.zq_attn_varlen_fwd(_varlen(dtype=1, **{kw: A + 2}), None) == zq.ZQ_ERR_ALIGN


@pytest.mark.parametrize("flags", [2, -1, 1 << 30])
def test_unknown_debug_flags_are_refused(flags):
    assert zq.zq_attn_varlen_debug(_varlen(), flags, None) == zq.ZQ_ERR_UNSUPPORTED


def test_debug_entry_checks_its_arguments():
    assert zq.zq_attn_varlen_debug(_varlen(q=None), 1, None) == zq.ZQ_ERR_NULL
