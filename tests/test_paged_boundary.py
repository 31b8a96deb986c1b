"""Refusals of the paged-cache operators, on a host without a GPU: no call
here has valid arguments, so nothing can reach a launch."""
import pytest
import torch

import bf16_causal_prefill_02_b200 as zq

A = 1 << 20  # a 16-byte aligned address that is never dereferenced

CACHE = dict(k_cache=A, v_cache=A, k_page_stride=0, v_page_stride=0, block_table=A, cache_seqlens=A, k_descale=None, v_descale=None,
             table_stride=0, table_width=4, num_pages=8, page_size=16, B=2, Hkv=2, d_qk=128, d_v=128, dtype=0, descale_per_head=0)


def _cache(**kw):
    c = zq.zq_paged_kv()
    for k, v in {**CACHE, **kw}.items():
        setattr(c, k, v)
    return c


BAD_CACHE = [
    (dict(k_cache=None), zq.ZQ_ERR_NULL),
    (dict(v_cache=None), zq.ZQ_ERR_NULL),
    (dict(block_table=None), zq.ZQ_ERR_NULL),
    (dict(cache_seqlens=None), zq.ZQ_ERR_NULL),
    (dict(B=0), zq.ZQ_ERR_SHAPE),
    (dict(B=65536), zq.ZQ_ERR_SHAPE),
    (dict(Hkv=0), zq.ZQ_ERR_SHAPE),
    (dict(num_pages=0), zq.ZQ_ERR_SHAPE),
    (dict(table_width=0), zq.ZQ_ERR_SHAPE),
    (dict(page_size=0), zq.ZQ_ERR_SHAPE),
    (dict(page_size=24), zq.ZQ_ERR_SHAPE),
    (dict(page_size=131072), zq.ZQ_ERR_SHAPE),
    (dict(table_width=1 << 27), zq.ZQ_ERR_SHAPE),
    (dict(table_stride=3), zq.ZQ_ERR_SHAPE),
    (dict(k_page_stride=16 * 2 * 128 - 8), zq.ZQ_ERR_SHAPE),
    (dict(v_page_stride=8), zq.ZQ_ERR_SHAPE),
    (dict(k_page_stride=-4096), zq.ZQ_ERR_SHAPE),
    (dict(k_page_stride=16 * 2 * 128 + 4), zq.ZQ_ERR_ALIGN),
    (dict(dtype=1, v_page_stride=16 * 2 * 128 + 8), zq.ZQ_ERR_ALIGN),
    (dict(k_cache=A + 8), zq.ZQ_ERR_ALIGN),
    (dict(v_cache=A + 2), zq.ZQ_ERR_ALIGN),
    (dict(d_qk=64), zq.ZQ_ERR_UNSUPPORTED),
    (dict(d_v=192), zq.ZQ_ERR_UNSUPPORTED),
    (dict(dtype=2), zq.ZQ_ERR_UNSUPPORTED),
    (dict(descale_per_head=2), zq.ZQ_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_bad_cache_is_refused_by_both(kw, code):
    c = _cache(**kw)
    assert zq.zq_kv_append(c, A, A, 0, 0, A, 5, None) == code
    assert zq.zq_attn_decode(c, A, 0, 4, 0.0, A, A, A, None) == code


@pytest.mark.parametrize("args,code", [
    ((None, A, 0, 0, A, 5), zq.ZQ_ERR_NULL),
    ((A, None, 0, 0, A, 5), zq.ZQ_ERR_NULL),
    ((A, A, 0, 0, A, -1), zq.ZQ_ERR_SHAPE),
    ((A, A, 0, 0, A, 1 << 31), zq.ZQ_ERR_SHAPE),
    ((A, A, 0, 0, None, 5), zq.ZQ_ERR_SHAPE),  # one token per sequence: T must be B
    ((A, A, 248, 0, A, 5), zq.ZQ_ERR_SHAPE),
    ((A, A, 0, -256, A, 5), zq.ZQ_ERR_SHAPE),
    ((A, A, 260, 0, A, 5), zq.ZQ_ERR_ALIGN),
    ((A + 2, A, 0, 0, A, 5), zq.ZQ_ERR_ALIGN),
    ((A, A + 8, 0, 0, A, 5), zq.ZQ_ERR_ALIGN),
])
def test_append_argument_errors(args, code):
    assert zq.zq_kv_append(_cache(), *args, None) == code


@pytest.mark.parametrize("args,code", [
    ((None, 0, 4, 0.0, A, A, A), zq.ZQ_ERR_NULL),
    ((A, 0, 4, 0.0, None, A, A), zq.ZQ_ERR_NULL),
    ((A, 0, 4, 0.0, A, A, None), zq.ZQ_ERR_NULL),
    ((A, 0, 0, 0.0, A, A, A), zq.ZQ_ERR_SHAPE),
    ((A, 0, 3, 0.0, A, A, A), zq.ZQ_ERR_SHAPE),  # Hq % Hkv
    ((A, 0, 8192, 0.0, A, A, A), zq.ZQ_ERR_SHAPE),
    ((A, 500, 4, 0.0, A, A, A), zq.ZQ_ERR_SHAPE),
    ((A, 0, 4, float("nan"), A, A, A), zq.ZQ_ERR_SHAPE),
    ((A, 516, 4, 0.0, A, A, A), zq.ZQ_ERR_ALIGN),
    ((A + 8, 0, 4, 0.0, A, A, A), zq.ZQ_ERR_ALIGN),
    ((A, 0, 4, 0.0, A + 2, A, A), zq.ZQ_ERR_ALIGN),
    ((A, 0, 4, 0.0, A, A + 4, A), zq.ZQ_ERR_ALIGN),
    ((A, 0, 4, 0.0, A, A, A + 4), zq.ZQ_ERR_ALIGN),
])
def test_decode_argument_errors(args, code):
    assert zq.zq_attn_decode(_cache(), *args, None) == code


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _good():
    return dict(k_cache=_t(8, 16, 2, 128), v_cache=_t(8, 16, 2, 128), block_table=_t(2, 4, dtype=torch.int32),
                cache_seqlens=_t(2, dtype=torch.int32))


@pytest.mark.parametrize("kw,err,msg", [
    (dict(k_cache=_t(8, 16, 256)), ValueError, "4-D"),
    (dict(k_cache=_t(8, 16, 2, 128, dtype=torch.float16)), TypeError, "both be bfloat16"),
    (dict(v_cache=_t(8, 16, 2, 128, dtype=torch.uint8)), TypeError, "both be bfloat16"),
    (dict(v_cache=_t(8, 16, 1, 128)), ValueError, "v_cache must have"),
    (dict(v_cache=_t(7, 16, 2, 128)), ValueError, "v_cache must have"),
    (dict(block_table=_t(2, 4, dtype=torch.int64)), ValueError, "block_table"),
    (dict(block_table=_t(8, dtype=torch.int32)), ValueError, "block_table"),
    (dict(block_table=_t(4, 2, dtype=torch.int32).t()), ValueError, "block_table must be contiguous"),
    (dict(block_table=_t(1, 4, dtype=torch.int32).expand(2, 4)), ValueError, "block_table must be contiguous"),
    (dict(cache_seqlens=_t(3, dtype=torch.int32)), ValueError, "cache_seqlens"),
    (dict(cache_seqlens=_t(2, dtype=torch.int64)), ValueError, "cache_seqlens"),
    (dict(cache_seqlens=_t(4, dtype=torch.int32)[::2]), ValueError, "cache_seqlens"),
    (dict(k_cache=_t(8, 2, 16, 128).transpose(1, 2)), ValueError, "k_cache must be contiguous"),
    (dict(), ValueError, "must be a CUDA tensor"),
])
def test_helpers_refuse_bad_caches(kw, err, msg):
    a = {**_good(), **kw}
    for call in (lambda: zq.kv_append(_t(2, 2, 128), _t(2, 2, 128), **a), lambda: zq.attn_decode(_t(2, 4, 128), **a)):
        with pytest.raises(err, match=msg):
            call()


def test_row_strides():
    t = _t(6, 2, 128)
    assert zq._row_stride("t", t) == 0
    assert zq._row_stride("t", _t(6, 4, 128)[:, 1:3]) == 512
    assert zq._row_stride("t", t[:0]) == 0
    for bad in (t.transpose(1, 2), t[:1].expand(6, 2, 128), t[:, :, ::2], t.transpose(0, 1)):
        with pytest.raises(ValueError, match="must be contiguous in all but"):
            zq._row_stride("t", bad)


def test_descales_of_a_cache():
    c = dict(_good(), k_cache=_t(8, 16, 2, 128, dtype=torch.uint8), v_cache=_t(8, 16, 2, 128, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous float32"):
        zq.attn_decode(_t(2, 4, 128), **c, k_descale=torch.ones(2, dtype=torch.float64))
    with pytest.raises(ValueError, match="descales must all hold"):
        zq.attn_decode(_t(2, 4, 128), **c, k_descale=torch.ones(2), v_descale=torch.ones(1))
    with pytest.raises(ValueError, match="descales must all hold"):
        zq.kv_append(_t(2, 2, 128), _t(2, 2, 128), **c, k_descale=torch.ones(3))


# ------------------------------------------------------------ packed prompts
def _varlen(**kw):
    a = zq.zq_varlen_args()
    d = dict(q=A, k=A, v=A, out=A, lse=None, cu_seqlens_q=A, cu_seqlens_k=A, B=2, total_q=300, total_k=300, Hq=4, Hkv=2, d_qk=128, d_v=128,
             softmax_scale=0.0, causal=1, dtype=0, q_descale=None, k_descale=None, v_descale=None, softmax_mode=zq.ZQ_SOFTMAX_LEANP,
             block_scale=1, headroom_T=8, status=None, descale_layout=0)
    for k, v in {**d, **kw}.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), zq.ZQ_ERR_NULL),
    (dict(k=None), zq.ZQ_ERR_NULL),
    (dict(v=None), zq.ZQ_ERR_NULL),
    (dict(out=None), zq.ZQ_ERR_NULL),
    (dict(cu_seqlens_q=None), zq.ZQ_ERR_NULL),
    (dict(cu_seqlens_k=None, total_q=0), zq.ZQ_ERR_NULL),
    (dict(B=0), zq.ZQ_ERR_SHAPE),
    (dict(B=65536), zq.ZQ_ERR_SHAPE),
    (dict(total_q=-1), zq.ZQ_ERR_SHAPE),
    (dict(total_k=-1), zq.ZQ_ERR_SHAPE),
    (dict(Hq=3), zq.ZQ_ERR_SHAPE),
    (dict(Hkv=0), zq.ZQ_ERR_SHAPE),
    (dict(Hq=8192), zq.ZQ_ERR_SHAPE),
    (dict(total_q=(1 << 31) - 1, Hq=4096), zq.ZQ_ERR_SHAPE),
    (dict(softmax_scale=float("inf")), zq.ZQ_ERR_SHAPE),
    (dict(d_qk=64), zq.ZQ_ERR_UNSUPPORTED),
    (dict(d_v=192), zq.ZQ_ERR_UNSUPPORTED),
    (dict(dtype=2), zq.ZQ_ERR_UNSUPPORTED),
    (dict(dtype=1, softmax_mode=2), zq.ZQ_ERR_UNSUPPORTED),
    (dict(dtype=1, block_scale=2), zq.ZQ_ERR_UNSUPPORTED),
    (dict(dtype=1, headroom_T=9), zq.ZQ_ERR_UNSUPPORTED),
    (dict(dtype=1, descale_layout=2), zq.ZQ_ERR_UNSUPPORTED),
    (dict(q=A + 8), zq.ZQ_ERR_ALIGN),
    (dict(v=A + 2), zq.ZQ_ERR_ALIGN),
    (dict(out=A + 4), zq.ZQ_ERR_ALIGN),
    (dict(lse=A + 4), zq.ZQ_ERR_ALIGN),
])
def test_varlen_argument_errors(kw, code):
    assert zq.zq_attn_varlen_fwd(_varlen(**kw), None) == code


def _cu(n):
    return torch.zeros(n, dtype=torch.int32)


@pytest.mark.parametrize("kw,err,msg", [
    (dict(q=_t(1, 8, 4, 128)), ValueError, "must be 3-D"),
    (dict(q=_t(4, 8, 128).transpose(0, 1)), ValueError, "must be contiguous"),
    (dict(k=_t(8, 2, 128, dtype=torch.uint8)), TypeError, "all be bfloat16"),
    (dict(k=_t(8, 2, 192)), ValueError, "head dim"),
    (dict(v=_t(9, 2, 128)), ValueError, "k's rows"),
    (dict(v=_t(8, 1, 128)), ValueError, "k's rows"),
    (dict(cu_seqlens_q=_cu(1), cu_seqlens_k=_cu(1)), ValueError, "B \\+ 1 offsets"),
    (dict(cu_seqlens_k=_cu(4)), ValueError, "B \\+ 1 offsets"),
    (dict(cu_seqlens_q=_cu(3).long()), ValueError, "B \\+ 1 offsets"),
    (dict(cu_seqlens_k=_cu(6)[::2]), ValueError, "B \\+ 1 offsets"),
    (dict(out=_t(8, 4, 192)), ValueError, "out must have shape"),
    (dict(lse=_t(8, 4, dtype=torch.float32)), ValueError, "lse must have shape"),
    (dict(status=_t(1)), ValueError, "status"),
    (dict(), ValueError, "must be a CUDA tensor"),
])
def test_varlen_helper_refuses(kw, err, msg):
    a = {**dict(q=_t(8, 4, 128), k=_t(8, 2, 128), v=_t(8, 2, 128), cu_seqlens_q=_cu(3), cu_seqlens_k=_cu(3)), **kw}
    with pytest.raises(err, match=msg):
        zq.attn_varlen(**a)


def test_varlen_helper_refuses_bad_descales():
    a = dict(q=_t(8, 4, 128, dtype=torch.uint8), k=_t(8, 2, 128, dtype=torch.uint8), v=_t(8, 2, 128, dtype=torch.uint8),
             cu_seqlens_q=_cu(3), cu_seqlens_k=_cu(3))
    with pytest.raises(ValueError, match="contiguous float32"):
        zq.attn_varlen(**a, q_descale=torch.ones(1, dtype=torch.float64))
    with pytest.raises(ValueError, match="descales must all hold"):
        zq.attn_varlen(**a, q_descale=torch.ones(4), k_descale=torch.ones(2))
