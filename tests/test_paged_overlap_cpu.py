"""fx_paged_append refuses memory whose rows share their bytes (addresses are never used: nothing is launched)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def fx():
    import kv_cache_token_fx_gb300 as fxm
    from kv_cache_token_fx_gb300 import build
    build.build()
    fxm.load_library()
    return fxm


def append(fx, cache=None, n=0, **rows):
    """Status of an append to a 4-bit cache of 10 pages of 32 rows of 4 heads, 16 query heads."""
    d = fx.PagedDesc(256, 512, 768, 1024, 1280, 1536, 4 * 32 * 64, 32 * 64, 64, 4 * 32 * 8, 32 * 8, 8, 5, 1, 2, 4, 128, 32,
                     10, 5, 0, 0)
    for k, v in (cache or {}).items():
        setattr(d, k, v)
    r = fx.PagedRows(256, 512, 512, 128, 1024, 2048, 512, 128, 2048, 128, 256, 256, None, 256, n, 16, 128, 9, 0)
    for k, v in rows.items():
        setattr(r, k, v)
    return fx.load_library().fx_paged_append(ctypes.byref(d), bytes(r), 0, None)


BF16 = dict(format=0, k_scale=None, v_scale=None, stride_page=4 * 32 * 128, stride_h=32 * 128, stride_t=128)


@pytest.mark.parametrize("cache", [dict(stride_page=0), dict(stride_h=0), dict(stride_t=48), dict(scale_stride_page=0),
                                   dict(scale_stride_h=0), dict(scale_stride_t=0), dict(BF16, stride_t=64),
                                   dict(BF16, stride_h=0)])
def test_pools_whose_rows_share_memory(fx, cache):
    assert append(fx, cache) == 1 and b"share memory" in fx.load_library().fx_last_error()


def test_outputs_whose_rows_share_memory(fx):
    for rows in (dict(n=3, qo_stride_n=0), dict(n=3, qo_stride_n=64), dict(qo_stride_h=0), dict(qo_stride_h=120)):
        assert append(fx, **rows) == 1 and b"share memory" in fx.load_library().fx_last_error(), rows


def test_strides_that_address_nothing_may_be_anything(fx):
    """Of a dimension of one entry; and inputs may be broadcast.  (n = 0: the checks pass, nothing is launched.)"""
    assert append(fx) == 0 and append(fx, BF16) == 0
    assert append(fx, dict(Hkv=1, stride_h=0, scale_stride_h=0), Hq=1, qo_stride_h=0, qo_stride_n=0) == 0
    assert append(fx, dict(n_pages=1, stride_page=0, scale_stride_page=0)) == 0
    assert append(fx, stride_n=0, stride_h=0, q_stride_n=0, q_stride_h=0) == 0
