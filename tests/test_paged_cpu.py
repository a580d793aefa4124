"""The paged-cache calls without a GPU: argument checks of the C entry points, and the plain statements that the
GPU tests compare with, held to closed forms."""
import ctypes

import numpy as np
import pytest
import torch

from tests import paged_ref as pr


@pytest.fixture(scope="module")
def lib():
    import kv_cache_token_fx_gb300 as fx
    from kv_cache_token_fx_gb300 import build
    build.build()
    return fx.load_library()


def desc(**kw):
    """A valid 4-bit cache (addresses are never used: every call here is refused before any device work)."""
    from kv_cache_token_fx_gb300 import PagedDesc
    d = PagedDesc(256, 512, 768, 1024, 1280, 1536, 4 * 32 * 64, 32 * 64, 64, 4 * 32 * 8, 32 * 8, 8, 5, 1, 2, 4, 128, 32,
                  10, 5, 0, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


BF16 = dict(format=0, k_scale=None, v_scale=None)
BAD_CACHES = [
    (dict(format=2), 1, b"format"), (dict(k=None), 1, b"non-NULL"), (dict(table=None), 1, b"non-NULL"),
    (dict(d=64), 2, b"head dim"), (dict(B=0), 1, b"B"), (dict(Hkv=0), 1, b"Hkv"), (dict(n_pages=0), 1, b"n_pages"),
    (dict(max_pages=0), 1, b"max_pages"), (dict(table_stride=4), 1, b"table_stride"), (dict(page_rows=8), 2, b"page_rows"),
    (dict(page_rows=48), 2, b"page_rows"), (dict(page_rows=2048), 2, b"page_rows"),
    (dict(n_pages=1 << 26), 2, b"rows"), (dict(max_pages=1 << 25, table_stride=1 << 25), 2, b"rows"),
    (dict(B=65536), 2, b"65535"), (dict(stride_page=1 << 31), 2, b"2^31 bytes"), (dict(scale_stride_t=1 << 32), 2, b"2^31 bytes"),
    (dict(BF16, stride_t=1 << 30), 2, b"2^31 bytes"), (dict(k=264), 1, b"aligned"), (dict(stride_t=72), 1, b"16 bytes"),
    (dict(stride_h=-64), 1, b"16 bytes"), (dict(k_scale=None), 1, b"k_scale"), (dict(v_scale=1028), 1, b"8-byte"),
    (dict(scale_stride_t=4), 1, b"8-byte"), (dict(k_exp=65), 1, b"k_exp"), (dict(v_exp=-65), 1, b"v_exp"),
    (dict(format=0), 1, b"no scales"), (dict(BF16, k_exp=1), 1, b"exponents"), (dict(BF16, stride_t=68), 1, b"16 bytes"),
]


@pytest.mark.parametrize("change,status,word", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, change, status, word):
    from kv_cache_token_fx_gb300 import PagedRows
    d = ctypes.byref(desc(**change))
    rows = PagedRows(256, 256, 512, 128)
    rows.seq, rows.pos, rows.n = 256, 256, 1
    for call in (lambda: lib.fx_paged_append(d, bytes(rows), 0, None),
                 lambda: lib.fx_paged_gather(d, None, None, 1, 256, 256, 0, None),
                 lambda: lib.fx_paged_decode(d, 256, 0, 0, 0, 4, 1, None, 0, None, 1.0, 256, None, None, 0, 0, None),
                 lambda: lib.fx_paged_importance(d, 256, 0, 0, 0, 4, 1, 256, 1.0, 0, 1, 256, 0, None)):
        assert call() == status
        assert word in lib.fx_last_error(), lib.fx_last_error()


def test_append_refusals(lib):
    from kv_cache_token_fx_gb300 import PagedRows

    def call(cache=None, flags=0, **kw):
        r = PagedRows(256, 512, 512, 128, 1024, 2048, 512, 128, 512, 128, 256, 256, None, 256, 3, 4, 128, 9, 0)
        for k, v in kw.items():
            setattr(r, k, v)
        return lib.fx_paged_append(ctypes.byref(cache or desc()), bytes(r), flags, None)
    assert lib.fx_paged_append(None, None, 0, None) == 1
    assert lib.fx_paged_append(ctypes.byref(desc()), None, 0, None) == 1 and b"rows" in lib.fx_last_error()
    for kw, status, word in ((dict(n=-1), 1, b"n must"), (dict(k=None), 1, b"non-NULL"), (dict(seq=None), 1, b"non-NULL"),
                             (dict(v=520), 1, b"aligned"), (dict(stride_n=4), 1, b"strides"),
                             (dict(q_out=None), 1, b"together"), (dict(q=None), 1, b"together"),
                             (dict(q=1032), 1, b"aligned"), (dict(Hq=0), 1, b"Hq"), (dict(qo_stride_h=12), 1, b"q strides"),
                             (dict(q_out=1024, qo_stride_n=1024), 1, b"in the place"), (dict(rot=16), 2, b"rot"),
                             (dict(rot=144), 2, b"rot"), (dict(rot=-16), 2, b"rot"), (dict(cos_sin=None), 1, b"cos_sin"),
                             (dict(cos_sin=260), 1, b"cos_sin"), (dict(n_pos=0), 1, b"n_pos"),
                             (dict(Hq=65536), 2, b"rows"), (dict(flags=4), 1, b"flags")):
        assert call(**kw) == status, kw
        assert word in lib.fx_last_error(), (kw, lib.fx_last_error())
    assert call(n=0) == 0                                   # nothing to do: nothing is launched
    assert call(cache=desc(len=None), n=0) == 0             # the append does not read lengths


def test_gather_refusals(lib):
    d = ctypes.byref(desc())
    call = lambda idx, lo, n, k, v, flags=0: lib.fx_paged_gather(d, idx, lo, n, k, v, flags, None)  # noqa: E731
    assert call(None, None, -1, 256, 256) == 1
    assert call(None, None, (1 << 30) + 1, 256, 256) == 2
    assert call(256, 256, 1, 256, 256) == 1 and b"exclude" in lib.fx_last_error()
    assert call(None, None, 1, None, 256) == 1 and call(None, None, 1, 256, 264) == 1
    assert call(None, None, 1, 256, 256, 8) == 1
    assert call(None, None, 0, 256, 256) == 0
    assert lib.fx_paged_gather(ctypes.byref(desc(len=None)), None, None, 1, 256, 256, 0, None) == 1


def test_decode_and_importance_refusals(lib):
    d = ctypes.byref(desc())
    need = lib.fx_paged_decode_workspace_bytes(2, 4, 16, 2)
    assert need > 0 and lib.fx_paged_decode_workspace_bytes(0, 4, 16, 2) == 0
    assert lib.fx_paged_decode_workspace_bytes(2, 4, 2, 1) == 0 and lib.fx_paged_decode_workspace_bytes(2, 1, 65, 1) == 0

    def dec(q=256, sb=0, sh=0, si=0, Hq=16, Mq=2, idx=None, k=0, tail=None, scale=1.0, out=256, lse=None, ws=256,
            nb=need, flags=0):
        return lib.fx_paged_decode(d, q, sb, sh, si, Hq, Mq, idx, k, tail, scale, out, lse, ws, nb, flags, None)
    for kw, status in ((dict(q=None), 1), (dict(q=264), 1), (dict(sb=4), 1), (dict(si=-8), 1), (dict(Hq=15), 1),
                       (dict(Mq=0), 1), (dict(Mq=17), 2), (dict(k=-1), 1), (dict(k=3), 1), (dict(scale=float("nan")), 1),
                       (dict(scale=float("inf")), 1), (dict(out=None), 1), (dict(out=264), 1), (dict(ws=None), 3),
                       (dict(ws=264), 3), (dict(nb=need - 1), 3), (dict(flags=16), 1),
                       (dict(idx=256, k=(1 << 30) + 1), 2)):
        assert dec(**kw) == status, (kw, lib.fx_last_error())

    def imp(lse=256, lo=0, hi=10, scores=256, scale=1.0, Mq=2, flags=0):
        return lib.fx_paged_importance(d, 256, 0, 0, 0, 16, Mq, lse, scale, lo, hi, scores, flags, None)
    for kw in (dict(lse=None), dict(scores=None), dict(lo=-1), dict(lo=11), dict(hi=5 * 32 + 1),
               dict(scale=float("inf")), dict(flags=16)):
        assert imp(**kw) == 1, kw
    assert imp(Mq=17) == 2
    assert imp(lo=10) == 0                                  # no candidates
    d = ctypes.byref(desc(B=65535, Hkv=65535))              # 4e9 heads: their tiles are not counted in 32 bits
    assert dec(Hq=65535, Mq=1) == 2 and b"tiles" in lib.fx_last_error()
    assert lib.fx_paged_importance(d, 256, 0, 0, 0, 65535, 1, 256, 1.0, 0, 1, 256, 0, None) == 2
    d = ctypes.byref(desc(B=65535, Hkv=1000, max_pages=1, page_rows=16))   # few rows, but too many starts
    assert dec(Hq=1000, Mq=1) == 2 and b"tiles" in lib.fx_last_error()
    d = ctypes.byref(desc(B=64, Hkv=64))
    assert dec(Hq=64, Mq=1, idx=256, k=1 << 29) == 2 and b"tiles" in lib.fx_last_error()


def test_binding_refuses_other_tensors():
    import kv_cache_token_fx_gb300 as fx
    k = torch.zeros(2, 1, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(fx.FxError):
        fx.PagedKV(k, k, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(fx.FxError):
        fx.fx_paged_gather("no cache", 1)


# ---------------------------------------------------------------------------------------- the plain statements
def test_e4m3_table_matches_torch():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, pr.E4M3, equal_nan=True)


def test_quantize_takes_the_nearest_value():
    g = np.random.default_rng(1)
    x = pr.bf16(g.standard_normal((50, 128)) * np.exp(3 * g.standard_normal((50, 128))))
    codes, scales = pr.quantize(x)
    y = pr.dequantize(codes, scales)
    s = np.repeat(pr.E4M3[scales], 16, -1)
    every = np.concatenate((-pr.GRID[::-1], pr.GRID))
    best = np.abs(x[..., None] - every * s[..., None]).min(-1)
    assert np.array_equal(np.abs(x - y), best)
    a = np.abs(x).reshape(50, 8, 16).max(-1) / 6
    other = np.abs(a[..., None] - pr.E4M3[1:127]).min(-1)
    assert np.array_equal(np.abs(a - pr.E4M3[scales]), other)
    # every value held is a bf16 value
    assert np.array_equal(y, pr.bf16(y))


def test_quantize_borders_and_blocks_that_are_not_finite():
    row = np.zeros(128)
    row[:16] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -2.5, -0.25, 0.5, 4, -0.0, 0.0]
    row[16:32] = 2.0 ** -12                         # below the smallest scale times 0.25: zeros
    row[32] = np.inf
    row[48] = np.nan
    row[64] = 1e5                                   # above 6 * 448: saturates
    codes, scales = pr.quantize(row)
    y = pr.dequantize(codes, scales)
    assert list(y[:16]) == [6, 4, 4, 2, 2, 1, 1, 0, -4, -4, -2, 0, 0.5, 4, 0, 0]
    assert np.all(y[16:32] == 0) and scales[1] == 1
    assert np.isnan(y[32:64]).all() and y[64] == 2688


def test_attend_closed_forms():
    c = pr.Cache("bf16", [5, 0, 20], 2, 16, seed=3)
    q = np.zeros((3, 4, 2, 128))
    out, lse, _, _, _ = pr.attend(c, q, 1.0)
    assert np.allclose(out[0, 0, 1], c.rows(1, 0, 0, range(5)).mean(0)) and np.allclose(lse[0, :, 1], np.log(5))
    assert np.allclose(out[0, 3, 0], c.rows(1, 0, 1, range(4)).mean(0))        # query 0 does not see the last row
    assert not out[1].any() and np.all(lse[1] == -np.inf)
    s, _ = pr.importance(c, q, lse, 1.0, 0, 20)
    assert np.allclose(s.sum(-1), [[4, 4], [0, 0], [4, 4]])                    # 2 heads x 2 positions
    idx = np.array([[[3, 3, -1]] * 2, [[0, 1, 2]] * 2, [[19, 2, 7]] * 2])
    out, lse, _, _, _ = pr.attend(c, q, 1.0, idx, [4, 0, 20])
    v = lambda at: c.rows(1, 0, 0, at)  # noqa: E731
    assert np.allclose(out[0, 0, 1], (2 * v(3) + v(4)) / 3) and np.allclose(out[0, 0, 0], v(3))
