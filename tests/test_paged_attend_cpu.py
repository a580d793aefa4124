"""fx_paged_attend, fx_paged_append_axes, fx_paged_compact and fx_paged_copy without a GPU: argument checks of the C entry
points (every call here is refused, or has nothing to do, before any device work), the axes of rotated pairs, and the
host's tensors in the binding."""
import ctypes

import pytest
import torch

from tests.test_paged_cpu import BAD_CACHES, BF16, desc, lib  # noqa: F401


def queries(**kw):
    from kv_cache_token_fx_gb300 import PagedQueries
    q = PagedQueries(256, 512, 128, 256, None, None, None, 512, None, 6, 4, 3, 0, 1.0, 0.0)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def rows(**kw):
    from kv_cache_token_fx_gb300 import PagedRows
    r = PagedRows(256, 512, 512, 128, 1024, 2048, 512, 128, 512, 128, 256, 256, 256, 256, 3, 4, 128, 9, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


@pytest.mark.parametrize("change,status,word", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, change, status, word):  # noqa: F811
    d, good = ctypes.byref(desc(**change)), ctypes.byref(desc(table=2560, len=2816))
    for call in (lambda: lib.fx_paged_attend(d, bytes(queries()), 256, 1 << 30, 0, None),
                 lambda: lib.fx_paged_append_axes(d, bytes(rows()), bytes(64), 3, 0, None),
                 lambda: lib.fx_paged_compact(d, good, None, 0, 256, 0, None),
                 lambda: lib.fx_paged_compact(good, d, None, 0, 256, 0, None),
                 lambda: lib.fx_paged_copy(d, 256, 256, 1, 0, None)):
        assert call() == status
        assert word in lib.fx_last_error(), lib.fx_last_error()


def test_attend_refusals(lib):  # noqa: F811
    def call(cache=None, ws=256, ws_bytes=1 << 30, flags=0, **kw):
        return lib.fx_paged_attend(ctypes.byref(cache or desc()), bytes(queries(**kw)), ws, ws_bytes, flags, None)
    assert lib.fx_paged_attend(None, bytes(queries()), 256, 1 << 30, 0, None) == 1
    assert lib.fx_paged_attend(ctypes.byref(desc()), None, 256, 1 << 30, 0, None) == 1 and b"queries" in lib.fx_last_error()
    nan, inf = float("nan"), float("inf")
    for kw, status, word in ((dict(n=-1), 1, b"n and max_new"), (dict(max_new=-1), 1, b"n and max_new"), (dict(Hq=0), 1, b"Hq"),
                             (dict(Hq=5), 1, b"Hq"), (dict(Hq=260), 2, b"query rows"), (dict(start=None, n=5), 1, b"start"),
                             (dict(scale=nan), 1, b"scale"), (dict(scale=-inf), 1, b"scale"), (dict(cap=-1.0), 1, b"cap"),
                             (dict(cap=nan), 1, b"cap"), (dict(cap=inf), 1, b"cap"), (dict(cap=2.0 ** -65), 1, b"cap"),
                             (dict(window=-1), 1, b"window"), (dict(stride_n=4), 1, b"strides"),
                             (dict(stride_h=-8), 1, b"strides"), (dict(q=None), 1, b"q must"), (dict(q=264), 1, b"q must"),
                             (dict(out=None), 1, b"out must"), (dict(out=520), 1, b"out must"),
                             (dict(max_new=(1 << 30) + 1), 2, b"too many"), (dict(n=1 << 29), 2, b"too many"),
                             (dict(n=(1 << 30) + 1, Hq=4, cache=desc(Hkv=1)), 2, b"too many"),
                             (dict(max_new=1 << 25), 2, b"too many"),
                             (dict(ws=None), 3, b"workspace"), (dict(ws_bytes=64), 3, b"workspace"),
                             (dict(ws_bytes=64, max_new=300), 3, b"workspace"), (dict(flags=4), 1, b"flags")):
        assert call(**kw) == status, (kw, lib.fx_last_error())
        assert word in lib.fx_last_error(), (kw, lib.fx_last_error())
    assert call(n=0, q=None, out=None, ws=None, ws_bytes=0) == 0          # nothing to do
    assert call(max_new=0, ws=None, ws_bytes=0) == 0


def test_attend_workspace():
    import kv_cache_token_fx_gb300 as fx
    w = fx.fx_paged_attend_workspace_bytes
    assert w(4, 2, 8, 1) >= fx.fx_paged_decode_workspace_bytes(4, 2, 8, 1) > 0
    assert w(64, 8, 64, 8) >= fx.fx_paged_decode_workspace_bytes(64, 8, 64, 8)
    assert w(1, 1, 4, 100) > w(64, 8, 32, 4096) > 0       # only calls of few blocks are cut into parts
    for bad in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 2, 1, 1), (1, 1, 1, 0), (1, 1, 2, 1 << 30)):
        assert w(*bad) == 0


def test_append_axes_refusals(lib):  # noqa: F811
    def call(axis=bytes(64), n_axes=3, flags=0, **kw):
        return lib.fx_paged_append_axes(ctypes.byref(desc()), bytes(rows(**kw)), axis, n_axes, flags, None)
    for kw, status, word in ((dict(n_axes=0), 2, b"axes"), (dict(n_axes=5), 2, b"axes"), (dict(axis=None), 1, b"axes"),
                             (dict(rope_pos=None), 1, b"axes"), (dict(rot=0), 1, b"axes"),
                             (dict(axis=bytes(63) + b"\3"), 1, b"pair 63"), (dict(axis=b"\2" * 64, n_axes=2), 1, b"pair 0"),
                             (dict(rot=16), 2, b"rot"), (dict(n=-1), 1, b"n must"), (dict(flags=8), 1, b"flags")):
        assert call(**kw) == status, (kw, lib.fx_last_error())
        assert word in lib.fx_last_error(), (kw, lib.fx_last_error())
    assert call(n=0) == 0
    # the axes of pairs past rot/2 are not read
    assert call(n=0, rot=64, axis=bytes(32) + b"\xff" * 32) == 0


def test_compact_and_copy_refusals(lib):  # noqa: F811
    src, other = desc(), dict(table=2560, len=2816)

    def call(idx=None, k=0, lo=256, flags=0, dst=None, **kw):
        return lib.fx_paged_compact(ctypes.byref(src), ctypes.byref(dst or desc(**(other | kw))), idx, k, lo, flags, None)
    for kw, status, word in ((dict(len=src.len), 1, b"of its own"), (dict(lo=other["len"]), 1, b"of its own"), (dict(table=src.table), 1, b"of its own"),
                             (dict(B=1), 1, b"one format"), (dict(Hkv=1), 1, b"one format"), (dict(k_exp=1), 1, b"one format"),
                             (dict(v_exp=-1), 1, b"one format"), (dict(dst=desc(**(other | BF16))), 1, b"one format"),
                             (dict(stride_t=0), 1, b"share memory"), (dict(scale_stride_h=0), 1, b"share memory"),
                             (dict(k=-1), 1, b"k >= 0"), (dict(k=1), 1, b"k >= 0"), (dict(k=(1 << 30) + 1, idx=256), 2, b"2^30"),
                             (dict(flags=16), 1, b"flags")):
        assert call(**kw) == status, (kw, lib.fx_last_error())
        assert word in lib.fx_last_error(), (kw, lib.fx_last_error())
    assert lib.fx_paged_compact(None, ctypes.byref(src), None, 0, 256, 0, None) == 1
    assert lib.fx_paged_compact(ctypes.byref(src), None, None, 0, 256, 0, None) == 1

    def copy(s=256, d=512, n=1, flags=0, **kw):
        return lib.fx_paged_copy(ctypes.byref(desc(**kw)), s, d, n, flags, None)
    for kw, status, word in ((dict(s=None), 1, b"non-NULL"), (dict(d=None), 1, b"non-NULL"), (dict(n=-1), 1, b"n must"),
                             (dict(stride_h=0), 1, b"share memory"), (dict(flags=4), 1, b"flags")):
        assert copy(**kw) == status, kw
        assert word in lib.fx_last_error(), kw
    assert copy(n=0, s=None, d=None) == 0 and copy(n=0, len=None) == 0    # lengths are not read


def test_rope_axes():
    import kv_cache_token_fx_gb300 as fx
    assert fx.fx_rope_axes((2, 0, 3)) == bytes([0, 0, 2, 2, 2])
    assert fx.fx_rope_axes((3, 1, 2), cyclic=True) == bytes([0, 1, 2, 0, 2, 0])
    assert fx.fx_rope_axes([64]) == bytes(64)
    for bad in ((), (1, 1, 1, 1, 1), (-1, 3), (40, 25)):
        with pytest.raises(fx.FxError):
            fx.fx_rope_axes(bad)


def test_binding_refuses_hosts_tensors():
    import kv_cache_token_fx_gb300 as fx
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    ids = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: fx.fx_paged_attend(None, q), lambda: fx.fx_paged_compact(None, None),
                 lambda: fx.fx_paged_copy(None, ids, ids)):
        with pytest.raises(fx.FxError, match="cache must be a PagedKV"):
            call()
