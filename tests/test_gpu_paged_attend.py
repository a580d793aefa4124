"""GPU parity of fx_paged_attend against its plain 64-bit statement (attend_ref below).

Tolerances.  A logit is a sum of 128 exact products in fp32 accumulators -- at most 8 additions one after another, each
off by at most 2^-22 of what it adds to -- so it is off by less than 2^-19 of dl = |scale| sum |q_d k_d|; the cap adds
2^-20 of itself (a tanh off by at most 2^-21, and roundings), the bias by distance 2^-22 of its size: dx in all.  A weight
is off by twice that (numerator and sum), by 2^-22 of the exponential, and by its rounding for the product with V: 2^-8 of
itself in bf16, 2^-11 in f16, whose smallest step besides leaves 2^-25 on a scale where the row's largest weight is 2^6
at least: 2^-31 sum |v|.  Sums of T values in fp32, added 16 at a time to an accumulator that cuts at 2^-23 of itself,
leave T/16 2^-22.  The output is rounded to bf16: 2^-8 of itself.  So
  |out - ref| <= 2^-8 |ref| + (dp + 2 dx + 2^-20 + T 2^-26) (1 + 2^-8) sum p |v| [+ 2^-31 sum |v|],  dp = 2^-8 or 2^-11
  |lse - ref| <= dx + 2^-20 (1 + |ref|) + T 2^-26
"""
import numpy as np
import pytest
import torch

from tests import paged_ref as pr

pytestmark = pytest.mark.gpu

D = 128
FMT = ["bf16", "e2m1"]


@pytest.fixture(scope="module")
def fx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_token_fx_gb300 as fxm
    fxm.load_library()
    return fxm


@pytest.fixture(autouse=True)
def no_device_errors(fx):
    fx.fx_device_errors()
    yield
    assert fx.fx_device_errors() == 0


def cu(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).to("cuda")


def attend_ref(c, q, start, scale, first=None, last=None, window=0, cap=0.0, slope=None, skip=None):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits; rows of no sequence are NaN there.  skip(b, t): rows
    left out (bad pages)."""
    q = np.asarray(q, np.float64)
    n, Hq, _ = q.shape
    G = Hq // c.Hkv
    out, lse = np.full(q.shape, np.nan), np.full((n, Hq), np.nan)
    tol, ltol = np.zeros(q.shape), np.zeros((n, Hq))
    for b in range(c.B):
        nb = start[b + 1] - start[b]
        for j in range(nb):
            i, pos = start[b] + j, c.lens[b] - nb + j
            lo = max(0 if first is None else int(first[i]), pos - window + 1 if window else 0, 0)
            hi = min(pos + 1 if last is None else int(last[i]), c.lens[b])
            t = np.arange(lo, max(lo, hi))
            if skip is not None:
                t = t[~skip(b, t)]
            for g in range(Hq):
                if not len(t):
                    out[i, g], lse[i, g] = 0.0, -np.inf
                    continue
                k, v = c.rows(0, b, g // G, t), c.rows(1, b, g // G, t)
                with np.errstate(invalid="ignore", over="ignore"):
                    x = scale * (k @ q[i, g])
                    dx = 2.0 ** -19 * abs(scale) * (np.abs(k) @ np.abs(q[i, g])).max()
                    if cap:
                        x, dx = cap * np.tanh(x / cap), dx + cap * 2.0 ** -20
                    if slope is not None:
                        far = float(slope[g]) * np.abs(pos - t)
                        x, dx = x - far, dx + 2.0 ** -22 * np.abs(far).max()
                    m = x.max()
                    if m == -np.inf:
                        out[i, g], lse[i, g] = 0.0, -np.inf
                        continue
                    e = np.exp(x - m)
                    z = e.sum()
                    p = e / z
                    out[i, g], lse[i, g] = p @ v, m + np.log(z)
                    dp = 2.0 ** -8 if c.fmt == "bf16" else 2.0 ** -11
                    tol[i, g] = 2.0 ** -8 * np.abs(out[i, g]) + 1.004 * (dp + 2 * dx + 2.0 ** -20 + len(t) * 2.0 ** -26) * (p @ np.abs(v))
                    if c.fmt == "e2m1":
                        tol[i, g] += 2.0 ** -31 * np.abs(v).sum(0)
                    ltol[i, g] = dx + 2.0 ** -20 * (1 + abs(lse[i, g])) + len(t) * 2.0 ** -26
    return out, lse, tol + 1e-38, ltol


def check(c, got, ref, rows=slice(None)):
    out, lse = (x.double().cpu().numpy()[rows] for x in got)
    r, rl, tol, ltol = (x[rows] for x in ref)
    assert np.array_equal(lse == -np.inf, rl == -np.inf)
    assert np.all(out[rl == -np.inf] == 0)
    ok = rl != -np.inf
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(out - r) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:5], np.nanmax(np.abs(out - r) / tol))
        worst = np.abs(lse[ok] - rl[ok]) / ltol[ok]
    assert np.all(worst <= 1), worst.max()


def case(fmt, lens, news, Hkv, G, page, seed=0, layout="head", exps=(0, 0), scale=2.0, pad=2):
    c = pr.Cache(fmt, lens, Hkv, page, seed=seed, layout=layout, exps=(0, 0) if fmt == "bf16" else exps)
    g = np.random.default_rng(seed + 1)
    start = np.concatenate(([0], np.cumsum(news))).astype(np.int64)
    n = int(start[-1]) + pad
    q = pr.bf16(scale * g.standard_normal((n, Hkv * G, D)))
    return c, q, start


def intervals(kind, c, start, n, seed):
    """first, last (or None) of a kind of mask; rows of no sequence hold anything."""
    g = np.random.default_rng(seed)
    first, last = g.integers(-5, 1 << 30, n), g.integers(-(1 << 30), 5, n)
    for b in range(c.B):
        nb = start[b + 1] - start[b]
        ln = c.lens[b]
        cuts = np.unique(np.concatenate(([0, ln], g.integers(0, ln + 1, 4))))
        for j in range(nb):
            i, pos = start[b] + j, ln - nb + j
            k = np.searchsorted(cuts, max(pos, 0), side="right") - 1
            a, e = cuts[min(k, len(cuts) - 1)], cuts[min(k + 1, len(cuts) - 1)]
            if kind == "docs":
                first[i], last[i] = a, pos + 1
            elif kind == "spans":
                first[i], last[i] = 0, max(e, pos + 1)
            elif kind == "wild":   # anything, empty and reversed ones among them
                first[i], last[i] = g.integers(-3, ln + 3), g.integers(-3, ln + 3)
    return (None if kind == "spans" else first), (None if kind == "docs" else last)


CASES = [  # lens, new tokens of each, Hkv, G, page, layout, exps
    ([1], [1], 1, 1, 16, "head", (0, 0)),
    ([17, 1, 300], [1, 1, 1], 2, 4, 16, "row", (0, 0)),
    ([129, 0, 128, 65], [1, 0, 3, 7], 2, 3, 32, "gap", (-4, 3)),
    ([40, 200], [40, 200], 1, 1, 16, "head", (0, 0)),
    ([130, 257, 5], [130, 33, 5], 2, 2, 64, "row", (2, -6)),
    ([700], [300], 1, 5, 256, "head", (0, 0)),
    ([333, 64], [333, 64], 2, 8, 128, "gap", (0, 0)),
    ([600, 20], [9, 20], 1, 16, 16, "head", (0, 0)),
    ([5, 9], [12, 9], 1, 2, 16, "head", (0, 0)),     # more new tokens than rows: the first of them see nothing
    ([900], [2], 1, 64, 1024, "row", (0, 0)),
]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("lens,news,Hkv,G,page,layout,exps", CASES)
def test_attend(fx, fmt, lens, news, Hkv, G, page, layout, exps):
    c, q, start = case(fmt, lens, news, Hkv, G, page, seed=len(lens) + page + G, layout=layout, exps=exps)
    dev = c.device(fx)
    n = q.shape[0]
    t = cu(q, torch.bfloat16)
    out = torch.full((n, Hkv * G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, Hkv * G), 5.0, device="cuda")
    scale = 0.11
    got = fx.fx_paged_attend(dev, t, cu(start, torch.int32), max_new=max(news), scale=scale, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    check(c, got, attend_ref(c, q, start, scale), slice(0, start[-1]))
    assert torch.all(out[start[-1]:] == 7.0) and torch.all(lse[start[-1]:] == 5.0)


SHAPES = [  # window, cap, slope, mask
    (0, 3.0, False, None), (0, 0.0, True, None), (50, 0.0, False, None), (1, 20.0, True, None), (0, 0.0, False, "docs"),
    (0, 0.0, False, "spans"), (70, 5.0, True, "spans"), (0, 0.0, False, "wild"), (9, 2.0, True, "wild"),
]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("window,cap,slope,mask", SHAPES)
@pytest.mark.parametrize("lens,news,Hkv,G", [([300, 40], [1, 1], 2, 2), ([290, 150], [290, 60], 1, 3), ([520], [90], 2, 4)])
def test_attend_scores_and_masks(fx, fmt, window, cap, slope, mask, lens, news, Hkv, G):
    c, q, start = case(fmt, lens, news, Hkv, G, 32, seed=window + len(lens))
    n = q.shape[0]
    first, last = intervals(mask, c, start, n, 3) if mask else (None, None)
    sl = 2.0 ** -np.arange(1, Hkv * G + 1) if slope else None
    got = fx.fx_paged_attend(c.device(fx), cu(q, torch.bfloat16), cu(start, torch.int32), max_new=max(news), window=window,
                             cap=cap, slope=None if sl is None else cu(sl, torch.float32),
                             first=None if first is None else cu(first, torch.int32),
                             last=None if last is None else cu(last, torch.int32), want_lse=True)
    ref = attend_ref(c, q, start, D ** -0.5, first, last, window, cap, sl)
    check(c, got, ref, slice(0, start[-1]))


@pytest.mark.parametrize("fmt", FMT)
def test_attend_scales(fx, fmt):
    """Negative, zero and large scales, without and with a cap."""
    c, q, start = case(fmt, [200], [5], 1, 4, 16, seed=8)
    dev, t, st = c.device(fx), cu(q, torch.bfloat16), cu(start, torch.int32)
    for scale in (-0.2, 0.0, 3.0, -40.0):
        for cap in (0.0, 4.0):
            got = fx.fx_paged_attend(dev, t, st, max_new=5, scale=scale, cap=cap, want_lse=True)
            check(c, got, attend_ref(c, q, start, scale, cap=cap), slice(0, 5))
