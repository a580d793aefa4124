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


# ---------------------------------------------------------------------------------------- edges
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("lens,news", [([300, 90], [1, 1]), ([300, 90], [6, 3]), ([300, 200], [300, 130])])
def test_attend_bad_pages(fx, fmt, lens, news):
    """Rows of a bad page are left out; the bit is set."""
    c, q, start = case(fmt, lens, news, 2, 2, 16, seed=5)
    dev = c.device(fx)
    dev.table[0, 3], dev.table[1, 0], dev.table[0, 18] = 1 << 29, -2, c.n_pages
    gone = {0: (3, 18), 1: (0,)}
    got = fx.fx_paged_attend(dev, cu(q, torch.bfloat16), cu(start, torch.int32), max_new=max(news), want_lse=True)
    assert fx.fx_device_errors() == fx.FX_DEVERR_PAGE
    ref = attend_ref(c, q, start, D ** -0.5, skip=lambda b, t: np.isin(t // 16, gone[b]))
    check(c, got, ref, slice(0, start[-1]))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("G,news", [(2, [40]), (8, [40]), (1, [3]), (4, [140])])
def test_attend_values_that_are_not_finite(fx, fmt, G, news):
    """A row whose V (or K) holds an infinity or NaN reaches the queries that see it and no others."""
    n = news[0]
    c, q, start = case(fmt, [200], news, 1, G, 16, seed=9, pad=0)
    dev = c.device(fx)
    at = np.array([200 - n // 2, 37])        # seen by the late queries, and by those whose first row lies before it
    first = np.zeros(n, np.int64)
    first[n // 3:] = 40
    for what in (0, 1):
        d = c.device(fx)
        for t in at:
            pg, row = c.spot(0, t)
            if fmt == "bf16":
                (d.k, d.v)[what][pg, 0, row, 5] = float("nan") if what == 0 or t % 2 else float("inf")
            else:
                (d.k_scale, d.v_scale)[what][pg, 0, row, 3] = 0x7f
        got = fx.fx_paged_attend(d, cu(q, torch.bfloat16), cu(start, torch.int32), max_new=n, first=cu(first, torch.int32),
                                 want_lse=True)
        ref = attend_ref(c, q, start, D ** -0.5, first=first)
        pos = 200 - n + np.arange(n)
        sees = ((at[None] <= pos[:, None]) & (at[None] >= first[:, None])).any(1)
        assert sees.any() and not sees.all()
        check(c, got, ref, np.flatnonzero(~sees))
        o = got[0].float().cpu().numpy()[sees]
        assert not np.isfinite(o).all(-1).any()            # it shows in every head that sees it
        assert np.isfinite(got[1].cpu().numpy()[sees]).all() or what == 0
    check(c, fx.fx_paged_attend(dev, cu(q, torch.bfloat16), cu(start, torch.int32), max_new=n, want_lse=True),
          attend_ref(c, q, start, D ** -0.5))


def test_attend_queries_that_are_not_finite(fx):
    """Such a query's own output is NaN, its neighbours' are not."""
    for fmt in FMT:
        for n in (5, 100):
            c, q, start = case(fmt, [150], [n], 1, 2, 16, seed=2, pad=0)
            t = cu(q, torch.bfloat16)
            t[n // 2, 1, 7] = float("nan")
            t[n - 1, 0, 3] = float("inf")
            out, lse = fx.fx_paged_attend(c.device(fx), t, cu(start, torch.int32), max_new=n, want_lse=True)
            bad = np.zeros((n, 2), bool)
            bad[n // 2, 1] = bad[n - 1, 0] = True
            assert np.array_equal(np.isnan(out.float().cpu().numpy()).all(-1), bad)
            r, _, tol, _ = attend_ref(c, q, start, D ** -0.5)
            ok = ~bad
            assert np.all(np.abs(out.double().cpu().numpy() - r)[ok] <= tol[ok])


@pytest.mark.parametrize("n", [3, 90])
def test_attend_bad_offsets_and_lengths(fx, n):
    """A sequence whose offsets are not good is skipped, one with too many tokens is cut; lengths are clamped."""
    c, q, _ = case("bf16", [100, 95, 120], [n] * 3, 1, 2, 16, seed=4, pad=0)
    dev, t = c.device(fx), cu(q, torch.bfloat16)
    whole = np.array([0, n, 2 * n, 3 * n])
    ref = attend_ref(c, q, whole, D ** -0.5)
    for start, rows in (([0, n, 2 * n, 3 * n + 1], np.r_[0:2 * n]), ([-1, n, 2 * n, 3 * n], np.r_[n:3 * n]),
                        ([0, n, n - 1, n - 1], np.r_[0:n])):
        out = torch.full((3 * n, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((3 * n, 2), 7.0, device="cuda")
        fx.fx_paged_attend(dev, t, cu(start, torch.int32), max_new=n, out=out, lse=lse)
        assert fx.fx_device_errors() == fx.FX_DEVERR_OFFSETS
        check(c, (out, lse), ref, rows)
        rest = np.setdiff1d(np.arange(3 * n), rows)
        assert torch.all(out[rest] == 7.0) and torch.all(lse[rest] == 7.0)
    out = torch.full((3 * n, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3 * n, 2), 7.0, device="cuda")
    fx.fx_paged_attend(dev, t, cu(whole, torch.int32), max_new=n - 1, out=out, lse=lse)
    assert fx.fx_device_errors() == fx.FX_DEVERR_OFFSETS
    last = whole[1:] - 1
    check(c, (out, lse), ref, np.setdiff1d(np.arange(3 * n), last))
    assert torch.all(out[last] == 7.0)
    # lengths outside the cache: clamped (the largest to the whole capacity, whose pages exist for none of the rows past)
    dev.length[0] = -4
    got = fx.fx_paged_attend(dev, t, cu(whole, torch.int32), max_new=n, want_lse=True)
    assert fx.fx_device_errors() == fx.FX_DEVERR_LEN
    assert torch.all(got[0][:n] == 0) and torch.all(got[1][:n] == -float("inf"))
    check(c, got, ref, np.r_[n:3 * n])


@pytest.mark.parametrize("fmt", FMT)
def test_attend_without_start_and_strided(fx, fmt):
    """Equal numbers of tokens need no offsets; queries are views of a fused projection; no tokens at all are fine."""
    c, q, start = case(fmt, [70, 70, 33], [2, 2, 2], 2, 2, 16, seed=6, pad=0)
    dev = c.device(fx)
    qkv = torch.randn(6, 9, D, device="cuda").to(torch.bfloat16)
    qkv[:, 3:7] = cu(q, torch.bfloat16)
    check(c, fx.fx_paged_attend(dev, qkv[:, 3:7], want_lse=True), attend_ref(c, q, start, D ** -0.5))
    heads = cu(q, torch.bfloat16).transpose(0, 1).contiguous().transpose(0, 1)
    check(c, fx.fx_paged_attend(dev, heads, cu(start, torch.int32), want_lse=True), attend_ref(c, q, start, D ** -0.5))
    assert fx.fx_paged_attend(dev, qkv[:0, :4]).shape == (0, 4, D)
    for bad in (dict(max_new=3), dict(first=torch.zeros(5, dtype=torch.int32, device="cuda")),
                dict(slope=torch.ones(3, device="cuda")), dict(out=torch.zeros(6, 4, D, device="cuda")),
                dict(lse=torch.zeros(4, 6, device="cuda")), dict(start=torch.zeros(3, dtype=torch.int32, device="cuda")),
                dict(window=-1), dict(cap=-2.0), dict(scale=float("nan")), dict(window=1 << 31), dict(window=0.5),
                dict(scale=1e300), dict(cap="30")):
        with pytest.raises(fx.FxError):
            fx.fx_paged_attend(dev, heads, **bad)
    with pytest.raises(fx.FxError):
        fx.fx_paged_attend(dev, heads[:5])


def test_attend_large_values_stay_finite(fx):
    """Means of values near the type's largest are finite; the row's largest weight may come late."""
    for n in (2, 80):
        c, q, start = case("bf16", [400], [n], 1, 2, 16, seed=3, pad=0)
        c.pool[1] = np.sign(c.pool[1]) * pr.bf16(3.3e38)
        c.pool[0][c.table[0, 20]] *= 32.0       # (still bf16 values)
        got = fx.fx_paged_attend(c.device(fx), cu(q, torch.bfloat16), cu(start, torch.int32), max_new=n, want_lse=True)
        assert torch.isfinite(got[0]).all()
        check(c, got, attend_ref(c, q, start, D ** -0.5))


@pytest.mark.parametrize("new", [1, 64])
def test_attend_streams_graphs_and_workspaces(fx, new):
    """Two streams at once, two captured graphs replayed in turn with new contents, and chained programmatic launches, all
    with workspaces of the library's choice: the same bits as one call."""
    made = []
    for seed in (1, 2):
        c, q, start = case("e2m1" if seed == 1 else "bf16", [900, 500], [new, new], 1, 4, 16, seed=seed, pad=0)
        made.append((c, q, start, c.device(fx), cu(q, torch.bfloat16), cu(start, torch.int32)))
    alone = []
    for c, q, start, dev, t, st in made:
        alone.append(fx.fx_paged_attend(dev, t, st, max_new=new, want_lse=True))
        check(c, alone[-1], attend_ref(c, q, start, D ** -0.5))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    outs = [[] for _ in made]
    for _ in range(20):
        for s, o, (c, q, start, dev, t, st) in zip(streams, outs, made):
            o.append(fx.fx_paged_attend(dev, t, st, max_new=new, want_lse=True, stream=s))
    torch.cuda.synchronize()
    for o, a in zip(outs, alone):
        for x in o:
            assert torch.equal(x[0], a[0]) and torch.equal(x[1], a[1])
    graphs = []
    for c, q, start, dev, t, st in made:
        side = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            first = fx.fx_paged_attend(dev, t, st, max_new=new, want_lse=True)
            second = fx.fx_paged_attend(dev, t, st, max_new=new, want_lse=True, flags=fx.FX_LAUNCH_PDL)
        graphs.append((g, first, second))
    for turn in range(3):
        for (c, q, start, dev, t, st), (g, first, second) in zip(made, graphs):
            t.neg_()
            g.replay()
        torch.cuda.synchronize()
        for (c, q, start, dev, t, st), (g, first, second) in zip(made, graphs):
            eager = fx.fx_paged_attend(dev, t, st, max_new=new, want_lse=True)
            for got in (first, second):
                assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])


def test_attend_many_sequences_and_spare_pages(fx):
    """Batches around the scans' sizes, lengths of zero, tables with far more room than rows."""
    for B, new, G in ((33, 1, 2), (140, 2, 1), (300, 1, 1), (40, 9, 8), (200, 66, 1)):
        g = np.random.default_rng(B)
        lens = [int(x) for x in g.integers(0, 60, B)]
        news = [int(min(n, g.integers(0, new + 1))) for n in lens]
        start = np.concatenate(([0], np.cumsum(news)))
        c = pr.Cache("bf16", lens, 1, 16, seed=B, max_pages=500)
        q = pr.bf16(2.0 * g.standard_normal((max(int(start[-1]), 1), G, D)))
        got = fx.fx_paged_attend(c.device(fx), cu(q, torch.bfloat16), cu(start, torch.int32), max_new=new, want_lse=True)
        check(c, got, attend_ref(c, q, start, D ** -0.5), slice(0, start[-1]))


@pytest.mark.parametrize("fmt", FMT)
def test_attend_long_rows_in_parts(fx, fmt):
    """A chunk of few blocks over a long cache is cut into many parts; a window and documents leave some of them empty."""
    c, q, start = case(fmt, [5000, 2500], [70, 33], 1, 2, 64, seed=12, pad=0)
    dev, t, st = c.device(fx), cu(q, torch.bfloat16), cu(start, torch.int32)
    n = q.shape[0]
    first = np.zeros(n, np.int64)
    first[:40], first[70:90] = 4300, 2490
    sl = np.array([0.01, 0.0001])
    for kw in (dict(), dict(window=700), dict(first=first, cap=8.0), dict(slope=sl)):
        dk = {k: cu(v, torch.int32 if k == "first" else torch.float32) if k in ("first", "slope") else v for k, v in kw.items()}
        got = fx.fx_paged_attend(dev, t, st, max_new=70, want_lse=True, **dk)
        check(c, got, attend_ref(c, q, start, D ** -0.5, **kw))


def test_attend_far_pages_and_wide_windows(fx):
    """Pages past 2^32 bytes of the pool, for a step and for a prompt; a window as wide as an int holds."""
    pages = (5 << 30) // (16 * 256)
    k, v = (torch.empty(pages, 1, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c = pr.Cache("bf16", [150, 40], 1, 16, seed=2)
    used = np.concatenate([c.table[b, :-(-n // 16)] for b, n in enumerate(c.lens)])
    far = {int(p): pages - 1 - 7 * i for i, p in enumerate(used)}
    table = torch.full((2, c.max_pages), -1, dtype=torch.int32)
    for b, n in enumerate(c.lens):
        for j in range(-(-n // 16)):
            at = far[int(c.table[b, j])]
            table[b, j] = at
            for t, p in ((k, c.pool[0]), (v, c.pool[1])):
                t[at] = cu(p[c.table[b, j]], torch.bfloat16)
    dev = fx.PagedKV(k, v, table.cuda(), cu(c.lens, torch.int32))
    for news in ([1, 1], [150, 40], [90, 3]):
        g = np.random.default_rng(3)
        start = np.concatenate(([0], np.cumsum(news)))
        q = pr.bf16(2.0 * g.standard_normal((start[-1], 2, D)))
        for window in (0, (1 << 31) - 1):
            got = fx.fx_paged_attend(dev, cu(q, torch.bfloat16), cu(start, torch.int32), max_new=max(news), window=window,
                                     want_lse=True)
            check(c, got, attend_ref(c, q, start, D ** -0.5))
    # rows of those pages copied, and moved, where 32 bits do not reach
    ids = torch.tensor(sorted(far.values()), dtype=torch.int32, device="cuda")
    fx.fx_paged_copy(dev, ids, ids - 1)
    assert torch.equal(k[ids.long()], k[ids.long() - 1]) and torch.equal(v[ids.long()], v[ids.long() - 1])
    to = fx.PagedKV(k, v, (table - 2).clamp(min=-1).cuda(), torch.zeros(2, dtype=torch.int32, device="cuda"))
    fx.fx_paged_compact(dev, to, tail_lo=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert to.length.tolist() == c.lens
    for a, b in zip(fx.fx_paged_gather(dev, 40), fx.fx_paged_gather(to, 40)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", FMT)
def test_attend_between_steps_and_prompts(fx, fmt):
    """17 to 64 query rows of a KV head, over tables with little room and with much: either kernel may take them."""
    for lens, news, G, pages, cap in (([300, 90], [5, 5], 4, None, 0.0), ([300, 90], [5, 2], 4, 5000, 0.0), ([300, 90], [8, 8], 4, 5000, 6.0),
                                      ([200, 260], [8, 7], 8, 5000, 6.0), ([200, 260], [16, 3], 4, None, 0.0)):
        c = pr.Cache(fmt, lens, 1, 16, seed=G, max_pages=pages)
        g = np.random.default_rng(G)
        start = np.concatenate(([0], np.cumsum(news)))
        q = pr.bf16(2.0 * g.standard_normal((int(start[-1]), G, D)))
        sl = 2.0 ** -np.arange(1, G + 1)
        got = fx.fx_paged_attend(c.device(fx), cu(q, torch.bfloat16), cu(start, torch.int32), max_new=max(news), cap=cap,
                                 slope=cu(sl, torch.float32), want_lse=True)
        check(c, got, attend_ref(c, q, start, D ** -0.5, cap=cap, slope=sl))
