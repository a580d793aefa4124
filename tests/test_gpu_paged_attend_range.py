"""GPU tests of fx_paged_attend at the ends of the ranges that its arguments may take, against its plain 64-bit statement
(attend_ref in test_gpu_paged_attend.py, which derives the tolerances unless a test here derives its own)."""
import numpy as np
import pytest
import torch

from tests import paged_ref as pr
from tests.test_gpu_paged_attend import FMT, attend_ref, check, cu, fx, no_device_errors  # noqa: F401

pytestmark = pytest.mark.gpu

D = 128
LOWEST, HIGHEST = -(1 << 31), (1 << 31) - 1


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("lens,news,G,pages", [
    ([700], [3], 4, 16384),            # a step's kernel; table room for more than half a million rows: tiles in pairs
    ([700, 290], [3, 1], 2, None),     # and one at a time
    ([500], [40], 3, None),            # prompts, cut along the cache
    ([300] * 76, [17] * 76, 4, None),  # and whole
])
def test_attend_interval_ends(fx, fmt, lens, news, G, pages):  # noqa: F811
    """first and last may hold any int: a token that either leaves without rows sees none, whatever its neighbours see."""
    Hkv = 1 if len(lens) < 76 else 2
    c = pr.Cache(fmt, lens, Hkv, 32, seed=len(lens), max_pages=pages)
    g = np.random.default_rng(4)
    start = np.concatenate(([0], np.cumsum(news)))
    n = int(start[-1])
    q = pr.bf16(2.0 * g.standard_normal((n, Hkv * G, D)))
    dev, t, st = c.device(fx), cu(q, torch.bfloat16), cu(start, torch.int32)
    ends = np.array([LOWEST, LOWEST + 1, LOWEST + 40, -(1 << 30), -1])
    for kind in ("last", "last after first", "first", "both"):
        first, last = np.full(n, 70, np.int64), np.concatenate([ln - m + 1 + np.arange(m) for ln, m in zip(lens, news)])
        hit = np.arange(n) % 3 == 1
        some = ends[np.arange(n) % 5]
        if kind.startswith("last"):
            last[hit] = some[hit]
        elif kind == "first":
            first[hit] = -1 - some[hit]              # HIGHEST and what lies below it; 0 for the last
        else:
            first[hit], last[hit] = some[hit], HIGHEST - np.arange(n)[hit] % 50     # all rows
        if kind == "last":
            first[:] = 0
        got = fx.fx_paged_attend(dev, t, st, max_new=max(news), first=cu(first, torch.int32), last=cu(last, torch.int32),
                                 want_lse=True)
        check(c, got, attend_ref(c, q, start, D ** -0.5, first, last), slice(0, n))


def tight_ref(c, q, start, scale, cap=0.0, slope=None, mixed=False):
    """attend_ref over the rows up to each token, with tolerances that follow each logit's own error.

    The products of a logit x leave 2^-19 of |scale| sum |q_d k_d| (test_gpu_paged_attend.py).  Under the cap, cap tanh(x / cap)
    has a slope of at most 1 for that, and four products (scale, 1 / cap, cap, log2 e) and a tanh off by 2^-21.5 of itself at
    most (a polynomial off by 2^-22; past 1, exp off by 2^-22 of itself and 2^-24 of its argument, whose quotient is below 1/4 of
    1 - 2 / (exp + 1)) leave 2^-20 of the capped logit.  mixed: kernels that may take the second form below 1 too, for caps up
    to 64: 2^-21 of the cap.  A bias leaves 2^-22 of itself.  A weight p is then off by p (dx + sum p dx) and its rounding.
    """
    n, Hq, _ = q.shape
    G = Hq // c.Hkv
    out, lse = np.zeros(q.shape), np.zeros((n, Hq))
    tol, ltol = np.zeros(q.shape), np.zeros((n, Hq))
    for b in range(c.B):
        nb = start[b + 1] - start[b]
        for j in range(nb):
            i, pos = start[b] + j, c.lens[b] - nb + j
            t = np.arange(pos + 1)
            for g in range(Hq):
                k, v = c.rows(0, b, g // G, t), c.rows(1, b, g // G, t)
                x = scale * (k @ q[i, g])
                dx = 2.0 ** -19 * abs(scale) * (np.abs(k) @ np.abs(q[i, g]))
                if cap:
                    x = cap * np.tanh(x / cap)
                    dx = dx + 2.0 ** -20 * np.abs(x) + (2.0 ** -21 * cap if mixed and cap <= 64 else 0.0)
                if slope is not None:
                    far = slope[g] * np.abs(pos - t)
                    x, dx = x - far, dx + 2.0 ** -22 * (np.abs(far) + np.abs(x))
                m = x.max()
                p = np.exp(x - m)
                z = p.sum()
                p /= z
                out[i, g], lse[i, g] = p @ v, m + np.log(z)
                mean = p @ dx
                dp = (2.0 ** -8 if c.fmt == "bf16" else 2.0 ** -11) + 2.0 ** -20 + len(t) * 2.0 ** -26
                tol[i, g] = 2.0 ** -8 * np.abs(out[i, g]) + 1.004 * ((p * (dp + dx + mean)) @ np.abs(v))
                if c.fmt == "e2m1":
                    tol[i, g] += 2.0 ** -31 * np.abs(v).sum(0)
                ltol[i, g] = mean + 2.0 ** -20 * (1 + abs(lse[i, g])) + len(t) * 2.0 ** -26
    return out, lse, tol + 1e-38, ltol


CAPS = [50.0, 1000.0, 1e5, 1e6, 2.0 ** 30, 2.0 ** 64]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("lens,news,G", [([300, 90], [4, 1], 3), ([300, 90], [100, 35], 2)])
def test_attend_caps_of_any_size(fx, fmt, cap, lens, news, G):  # noqa: F811
    """Ordinary logits under caps of any size keep their fp32 bits, in steps and in prompts, also beside a query whose logits
    lie past the cap."""
    c = pr.Cache(fmt, lens, 1, 32, seed=G)
    g = np.random.default_rng(7)
    start = np.concatenate(([0], np.cumsum(news)))
    n = int(start[-1])
    q = pr.bf16(4.0 * g.standard_normal((n, G, D)))
    q[1, 0] = pr.bf16(np.clip(cap, 1e3, 2.0 ** 64) * q[1, 0])
    rest = np.ones((n, G), bool)
    rest[1, 0] = False
    sl = np.full(G, 2.0 ** -7)
    dev, t, st = c.device(fx), cu(q, torch.bfloat16), cu(start, torch.int32)
    mixed = max(news) * G > 64
    for slope in (None, sl):
        got = fx.fx_paged_attend(dev, t, st, max_new=max(news), cap=cap, want_lse=True,
                                 slope=None if slope is None else cu(slope, torch.float32))
        out, lse = (x.double().cpu().numpy() for x in got)
        assert np.isfinite(out).all() and np.isfinite(lse).all()
        q1 = q.copy()
        q1[1, 0] = 0.0                               # (not compared)
        r, rl, tol, ltol = tight_ref(c, q1, start, D ** -0.5, cap, slope, mixed)
        assert np.all((np.abs(lse - rl) <= ltol)[rest]), (np.abs(lse - rl) / ltol)[rest].max()
        assert np.all((np.abs(out - r) <= tol)[rest]), (np.abs(out - r) / tol)[rest].max()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("G,n", [(2, 2), (4, 4), (2, 90)])
def test_attend_scales_far_from_caps(fx, fmt, G, n):  # noqa: F811
    """Scales whose quotient by the cap leaves the range of fp32: ordinary logits, and queries of zeros under them.  (Queries
    stay below 2^122 and the magnitudes of a logit's products below 2^127 in all, so that fp32 holds the sums.)"""
    c = pr.Cache(fmt, [200], 1, 32, seed=G)
    g = np.random.default_rng(9)
    start = np.array([0, n])
    dev, st = c.device(fx), cu(start, torch.int32)
    q = pr.bf16(4.0 * g.standard_normal((n, G, D)))
    q[n // 2] = 0.0
    for e, cap in ((-80, 2.0 ** 64), (-100, 2.0 ** 30), (-118, 60.0), (100, 2.0 ** -60), (70, 2.0 ** -64)):
        scale, q1 = 2.0 ** (e - 3), q * 2.0 ** -e
        got = fx.fx_paged_attend(dev, cu(q1, torch.bfloat16), st, max_new=n, scale=scale, cap=cap, want_lse=True)
        out, lse = (x.double().cpu().numpy() for x in got)
        r, rl, tol, ltol = tight_ref(c, q1, start, scale, cap, None, n * G > 64)
        assert np.all(np.abs(lse - rl) <= ltol), (e, cap, np.abs(lse - rl).max())
        assert np.all(np.abs(out - r) <= tol), (e, cap)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("n,G", [(1, 4), (5, 3), (90, 2)])
def test_attend_bias_far_into_a_cache(fx, fmt, n, G):  # noqa: F811
    """Distances of near rows are exact where positions are past 2^24, as at the start of a cache."""
    ahead = 1024 * 20001                                     # rows before the ones that are seen; fp32 holds every second
    c = pr.Cache(fmt, [300], 2, 1024, seed=n)
    g = np.random.default_rng(n)
    q = cu(pr.bf16(2.0 * g.standard_normal((n, 2 * G, D))), torch.bfloat16)
    sl = cu(2.0 ** (1 - np.arange(2 * G)), torch.float32)
    near = c.device(fx)
    table = torch.full((1, ahead // 1024 + 1), -7, dtype=torch.int32, device="cuda")
    table[:, ahead // 1024:] = near.table[:, :1]
    far = fx.PagedKV(near.k, near.v, table, near.length + ahead, k_scale=near.k_scale, v_scale=near.v_scale)
    start = np.array([0, n])
    for cap in (0.0, 20.0):
        kw = dict(max_new=n, slope=sl, cap=cap, want_lse=True)
        got = fx.fx_paged_attend(far, q, cu(start, torch.int32), first=torch.full((n,), ahead, dtype=torch.int32, device="cuda"), **kw)
        ref = attend_ref(c, q.double().cpu().numpy(), start, D ** -0.5, cap=cap, slope=sl.double().cpu().numpy())
        check(c, got, ref)
        check(c, fx.fx_paged_attend(near, q, cu(start, torch.int32), **kw), ref)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("lens,news", [([300, 90], [4, 1]), ([400, 90], [200, 80]),
                                       ([399, 90], [200, 80])])    # (a warp's first token sees itself as a tile's last key)
def test_attend_steep_biases(fx, fmt, lens, news):  # noqa: F811
    """A bias of any slope leaves the logits of near rows their fp32 bits."""
    G = 4
    c = pr.Cache(fmt, lens, 1, 32, seed=len(lens))
    g = np.random.default_rng(11)
    start = np.concatenate(([0], np.cumsum(news)))
    q = pr.bf16(2.0 * g.standard_normal((int(start[-1]), G, D)))
    for slopes in ([0.5, 0.0, 1.3, -0.02], [2.0, 30.0, 1000.0, 3e4], [-1.0, 1e6, 2.0 ** 20, 1.0]):
        sl = np.float32(slopes).astype(np.float64)
        got = fx.fx_paged_attend(c.device(fx), cu(q, torch.bfloat16), cu(start, torch.int32), max_new=max(news),
                                 slope=cu(sl, torch.float32), want_lse=True)
        out, lse = (x.double().cpu().numpy() for x in got)
        r, rl, tol, ltol = tight_ref(c, q, start, D ** -0.5, 0.0, sl)
        assert np.all(np.abs(lse - rl) <= ltol), (slopes, (np.abs(lse - rl) / ltol).max())
        assert np.all(np.abs(out - r) <= tol), (slopes, (np.abs(out - r) / tol).max())


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("n", [1, 70])
def test_attend_only_rows_far_away(fx, fmt, n):  # noqa: F811
    """Tokens that see nothing but rows millions of positions before them, with a bias: fp32 holds those logits to 2^-24 of
    themselves only, but the weights stay weights.  (n = 70: 140 query rows, of a prompt's kernel.)"""
    c = pr.Cache(fmt, [300], 1, 1024, seed=n)
    g = np.random.default_rng(n)
    near = c.device(fx)
    q = cu(pr.bf16(2.0 * g.standard_normal((n, 2, D))), torch.bfloat16)
    last = torch.full((n,), 300, dtype=torch.int32, device="cuda")
    start = cu(np.array([0, n]), torch.int32)
    v = c.rows(1, 0, 0, np.arange(300))
    for ahead in (1 << 22, 1 << 25, 1 << 27, 1 << 29):
        table = torch.full((1, ahead // 1024 + 1), -7, dtype=torch.int32, device="cuda")
        table[0, 0] = near.table[0, 0]
        far = fx.PagedKV(near.k, near.v, table, torch.tensor([ahead + 300], dtype=torch.int32, device="cuda"),
                         k_scale=near.k_scale, v_scale=near.v_scale)
        for slope in (0.7, 1.3):
            sl = torch.full((2,), slope, device="cuda")
            out, lse = fx.fx_paged_attend(far, q, start, max_new=n, last=last, slope=sl, want_lse=True)
            out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
            assert np.isfinite(out).all() and np.isfinite(lse).all()
            assert np.all(out <= v.max(0) + 0.01 * abs(v.max(0))) and np.all(out >= v.min(0) - 0.01 * abs(v.min(0)))
            assert np.all(np.abs(lse / -(slope * ahead) - 1) < 0.001)


@pytest.mark.parametrize("fmt,G,new", [("bf16", 4, 4), ("e2m1", 8, 1), ("bf16", 1, 1)])
def test_attend_steps_over_tables_with_room_for_billions(fx, fmt, G, new):  # noqa: F811
    """Steps whose tables have more room than the decode's kernels count tiles of: the prompts' kernel takes them."""
    B, Hkv, few = 2048, 8, 8
    pages = 1024 * (2 if G == 1 else 1)                  # of 1024 rows: 2^20 rows of room a sequence
    g = np.random.default_rng(G)
    lens = [int(x) for x in g.integers(new, 80, few)]
    c = pr.Cache(fmt, lens, Hkv, 1024, seed=G)
    dev = c.device(fx)
    table = torch.full((B, pages), -7, dtype=torch.int32, device="cuda")
    table[:, 0] = dev.table[:, 0].repeat(B // few)
    big = fx.PagedKV(dev.k, dev.v, table, dev.length.repeat(B // few), k_scale=dev.k_scale, v_scale=dev.v_scale)
    assert B * Hkv * (G * new // 4 + 1) * (pages * 64 + 34) >= 1 << 31
    q = pr.bf16(2.0 * g.standard_normal((few * new, Hkv * G, D)))
    t = cu(q, torch.bfloat16)
    out, lse = fx.fx_paged_attend(big, t.repeat(B // few, 1, 1), want_lse=True)
    out, lse = out.view(B // few, few * new, -1, D), lse.view(B // few, few * new, -1)
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    check(c, (out[0], lse[0]), attend_ref(c, q, np.arange(few + 1) * new, D ** -0.5))


def test_attend_one_workspace_for_prompt_chunks_and_steps(fx):  # noqa: F811
    """Scratch memory sized once, for the longest prompt, serves every shorter call of the same sequences (through the C entry
    point, which grows nothing)."""
    c = pr.Cache("bf16", [700], 2, 32, seed=1)
    dev, G = c.device(fx), 4
    g = np.random.default_rng(1)
    lib = fx.load_library()
    nbytes = fx.fx_paged_attend_workspace_bytes(1, 2, 2 * G, 8191)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    for n in (700, 1, 100, 4, 16, 65, 300):
        q = pr.bf16(2.0 * g.standard_normal((n, 2 * G, D)))
        t = cu(q, torch.bfloat16)
        out, lse = torch.zeros(n, 2 * G, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 2 * G, device="cuda")
        qs = fx.PagedQueries(t.data_ptr(), 2 * G * D, D, None, None, None, None, out.data_ptr(), lse.data_ptr(), n, 2 * G, n, 0,
                             D ** -0.5, 0.0)
        assert lib.fx_paged_attend(dev._ref, bytes(qs), ws.data_ptr(), nbytes, 0, None) == 0, lib.fx_last_error()
        check(c, (out, lse), attend_ref(c, q, np.array([0, n]), D ** -0.5))


def test_compact_lengths_between_the_rows_of_a_table(fx):  # noqa: F811
    """Lengths may lie in the room between a table's rows: nothing that is read is written."""
    c = pr.Cache("bf16", [50, 33], 1, 16, seed=3)
    src = c.device(fx)
    room = torch.full((2, 16), -1, dtype=torch.int32, device="cuda")
    room[:, :4] = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    k, v = (torch.zeros(8, 1, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dst = fx.PagedKV(k, v, room[:, :4], room.view(-1)[6:8])
    fx.fx_paged_compact(src, dst, tail_lo=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert dst.length.tolist() == c.lens
    for a, b in zip(fx.fx_paged_gather(src, 33), fx.fx_paged_gather(dst, 33)):
        assert torch.equal(a, b)


def shared_pages(fx, fmt, T, Hkv, B=1, positive=False, pages=32):  # noqa: F811
    """A cache of B sequences of T rows whose tables name a few pages of 1024 rows over and over: (cache, K and V of those pages in
    64 bits [pages, Hkv, 1024, 128])."""
    g = torch.Generator(device="cuda").manual_seed(T)
    shape = (pages, Hkv, 1024)
    if fmt == "bf16":
        k, v = (torch.randn(*shape, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        v = v.abs() + 1 if positive else v
        kw, vals = {}, [k.double(), v.double()]
    else:
        k, v = (torch.randint(0, 256, (*shape, D // 2), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
        v = v & 0x77 if positive else v
        kw = {n: torch.randint(0x30, 0x38, (*shape, 8), generator=g, device="cuda", dtype=torch.uint8) for n in ("k_scale", "v_scale")}
        grid = torch.tensor(np.concatenate((pr.GRID, -pr.GRID)), device="cuda")
        vals = [(grid[torch.stack((x & 15, x >> 4), -1).flatten(-2).long()].unflatten(-1, (8, 16)) *
                 kw[n].view(torch.float8_e4m3fn).double()[..., None]).flatten(-2) for x, n in ((k, "k_scale"), (v, "v_scale"))]
    table = (torch.arange(T // 1024, device="cuda") * 7 % pages).to(torch.int32).expand(B, -1).contiguous()
    return fx.PagedKV(k, v, table, torch.full((B,), T, dtype=torch.int32, device="cuda"), **kw), vals


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T,n", [(1 << 20, 160), (1 << 22, 160), (1 << 22, 16)])
def test_attend_sums_over_long_rows(fx, fmt, T, n):  # noqa: F811
    """Equal weights over millions of rows of values of one sign: no part of the sum is lost.

    64 query rows a token: 160 blocks, one to a CTA, or 16, cut along the cache.  Equal weights are powers of two, and so are the
    sums of their pages: nothing is rounded there.  O's sum in the tensor core loses up to 2^-23 of itself with each of 2^17 / 16
    products before it leaves for memory, 2^-10 in all; the sums there 2^-24 with each of T / 2^17 (2^-19 at most); the output is
    rounded by 2^-8."""
    G = 64
    cache, (k, v) = shared_pages(fx, fmt, T, 4, positive=True)
    q = torch.zeros(n, 4 * G, D, dtype=torch.bfloat16, device="cuda")
    out, lse = fx.fx_paged_attend(cache, q, last=torch.full((n,), T, dtype=torch.int32, device="cuda"), want_lse=True)
    want = v[cache.table[0].long()[:32]].mean((0, 2))          # (every page comes up as often)
    off = out.double().view(n, 4, G, D) / want[None, :, None] - 1
    assert float(off.abs().max()) <= 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -19, float(off.abs().max())
    assert float((lse.double() - np.log(T)).abs().max()) <= 2.0 ** -16


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("B,kw", [(160, {}), (160, dict(slope=True)), (160, dict(cap=5.0)), (160, dict(window=100000)),
                                  (160, dict(window=200000)), (3, dict(slope=True)), (1, {}), (1, dict(window=140000, cap=5.0))])
def test_attend_rows_past_a_flush(fx, fmt, B, kw):  # noqa: F811
    """More rows than O's sums stay in the tensor core for, with references that move between: against 64 bits."""
    T, G, n = 300 * 1024, 4, 17
    cache, (k, v) = shared_pages(fx, fmt, T, 1, B=B)
    g = torch.Generator(device="cuda").manual_seed(B)
    q = torch.randn(B * n, G, D, generator=g, device="cuda").mul_(2).to(torch.bfloat16)
    slope = torch.tensor([3e-5, -1e-4, 2e-3, 0.0], device="cuda") if kw.get("slope") else None
    first = torch.zeros(B * n, dtype=torch.int32, device="cuda")
    first[3::n], first[5::n] = 250000, T                        # one that sees the end only, one nothing
    args = dict(max_new=n, first=first, slope=slope, window=kw.get("window", 0), cap=kw.get("cap", 0.0), want_lse=True)
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    out, lse = fx.fx_paged_attend(cache, q, start, **args)
    again = fx.fx_paged_attend(cache, q, start, **args)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    at = cache.table[0].long()
    kk, vv = k[at, 0].flatten(0, 1), v[at, 0].flatten(0, 1)
    t = torch.arange(T, device="cuda")
    for b in sorted({0, B // 2, B - 1}):
        for i in range(n):
            pos, row = T - n + i, b * n + i
            x = D ** -0.5 * q[row].double() @ kk.T
            dx = 2.0 ** -19 * D ** -0.5 * q[row].double().abs() @ kk.T.abs()
            if args["cap"]:
                x = args["cap"] * torch.tanh(x / args["cap"])
                dx = dx + 2.0 ** -20 * args["cap"]
            if slope is not None:
                far = slope.double()[:, None] * (pos - t).abs()
                x, dx = x - far, dx + 2.0 ** -22 * (far.abs() + x.abs())
            hidden = (t < first[row]) | (t > pos) | ((t <= pos - args["window"]) if args["window"] else False)
            x = x.masked_fill(hidden, -np.inf)
            z = torch.logsumexp(x, -1)
            if first[row] == T:
                assert torch.all(out[row] == 0) and torch.all(lse[row] == -np.inf)
                continue
            p = torch.exp(x - z[:, None])
            mean = (p * dx).sum(-1, keepdim=True)
            dp = (2.0 ** -8 if fmt == "bf16" else 2.0 ** -11) + 2.0 ** -20 + 2.0 ** -10     # (2^-10: the sums' part, as above)
            ref = p @ vv
            tol = 2.0 ** -8 * ref.abs() + 1.004 * (p * (dp + dx + mean)) @ vv.abs() + 2.0 ** -31 * vv.abs().sum(0)
            assert torch.all((out[row].double() - ref).abs() <= tol), (b, i, float(((out[row].double() - ref).abs() / tol).max()))
            assert torch.all((lse[row].double() - z).abs() <= mean[:, 0] + 2.0 ** -20 * (1 + z.abs()) + T / 128 * 2.0 ** -24)


def test_attend_long_rows_at_once(fx):  # noqa: F811
    """Calls over long rows on two streams at the same time, one after the other as programmatic launches, and in two graphs:
    the bits of a call alone (sums in memory lie in each call's own scratch)."""
    made = []
    for seed, fmt in enumerate(FMT):
        cache, _ = shared_pages(fx, fmt, 150 * 1024, 2, B=90)
        g = torch.Generator(device="cuda").manual_seed(seed)
        made.append((cache, torch.randn(90 * 20, 8, D, generator=g, device="cuda").mul_(2).to(torch.bfloat16)))
    alone = [fx.fx_paged_attend(c, q, want_lse=True) for c, q in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    outs = [[], []]
    for _ in range(3):
        for s, o, (c, q) in zip(streams, outs, made):
            o.append(fx.fx_paged_attend(c, q, want_lse=True, stream=s))
            o.append(fx.fx_paged_attend(c, q, want_lse=True, stream=s, flags=fx.FX_LAUNCH_PDL))
    torch.cuda.synchronize()
    graphs = []
    for c, q in made:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            got = fx.fx_paged_attend(c, q, want_lse=True)
        graphs.append((g, got))
    for _ in range(2):
        for s, (g, got) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, (g, got), a in zip(outs, graphs, alone):
        for x in o + [got]:
            assert torch.equal(x[0], a[0]) and torch.equal(x[1], a[1])
