"""GPU tests of the paged append with positions of several axes, of compaction and copies of pages, and of a run of them as
they are used: a prompt with pictures, its retention, forks.  What is stored or moved is bit-exact (the rotation's roundings
are part of its definition); the attention's tolerances are derived in test_gpu_paged_attend.py."""
import numpy as np
import pytest
import torch

from tests import paged_ref as pr
from tests.test_gpu_paged import FMT, bits, cu, fx, no_device_errors, storage, table_of  # noqa: F401
from tests.test_gpu_paged_attend import attend_ref, check

pytestmark = pytest.mark.gpu

D = 128


def rotate_axes(x, cs, at, axis, inter):
    """x [n, heads, 128] with pair j turned by cs[at[axis[j]]]: rounded as stated."""
    half = len(axis)
    rows = np.concatenate([np.stack([cs[at[a], k * half + j] for j, a in enumerate(axis)], 1) for k in (0, 1)], 1)
    return pr.rotate(x, rows, inter)[0]


AXES = [  # rows added per sequence, Hkv, G, page, rot, interleaved, sections, cyclic
    ([1], 1, 1, 16, 128, False, (16, 24, 24), False),
    ([3, 1, 1], 2, 2, 32, 128, False, (24, 20, 20), True),
    ([1, 2], 2, 4, 64, 64, True, (8, 12, 12), False),
    ([40, 0, 7], 1, 3, 16, 96, False, (17, 5, 26), False),
    ([300, 90], 3, 8, 128, 32, True, (5, 0, 4, 7), True),
    ([700, 500], 2, 6, 256, 128, False, (64,), False),
    ([500, 800], 2, 8, 16, 128, True, (1, 63), False),
]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("news,Hkv,G,page,rot,inter,sections,cyclic", AXES)
def test_append_axes(fx, fmt, news, Hkv, G, page, rot, inter, sections, cyclic):  # noqa: F811
    g = np.random.default_rng(rot + page)
    olds = [int(g.integers(0, 2 * page)) for _ in news]
    c = pr.Cache(fmt, [o + n for o, n in zip(olds, news)], Hkv, page, seed=page + rot, layout=("head", "row", "gap")[G % 3])
    dev = c.device(fx)
    want = storage(fx, c, dev)
    n, Hq = sum(news), G * Hkv
    seq = np.append(np.repeat(np.arange(c.B), news), -1)
    pos = np.append(np.concatenate([np.arange(o, o + m) for o, m in zip(olds, news)]), 3)
    n_pos = 777
    at = g.integers(0, n_pos, (len(sections), n + 1))
    at[:, n] = -4                                       # padding: its positions may be anything
    x = pr.bf16(g.standard_normal((n + 1, (G + 2) * Hkv, D)))
    cs = table_of(rot, n_pos)
    t = cu(x, torch.bfloat16)
    q_out = torch.full((n + 1, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    axes = fx.fx_rope_axes(sections, cyclic=cyclic)
    fx.fx_paged_append(dev, t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:], cu(seq, torch.int32), cu(pos, torch.int32), cos_sin=cu(cs),
                       rope_pos=cu(at, torch.int32), axes=axes, interleaved=inter, q=t[:, :Hq], q_out=q_out)
    r = rotate_axes(x[:n, :Hq + Hkv], cs, at[:, :n], list(axes), inter)
    assert np.array_equal(q_out[:n].double().cpu().numpy(), r[:, :Hq])
    assert torch.all(q_out[n] == 7.0)
    for i in range(n):
        pg, row = c.spot(seq[i], pos[i])
        for w, v in ((0, r[i, Hq:]), (1, x[i, Hq + Hkv:])):
            if fmt == "bf16":
                want[w][pg, :, row] = torch.from_numpy(v).to(torch.bfloat16)
            else:
                cd, sc = pr.quantize(v)
                want[w][pg, :, row], want[2 + w][pg, :, row] = torch.from_numpy(cd), torch.from_numpy(sc)
    for a, b in zip(storage(fx, c, dev), want):
        assert torch.equal(bits(a), bits(b))


def test_one_axis_is_the_plain_append(fx):  # noqa: F811
    """A single axis, and three axes at one position, give the bits of the append without axes."""
    g = np.random.default_rng(5)
    x = cu(pr.bf16(g.standard_normal((600, 12, D))), torch.bfloat16)
    at = cu(g.integers(0, 900, 600), torch.int32)
    cs = cu(table_of(128, 900))
    outs = []
    for rope, axes in ((at, None), (at[None].contiguous(), bytes(64)), (at.repeat(3, 1), fx.fx_rope_axes((20, 22, 22), True))):
        c = pr.Cache("e2m1", [600], 2, 64, seed=1)
        dev = c.device(fx)
        q = fx.fx_paged_append(dev, x[:, 8:10], x[:, 10:], torch.zeros(600, dtype=torch.int32, device="cuda"),
                               torch.arange(600, dtype=torch.int32, device="cuda"), cos_sin=cs, rope_pos=rope, axes=axes,
                               q=x[:, :8])
        outs.append([q.cpu()] + storage(fx, c, dev))
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(bits(a), bits(b))


def test_append_axes_bad_positions(fx):  # noqa: F811
    """A token with one axis outside the table is skipped, its queries included; the others are written."""
    c = pr.Cache("bf16", [4], 1, 16, seed=3)
    dev = c.device(fx)
    before = storage(fx, c, dev)
    x = cu(pr.bf16(np.random.default_rng(1).standard_normal((4, 3, D))), torch.bfloat16)
    at = torch.tensor([[0, 1, 2, 3], [5, 8, 0, 1], [0, 0, -1, 7]], dtype=torch.int32, device="cuda")
    q_out = torch.full((4, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    fx.fx_paged_append(dev, x[:, 1:2], x[:, 2:], torch.zeros(4, dtype=torch.int32, device="cuda"),
                       torch.arange(4, dtype=torch.int32, device="cuda"), cos_sin=cu(table_of(128, 8)), rope_pos=at,
                       axes=fx.fx_rope_axes((20, 22, 22)), q=x[:, :1], q_out=q_out)
    assert fx.fx_device_errors() == fx.FX_DEVERR_INDEX
    after = storage(fx, c, dev)
    pg, row = c.spot(0, np.arange(4))
    for a, b in zip(after, before):
        same = [torch.equal(bits(a[pg[i], :, row[i]]), bits(b[pg[i], :, row[i]])) for i in range(4)]
        assert same == [False, True, True, False]
    assert [bool(torch.all(q_out[i] == 7.0)) for i in range(4)] == [False, True, True, False]


# ---------------------------------------------------------------------------------------- compaction and copies
def empty_like(c, lens, page, seed, layout="head"):
    """A cache of c's format for sequences of those lengths, its pool filled with other rows."""
    return pr.Cache(c.fmt, lens, c.Hkv, page, seed=seed, layout=layout, exps=c.exps, garbage=False)


def raw_rows(parts, table, page, b, at):
    """The stored rows of a sequence's positions, every tensor of a pool."""
    at = np.asarray(at, np.int64)
    return [p[table[b, at // page], :, at % page] for p in parts]


MOVES = [  # lens, Hkv, page, page of dst, k, tails, layouts, exps
    ([50, 9], 2, 16, 16, 5, [4, 0], ("head", "head"), (0, 0)),
    ([300, 1, 0], 1, 32, 128, 0, [300, 1, 0], ("row", "gap"), (2, -3)),
    ([1000, 333], 3, 64, 16, 100, [8, 60], ("gap", "row"), (0, 0)),
    ([700], 2, 16, 1024, 700, None, ("head", "row"), (0, 0)),
    ([2000, 900, 40], 4, 256, 64, 33, [1000, 900, 0], ("head", "head"), (-1, 1)),
]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("lens,Hkv,page,to,k,tails,layouts,exps", MOVES)
def test_compact(fx, fmt, lens, Hkv, page, to, k, tails, layouts, exps):  # noqa: F811
    g = np.random.default_rng(k + page)
    c = pr.Cache(fmt, lens, Hkv, page, seed=k + page, layout=layouts[0], exps=exps if fmt == "e2m1" else (0, 0))
    idx = None
    if k:
        idx = np.stack([[g.integers(0, max(n, 1), k) for _ in range(Hkv)] for n in lens])   # any order, some twice
    lo = None if tails is None else [n - t for n, t in zip(lens, tails)]
    sizes = [k + (0 if tails is None else t) for t in (tails or [0] * len(lens))]
    o = empty_like(c, sizes, to, seed=1, layout=layouts[1])
    src, dst = c.device(fx), o.device(fx)
    dst.length.fill_(-5)
    want = storage(fx, o, dst)
    have = storage(fx, c, src)
    got = fx.fx_paged_compact(src, dst, idx=None if idx is None else cu(idx, torch.int32),
                              tail_lo=None if lo is None else cu(lo, torch.int32))
    assert got is dst and dst.length.tolist() == sizes
    for b, n in enumerate(sizes):
        for h in range(Hkv):
            at = np.concatenate((idx[b, h] if k else [], np.arange(lo[b], lens[b]) if lo is not None else [])).astype(np.int64)
            for w, p in zip(want, raw_rows(have, c.table, page, b, at)):
                i = np.arange(n)
                w[o.table[b, i // to], h, i % to] = p[:, h]
    for a, b in zip(storage(fx, o, dst), want):
        assert torch.equal(bits(a), bits(b))
    for a, b in zip(storage(fx, c, src), have):
        assert torch.equal(bits(a), bits(b))


def test_compact_within_one_pool(fx):  # noqa: F811
    """src and dst share their pool; the destination's pages hold nothing that is read."""
    c = pr.Cache("bf16", [100, 70], 2, 16, seed=2)
    dev = c.device(fx)
    free = np.setdiff1d(np.arange(c.n_pages), np.concatenate([c.table[b, :-(-n // 16)] for b, n in enumerate(c.lens)]))
    table = cu(free[:2].reshape(2, 1), torch.int32)
    length = torch.zeros(2, dtype=torch.int32, device="cuda")
    dst = fx.PagedKV(dev.k, dev.v, table, length)
    idx = np.stack([np.sort(np.random.default_rng(b).permutation(n)[:2 * 10].reshape(2, 10), 1) for b, n in enumerate(c.lens)])
    fx.fx_paged_compact(dev, dst, idx=cu(idx, torch.int32))
    assert length.tolist() == [10, 10]
    k, v = fx.fx_paged_gather(dst, 10)
    for b in range(2):
        for h in range(2):
            assert np.array_equal(k[b, h].double().cpu().numpy(), c.rows(0, b, h, idx[b, h]))
            assert np.array_equal(v[b, h].double().cpu().numpy(), c.rows(1, b, h, idx[b, h]))


def test_compact_reports_what_it_skips(fx):  # noqa: F811
    c = pr.Cache("bf16", [20, 30], 1, 16, seed=4)
    src = c.device(fx)
    o = empty_like(c, [16, 16], 16, seed=1)
    dst = o.device(fx)
    before = storage(fx, o, dst)
    idx = torch.tensor([[[3, 20, -1]], [[1, 2, 29]]], dtype=torch.int32, device="cuda")
    fx.fx_paged_compact(src, dst, idx=idx)
    assert fx.fx_device_errors() == fx.FX_DEVERR_INDEX and dst.length.tolist() == [3, 3]
    after = storage(fx, o, dst)
    have = storage(fx, c, src)
    assert torch.equal(bits(after[0][o.table[0, 0], :, 0]), bits(have[0][c.table[0, 0], :, 3]))
    for i in (1, 2):
        assert torch.equal(bits(after[0][o.table[0, 0], :, i]), bits(before[0][o.table[0, 0], :, i]))
    fx.fx_paged_compact(src, dst, tail_lo=torch.tensor([-3, 40], dtype=torch.int32, device="cuda"))
    assert fx.fx_device_errors() == fx.FX_DEVERR_LEN | fx.FX_DEVERR_CAPACITY and dst.length.tolist() == [16, 0]
    # bad pages of the source and of the destination
    for t, at in ((src, (0, 0)), (dst, (1, 0))):
        keep = int(t.table[at])
        t.table[at] = 1 << 20
        fx.fx_paged_compact(src, dst, idx=idx.clamp(0, 15))
        assert fx.fx_device_errors() == fx.FX_DEVERR_PAGE
        t.table[at] = keep


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("Hkv,page,n,layout", [(1, 16, 1, "head"), (3, 32, 5, "row"), (2, 128, 3, "gap"), (2, 1024, 2, "head"),
                                               (8, 64, 40, "row")])
def test_copy(fx, fmt, Hkv, page, n, layout):  # noqa: F811
    c = pr.Cache(fmt, [page * (2 * n + 1)], Hkv, page, seed=n, layout=layout)
    dev = c.device(fx)
    want = storage(fx, c, dev)
    pages = np.random.default_rng(n).permutation(c.n_pages)
    src, dst = pages[:n].copy(), pages[n:2 * n].copy()
    if n > 3:
        src[1], dst[2], src[3] = -1, -1, src[0]        # left out, and one page copied twice
    for a, b in zip(src, dst):
        if a >= 0 and b >= 0:
            for w in want:
                w[b] = w[a]
    fx.fx_paged_copy(dev, cu(src, torch.int32), cu(dst, torch.int32))
    for a, b in zip(storage(fx, c, dev), want):
        assert torch.equal(bits(a), bits(b))
    fx.fx_paged_copy(dev, cu([c.n_pages, 0, -2], torch.int32), cu([1, 1 << 30, 2], torch.int32))
    assert fx.fx_device_errors() == fx.FX_DEVERR_PAGE
    for a, b in zip(storage(fx, c, dev), want):
        assert torch.equal(bits(a), bits(b))


# ---------------------------------------------------------------------------------------- a run of them
@pytest.mark.parametrize("fmt", FMT)
def test_prompt_retention_and_forks(fx, fmt):  # noqa: F811
    """Two prompts with pictures are appended and attended, one more token each, then the importance of a window picks the
    rows that stay: they move to other pages, the old ones are freed, a sequence forks and both ends go on by themselves.
    Every attention is checked against the rows that the pages hold."""
    g = np.random.default_rng(7)
    Hkv, G, page, k, W = 2, 3, 16, 24, 4
    Hq = Hkv * G
    pool = fx.PagePool(64, page, max_seqs=6, max_pages=16)
    parts = [torch.zeros(64, Hkv, page, D if fmt == "bf16" else D // 2, dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8,
                         device="cuda") for _ in range(2)]
    scales = {} if fmt == "bf16" else {n: torch.zeros(64, Hkv, page, 8, dtype=torch.uint8, device="cuda")
                                       for n in ("k_scale", "v_scale")}
    axes, cs = fx.fx_rope_axes((16, 24, 24)), cu(table_of(128, 256))

    def view(seqs):
        table, length = pool.batch(seqs)
        return fx.PagedKV(*parts, table.cuda(), length.cuda(), **scales)

    class Held:   # what the pages hold, for attend_ref
        def __init__(self, cache):
            self.fmt, self.B, self.Hkv = fmt, cache.B, Hkv
            self.lens = cache.length.tolist()
            self.kv = [x.double().cpu().numpy() for x in fx.fx_paged_gather(cache, max(max(self.lens), 1))]

        def rows(self, which, b, h, at):
            return self.kv[which][b, h, at]

    def go(seqs, news, spans=None):
        """Append news[i] tokens to each sequence and attend; returns (cache, rotated queries)."""
        for s, m in zip(seqs, news):
            pair = pool.append(s, m)
            if pair:
                fx.fx_paged_copy(view(seqs), *(torch.tensor([x], dtype=torch.int32, device="cuda") for x in pair))
        cache = view(seqs)
        lens = cache.length.tolist()
        n = sum(news)
        x = cu(pr.bf16(g.standard_normal((n, Hq + 2 * Hkv, D))), torch.bfloat16)
        seq = np.repeat(np.arange(len(seqs)), news)
        pos = np.concatenate([np.arange(ln - m, ln) for ln, m in zip(lens, news)])
        q = fx.fx_paged_append(cache, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cu(seq, torch.int32), cu(pos, torch.int32), cos_sin=cs,
                               rope_pos=cu(g.integers(0, 256, (3, n)), torch.int32), axes=axes, q=x[:, :Hq])
        last = pos + 1
        for i, (b, t) in enumerate(zip(seq, pos)):
            for a, e in (spans or {}).get(b, ()):
                if a <= t < e:
                    last[i] = e
        start = np.concatenate(([0], np.cumsum(news)))
        got = fx.fx_paged_attend(cache, q, cu(start, torch.int32), max_new=max(news), last=cu(last, torch.int32), cap=20.0,
                                 want_lse=True)
        check(None, got, attend_ref(Held(cache), q.double().cpu().numpy(), start, D ** -0.5, last=last, cap=20.0))
        return cache, q

    a, b = pool.open(), pool.open()
    cache, _ = go([a, b], [150, 61], {0: [(10, 90)], 1: [(0, 61)]})
    go([a, b], [1, 1])
    cache, q = go([a, b], [W, W])
    # the window's importance picks k rows of each head; they and the window's rows move to sequences of their own
    qw = q.view(2, W, Hq, D).transpose(1, 2)
    _, lse = fx.fx_paged_decode(cache, qw, want_lse=True)
    lens = cache.length.tolist()
    cand = min(lens) - W
    idx = fx.fx_topk_select(fx.fx_paged_importance(cache, qw, lse, cand=(0, cand)).contiguous(), k)
    kept = [pool.open(), pool.open()]
    for s in kept:
        pool.append(s, k + W)
    dst = view(kept)
    fx.fx_paged_compact(cache, dst, idx=idx, tail_lo=cu([n - W for n in lens], torch.int32))
    assert dst.length.tolist() == [k + W, k + W] == [pool.length(s) for s in kept]
    old, new = fx.fx_paged_gather(cache, max(lens)), fx.fx_paged_gather(dst, k + W)
    for x, y in zip(old, new):
        for i in range(2):
            for h in range(Hkv):
                at = torch.cat((idx[i, h].long(), torch.arange(lens[i] - W, lens[i], device="cuda")))
                assert torch.equal(x[i, h, at], y[i, h])
    free = pool.free_pages()
    assert pool.release(a) + pool.release(b) == pool.free_pages() - free > 0
    go(kept, [1, 3])
    f = pool.fork(kept[0])
    go([kept[0], f, kept[1]], [2, 5, 1])        # the fork's shared page is copied before its rows are written
    go([f, kept[0]], [1, 1])
    for s in kept + [f]:
        pool.release(s)
    assert pool.free_pages() == 64
