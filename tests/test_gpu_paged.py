"""GPU parity of the paged-cache calls against their plain 64-bit statements (tests/paged_ref.py).

Tolerances.  Stored rows, gathered rows and rotated queries: bit-exact (the rotation's roundings are part of its
definition; the 4-bit rounding is exact arithmetic).  Attention: every product is exact, a logit is a sum of 128
products in fp32 accumulators -- at most 8 additions one after another, each off by at most 2^-22 of what it adds
to -- so it is off by less than 2^-19 of dl = scale * sum |q_d k_d|; p by that (twice: numerator and sum), by its
split into two 16-bit parts (at most 2^-16) and by 2^-22 of the exponential, and fp32 sums of at most 2^12 values
add less than 2^-17: |out - ref| <= (2 * 2^-19 dl + 2^-15) * sum p |v|.  Besides, 4-bit rows multiply weights that
are f16: their smallest step is 2^-24, so the two parts leave a weight at most 2^-25 off, on a scale where the row's
largest is at least 2^11 -- 2^-36 of the largest weight, and the weights' sum is at least that one: + 2^-36 sum |v|.
(It shows where the rows that carry the weight hold zeros in some dimension.)  lse: 2^-19 dl + 2^-20 (1 + |lse|).
Importance: 2^-19 (dl + 1) of itself, with |lse| counted into dl.
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


def queries(c, G, Mq, seed, scale=2.0, layout="head"):
    g = np.random.default_rng(seed)
    q = pr.bf16(scale * g.standard_normal((c.B, c.Hkv * G, Mq, D)))
    t = torch.from_numpy(q).to(torch.bfloat16).to("cuda")
    if layout == "token":
        t = t.transpose(1, 2).contiguous().transpose(1, 2)
    return q, t


def bits(t):
    return t.cpu().view(torch.int16 if t.dtype == torch.bfloat16 else t.dtype)


def check_out(out, lse, ref, what=""):
    r, rl, mag, dl, far = ref
    o = out.double().cpu().numpy()
    tol = (2 * 2.0 ** -19 * dl[..., None] + 2.0 ** -15) * mag + 2.0 ** -36 * far + 1e-30
    assert np.all(np.abs(o - r) <= tol), (what, np.max(np.abs(o - r) / tol))
    if lse is not None:
        z = lse.double().cpu().numpy()
        assert np.array_equal(z == -np.inf, rl == -np.inf), what
        ok = rl != -np.inf
        assert np.all(np.abs(z[ok] - rl[ok]) <= (2.0 ** -19 * dl + 2.0 ** -20 * (1 + np.abs(np.where(ok, rl, 0))))[ok]), what


# ---------------------------------------------------------------------------------------- append and gather
def table_of(rot, n_pos, base=10000.0):
    half = rot // 2
    f = base ** (-np.arange(half) / half)
    a = np.arange(n_pos)[:, None] * f
    return np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)


def storage(fx, c, dev):
    """Pool tensors on the host: k, v[, k_scale, v_scale]."""
    ts = [dev.k, dev.v] + ([dev.k_scale, dev.v_scale] if c.fmt == "e2m1" else [])
    return [t.cpu().contiguous() for t in ts]


APPEND = [  # rows added per sequence, Hkv, G, page, rot, interleaved, layout, exps, separate rotation positions
    ([1, 1, 1], 1, 1, 16, 0, False, "head", (0, 0), False),
    ([1], 8, 4, 64, 128, False, "row", (0, 0), False),
    ([1, 0, 1, 1, 1], 2, 3, 32, 128, True, "gap", (0, 0), True),
    ([37, 5, 16, 0, 1], 3, 2, 16, 96, False, "head", (-3, 2), False),
    ([130, 63], 2, 8, 128, 64, True, "row", (5, -9), True),
    ([19, 300], 1, 5, 256, 32, False, "gap", (0, 0), False),
    ([3, 700], 2, 5, 256, 96, True, "head", (0, 0), False),
    ([900, 1], 5, 1, 64, 128, False, "row", (2, -2), False),
    ([40], 2, 1, 1024, 32, True, "head", (0, 64), False),
]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("news,Hkv,G,page,rot,inter,layout,exps,apart", APPEND)
def test_append_matches_its_definition(fx, fmt, news, Hkv, G, page, rot, inter, layout, exps, apart):
    if fmt == "bf16":
        exps = (0, 0)
    g = np.random.default_rng(rot + page)
    olds = [int(g.integers(0, 3 * page)) for _ in news]
    c = pr.Cache(fmt, [o + n for o, n in zip(olds, news)], Hkv, page, seed=page + rot, layout=layout, exps=exps)
    dev = c.device(fx)
    before = storage(fx, c, dev)
    n = sum(news)
    seq = np.repeat(np.arange(c.B), news)
    pos = np.concatenate([np.arange(o, o + m) for o, m in zip(olds, news)])
    order = g.permutation(n)                       # tokens in any order, padding after them
    seq, pos = np.append(seq[order], [-1, -1]), np.append(pos[order], [5, -9])
    at = g.integers(0, 700, n + 2) if apart else np.maximum(pos, 0)
    qkv = pr.bf16(g.standard_normal((n + 2, (G + 2) * Hkv, D)) * np.exp(g.standard_normal((n + 2, (G + 2) * Hkv, 1))))
    Hq = G * Hkv
    cs = table_of(rot, 1100 + 3 * page) if rot else None
    t = cu(qkv, torch.bfloat16)
    q_out = torch.full((n + 2, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = fx.fx_paged_append(dev, t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:], cu(seq, torch.int32), cu(pos, torch.int32),
                             cos_sin=None if cs is None else cu(cs), interleaved=inter, q=t[:, :Hq], q_out=q_out,
                             rope_pos=cu(at, torch.int32) if apart else None)
    assert got is q_out
    x = qkv[:n]
    if rot:
        r, free = pr.rotate(x, cs[at[:n]], inter)
        # the stated roundings cost at most half a bf16 step and three fp32 steps of the pair's size
        big = np.abs(x).max(-1, keepdims=True) * 2
        assert np.all(np.abs(r - free) <= np.abs(free) * 2.0 ** -8 * 1.001 + big * 2.0 ** -22)
        x = np.concatenate((r[:, :Hq + Hkv], x[:, Hq + Hkv:]), 1)
    assert np.array_equal(q_out[:n].double().cpu().numpy(), x[:, :Hq])
    assert torch.all(q_out[n:] == 7.0)                                  # padding: left as it was
    want = [b.clone() for b in before]
    for i in range(n):
        pg, row = c.spot(seq[i], pos[i])
        for w, e in ((0, exps[0]), (1, exps[1])):
            rows = x[i, Hq + w * Hkv:Hq + (w + 1) * Hkv]
            if fmt == "bf16":
                want[w][pg, :, row] = torch.from_numpy(rows).to(torch.bfloat16)
            else:
                cd, sc = pr.quantize(rows, e)
                want[w][pg, :, row], want[2 + w][pg, :, row] = torch.from_numpy(cd), torch.from_numpy(sc)
    for a, b in zip(storage(fx, c, dev), want):
        assert torch.equal(bits(a), bits(b))
    # and back: every row of every sequence, and nothing past a length
    T = c.max_pages * page
    k_out, v_out = (torch.full((c.B, Hkv, T, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fx.fx_paged_gather(dev, T, k_out=k_out, v_out=v_out)
    for w, o in ((0, k_out), (1, v_out)):
        ref = np.full((c.B, Hkv, T, D), 3.0)
        for b, ln in enumerate(c.lens):
            pg, row = c.spot(b, np.arange(ln))
            if fmt == "bf16":
                ref[b, :, :ln] = want[w].double().numpy()[pg, :, row].swapaxes(0, 1)
            else:
                v = pr.dequantize(want[w].numpy(), want[2 + w].numpy(), exps[w])
                ref[b, :, :ln] = v[pg, :, row].swapaxes(0, 1)
        assert np.array_equal(o.double().cpu().numpy(), ref)


def test_append_rotates_queries_in_place(fx):
    c = pr.Cache("bf16", [9, 4], 2, 16, seed=1)
    dev = c.device(fx)
    g = np.random.default_rng(2)
    for inter in (False, True):
        x = pr.bf16(g.standard_normal((2, 8, D)))
        cs = table_of(64, 16)
        t = cu(x, torch.bfloat16)
        fx.fx_paged_append(dev, t[:, 4:6], t[:, 6:], cu([0, 1], torch.int32), cu([8, 3], torch.int32), cos_sin=cu(cs),
                           interleaved=inter, q=t[:, :4], q_out=t[:, :4])
        r, _ = pr.rotate(x[:, :4], cs[[8, 3]], inter)
        assert np.array_equal(t[:, :4].double().cpu().numpy(), r)
        assert np.array_equal(t[:, 4:].double().cpu().numpy(), x[:, 4:])


def test_append_blocks_that_are_not_finite_and_borders(fx):
    c = pr.Cache("e2m1", [1, 1], 1, 16, seed=1, exps=(0, 3))
    dev = c.device(fx)
    row = np.zeros(D)
    row[:16] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -2.5, -0.25, 0.5, 4, -0.0, 0.0]
    row[16:32] = 2.0 ** -12
    row[32], row[48], row[64], row[80] = np.inf, np.nan, 1e5, 2.0 ** -130
    row[96:112] = 3.0e38
    row[112:128] = np.linspace(-1, 1, 16)
    row = pr.bf16(row)
    x = np.stack((row, row[::-1].copy()))[:, None]
    t = cu(x, torch.bfloat16)
    fx.fx_paged_append(dev, t, t, cu([0, 1], torch.int32), cu([0, 0], torch.int32))
    k, v = fx.fx_paged_gather(dev, 1)
    for got, e in ((k, 0), (v, 3)):
        ref = pr.dequantize(*pr.quantize(x, e), e)
        assert np.array_equal(got[:, :, 0].double().cpu().numpy(), ref, equal_nan=True)


def test_append_every_border_of_the_format(fx):
    """Rows of all bf16 magnitudes of four binades under every largest value of one: each block meets the borders of
    its codes exactly."""
    one = np.array([1 + m / 128 for m in range(128)])
    vals = np.concatenate([one * 2.0 ** e for e in (-3, -2, -1, 0)])
    rows = []
    for m in range(128):
        top = (1 + m / 128) * 2.0
        body = np.resize(vals, (len(vals) // 15 + 1, 15))
        rows.append(np.concatenate((np.full((len(body), 1), top), body), 1))
    x = np.concatenate(rows).reshape(-1)
    x = np.resize(x, (len(x) // D + 1, 1, D)) * np.where(np.arange(D) % 2, -1.0, 1.0)
    n = len(x)
    c = pr.Cache("e2m1", [n], 1, 64, seed=1)
    dev = c.device(fx)
    t = cu(x, torch.bfloat16)
    fx.fx_paged_append(dev, t, t, torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda"))
    codes, scales = pr.quantize(x)
    pg, row = c.spot(0, np.arange(n))
    assert np.array_equal(dev.k.cpu().numpy()[pg, :, row], codes)
    assert np.array_equal(dev.v_scale.cpu().numpy()[pg, :, row], scales)


def test_append_and_gather_report_bad_values(fx):
    c = pr.Cache("e2m1", [20, 20], 1, 16, seed=1)
    dev = c.device(fx)
    before = storage(fx, c, dev)
    x = torch.ones(4, 1, D, dtype=torch.bfloat16, device="cuda")
    cs = cu(table_of(32, 8))
    q_out = torch.zeros_like(x)

    def app(seq, pos, at):
        q_out.zero_()
        fx.fx_paged_append(dev, x, x, cu(seq, torch.int32), cu(pos, torch.int32), cos_sin=cs, q=x, q_out=q_out,
                           rope_pos=cu(at, torch.int32))
        return fx.fx_device_errors()
    assert app([2, -2, -1, -1], [0, 0, 0, 0], [0, 0, 0, 0]) == fx.FX_DEVERR_INDEX
    assert app([0, 1, -1, -1], [-1, 32, 0, 0], [0, 0, 0, 0]) == fx.FX_DEVERR_LEN
    assert app([0, 1, -1, -1], [0, 0, 0, 0], [-1, 8, 0, 0]) == fx.FX_DEVERR_INDEX
    assert not q_out.any()
    good = dev.table.clone()
    dev.table[1, 1] = c.n_pages
    dev.table[0, 1] = -1
    assert app([0, 1, -1, -1], [16, 31, 0, 0], [0, 0, 0, 0]) == fx.FX_DEVERR_PAGE
    assert q_out[:2].any() and not q_out[2:].any()
    for a, b in zip(storage(fx, c, dev), before):
        assert torch.equal(a, b)
    out = [torch.full((2, 1, 3, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fx.fx_paged_gather(dev, 3, idx=cu([[[-1, 20, 3]], [[1, 2, 17]]], torch.int32), k_out=out[0], v_out=out[1])
    assert fx.fx_device_errors() == fx.FX_DEVERR_INDEX | fx.FX_DEVERR_PAGE
    assert torch.all(out[0][0, 0, :2] == 3) and torch.all(out[1][1, 0, 2] == 3)
    assert np.array_equal(out[0][0, 0, 2].double().cpu().numpy(), c.rows(0, 0, 0, 3))
    assert np.array_equal(out[1][1, 0, :2].double().cpu().numpy(), c.rows(1, 1, 0, [1, 2]))
    fx.fx_paged_gather(dev, 3, lo=cu([-5, 30], torch.int32), k_out=out[0], v_out=out[1])
    assert fx.fx_device_errors() == fx.FX_DEVERR_LEN
    assert np.array_equal(out[0][0, 0].double().cpu().numpy(), c.rows(0, 0, 0, [0, 1, 2]))
    dev.table.copy_(good)
    dev.length.copy_(cu([-3, 1 << 20], torch.int32))
    fx.fx_paged_gather(dev, 1, k_out=out[0][:, :, :1].contiguous(), v_out=out[1][:, :, :1].contiguous())
    assert fx.fx_device_errors() == fx.FX_DEVERR_LEN


@pytest.mark.parametrize("fmt", FMT)
def test_gather_lists_and_starts(fx, fmt):
    c = pr.Cache(fmt, [77, 1, 0, 130], 3, 32, seed=8, layout="row", exps=(0, 0) if fmt == "bf16" else (4, -20))
    dev = c.device(fx)
    g = np.random.default_rng(4)
    idx = np.stack([g.integers(0, max(n, 1), (3, 45)) for n in c.lens])
    idx[2] = 0
    k, v = fx.fx_paged_gather(dev, 45, idx=cu(idx, torch.int32))
    assert fx.fx_device_errors() == fx.FX_DEVERR_INDEX                # the empty sequence has no row 0
    for b in (0, 1, 3):
        for h in range(3):
            assert np.array_equal(k[b, h].double().cpu().numpy(), c.rows(0, b, h, idx[b, h]))
            assert np.array_equal(v[b, h].double().cpu().numpy(), c.rows(1, b, h, idx[b, h]))
    out = [torch.full((4, 3, 50, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fx.fx_paged_gather(dev, 50, lo=cu([40, 0, 0, 129], torch.int32), k_out=out[0], v_out=out[1])
    for b, lo in enumerate([40, 0, 0, 129]):
        m = max(0, min(50, c.lens[b] - lo))
        for h in range(3):
            if m:
                assert np.array_equal(out[1][b, h, :m].double().cpu().numpy(), c.rows(1, b, h, np.arange(lo, lo + m)))
        assert torch.all(out[0][b, :, m:] == 9.0)


# ---------------------------------------------------------------------------------------- decode
LENS = [0, 1, 15, 16, 17, 63, 64, 65, 200, 333]
DECODE = [  # G, Mq, Hkv, page, layout, q layout
    (1, 1, 2, 16, "head", "head"), (2, 1, 3, 32, "row", "token"), (3, 1, 1, 64, "gap", "head"), (4, 1, 2, 128, "head", "token"),
    (5, 1, 1, 16, "row", "head"), (8, 1, 1, 256, "head", "head"), (12, 1, 1, 16, "head", "token"), (1, 4, 2, 16, "head", "head"),
    (2, 7, 2, 32, "row", "token"), (4, 8, 1, 64, "head", "token"), (8, 8, 1, 16, "gap", "head"), (64, 1, 1, 32, "head", "head"),
    (3, 2, 1, 512, "head", "token"), (1, 64, 1, 16, "row", "token"),
]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("G,Mq,Hkv,page,layout,ql", DECODE)
def test_decode_dense(fx, fmt, G, Mq, Hkv, page, layout, ql):
    exps = (0, 0) if fmt == "bf16" else (1, -2)
    c = pr.Cache(fmt, LENS, Hkv, page, seed=G * 10 + Mq, layout=layout, exps=exps)
    q, qt = queries(c, G, Mq, G + Mq, layout=ql)
    out, lse = fx.fx_paged_decode(c.device(fx), qt, want_lse=True)
    check_out(out, lse, pr.attend(c, q, 128 ** -0.5))
    assert not out[0].any()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("G,Mq,k,tail", [(2, 1, 5, 7), (4, 1, 16, 0), (1, 1, 33, 40), (8, 1, 100, 1), (2, 3, 21, 18),
                                         (12, 2, 17, 64)])
def test_decode_listed_rows_and_tail(fx, fmt, G, Mq, k, tail):
    c = pr.Cache(fmt, [150, 40, 333, 64, 1], 2, 32, seed=k)
    g = np.random.default_rng(k + tail)
    idx = np.stack([g.integers(0, n, (2, k)) for n in c.lens])       # any order, repeats among them
    lo = np.array([max(0, n - tail) for n in c.lens])
    q, qt = queries(c, G, Mq, k)
    dev = c.device(fx)
    out, lse = fx.fx_paged_decode(dev, qt, cu(idx, torch.int32), cu(lo, torch.int32), want_lse=True)
    check_out(out, lse, pr.attend(c, q, 128 ** -0.5, idx, lo))
    # a list alone: the tail starts at the length
    out, lse = fx.fx_paged_decode(dev, qt, cu(idx, torch.int32), cu(c.lens, torch.int32), want_lse=True)
    check_out(out, lse, pr.attend(c, q, 128 ** -0.5, idx, c.lens))
    # a tail alone, and starts that are no multiple of anything or lie past the length
    lo = np.array([3, 39, 17, 64, 200])
    out, lse = fx.fx_paged_decode(dev, qt, None, cu(lo, torch.int32), want_lse=True)
    check_out(out, lse, pr.attend(c, q, 128 ** -0.5, None, lo))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0, 1e-20])
def test_decode_scales_and_sharp_rows(fx, fmt, scale):
    c = pr.Cache(fmt, [400, 31], 1, 16, seed=5, channel=3.0)
    q, qt = queries(c, 4, 1, 7, scale=5.0)
    out, lse = fx.fx_paged_decode(c.device(fx), qt, scale=scale, want_lse=True)
    check_out(out, lse, pr.attend(c, q, np.float32(scale).astype(np.float64)))


@pytest.mark.parametrize("fmt", FMT)
def test_decode_many_small_weights_count(fx, fmt):
    """One row far above thousands of equal ones: what those add together is not lost to a 16-bit weight."""
    n, page = 4096, 64
    c = pr.Cache(fmt, [n], 1, page, seed=9)
    c.pool = [np.zeros_like(c.pool[0]), np.full_like(c.pool[1], 6.0)]     # keys, values of the many
    at = c.spot(0, 100)
    c.pool[0][at[0], 0, at[1], 0] = 6.0
    c.pool[1][at[0], 0, at[1]] = -6.0
    if fmt == "e2m1":
        c.packed = [pr.quantize(p) for p in c.pool]
        assert all(np.array_equal(pr.dequantize(*x), p) for x, p in zip(c.packed, c.pool))
    dev = c.device(fx)
    for drop in (8.0, 12.0, 18.0):                           # the others weigh e^-drop each
        q = np.zeros((1, 1, 1, D))
        q[..., 0] = 1.0
        s = np.float64(np.float32(drop / 6))
        r = pr.attend(c, q, s)[0] / 6
        o = fx.fx_paged_decode(dev, cu(q, torch.bfloat16), scale=s).double().cpu().numpy() / 6
        # o + 1 is twice the share of the small ones: each weight's split 2^-16, the exponential and the sums
        # 2^-17, the logits 2^-18 drop of it.  Beside the large weight, 1 in these units, a tile's 15 others are
        # cut off at 2^-23 each, and the additions of at most 4096 / 16 tiles and 8 warps, and the quotient, round
        # to 2^-24 each (at worst all one way)
        tol = (2.0 ** -15 + 2.0 ** -18 * drop) * (r + 1) + 15 * 2.0 ** -23 + (32 + 8 + 2) * 2.0 ** -24
        assert tol.max() < (r + 1).min() / 8
        assert np.all(np.abs(o - r) <= tol), (drop, np.abs(o - r).max(), tol.max())


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("G,Mq", [(1, 1), (8, 1), (4, 4)])
def test_weights_are_not_rounded_to_few_bits(fx, fmt, G, Mq):
    """Logits that are exact up to the scale: what is left are the roundings of fp32 arithmetic.

    In base 2 a logit is s * c + r with |s c| <= 10 * 0.09 * 1.45 < 1.4 and |r| <= 15: c is off by 2^-23 of itself (its
    product and its rounding), the sum is rounded once below 16: 1.4 * 2^-23 + 2^-21 of the exponent, so ln 2 times
    that, 2^-21.1, of a weight, and 2^-22 by the exponential: 2^-20.5.  Each part of a weight is exact to 2^-23 and
    products and sums of few rows lose 2^-22 more, so a weight counts within 2^-19.8; numerator and denominator both
    do, and the quotient's roundings are below 2^-22: outputs within 2^-18.8 of sum p |v|.  (Weights of 17 bits leave
    some 2^-18.)"""
    lens = [2, 3, 5, 16, 40]
    c = pr.Cache(fmt, lens, 1, 16, seed=6)
    g = np.random.default_rng(4)
    keys = np.zeros(c.pool[0].shape)
    keys[..., 0] = g.choice([-3.0, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3], keys.shape[:-1])
    c.pool[0] = keys
    if fmt == "e2m1":
        c.packed[0] = pr.quantize(keys)
        c.pool[0] = pr.dequantize(*c.packed[0])          # (1 / 6 is no scale: these keys are a little off, and exact in 6 bits)
    q = np.zeros((5, G, Mq, D))
    q[..., 0] = pr.bf16(g.uniform(-3, 3, q.shape[:-1]))
    out = fx.fx_paged_decode(c.device(fx), torch.from_numpy(q).to(torch.bfloat16).cuda(), scale=0.09)
    r, _, mag, _, _ = pr.attend(c, q, np.float32(0.09).astype(np.float64))
    assert np.all(np.abs(out.double().cpu().numpy() - r) <= 2.0 ** -18.8 * mag)


def test_decode_tiny_and_huge_queries(fx):
    c = pr.Cache("e2m1", [70], 1, 16, seed=6)
    for mag in (2.0 ** -120, 2.0 ** -60, 2.0 ** 20, 2.0 ** 60):
        q, _ = queries(c, 2, 1, 3, scale=1.0)
        q = q * mag
        s = float(np.float32(0.09 / mag))
        out, lse = fx.fx_paged_decode(c.device(fx), cu(q, torch.bfloat16), scale=s, want_lse=True)
        check_out(out, lse, pr.attend(c, q, s), mag)


@pytest.mark.parametrize("fmt", FMT)
def test_values_in_unseen_rows_reach_nothing(fx, fmt):
    """Draft rows of NaN: the queries before them do not see them, those after them are NaN."""
    c = pr.Cache(fmt, [40, 33], 1, 16, seed=2)
    q, qt = queries(c, 2, 4, 3)
    ref = pr.attend(c, q, 128 ** -0.5)
    dev = c.device(fx)
    for b in range(2):
        pg, row = c.spot(b, c.lens[b] - 2)                      # the row of query 2
        if fmt == "bf16":
            dev.v[pg, :, row] = float("nan")
        else:
            dev.v_scale[pg, :, row] = 0x7f
    out, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
    check_out(out[:, :, :2], lse[:, :, :2], tuple(x[:, :, :2] for x in ref))
    assert torch.isnan(out[:, :, 2:]).all()
    # a NaN key makes its readers NaN, and only them
    dev = c.device(fx)
    for b in range(2):
        pg, row = c.spot(b, c.lens[b] - 1)
        if fmt == "bf16":
            dev.k[pg, :, row] = float("nan")
        else:
            dev.k_scale[pg, :, row] = 0x7f
    out, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
    check_out(out[:, :, :3], lse[:, :, :3], tuple(x[:, :, :3] for x in ref))
    assert torch.isnan(out[:, :, 3]).all() and torch.isnan(lse[:, :, 3]).all()
    one = pr.Cache(fmt, [1], 1, 16, seed=2)                     # the only row is NaN
    dev = one.device(fx)
    (dev.k if fmt == "bf16" else dev.k_scale)[one.spot(0, 0)[0]] = float("nan") if fmt == "bf16" else 0x7f
    assert torch.isnan(fx.fx_paged_decode(dev, qt[:1, :, :1])).all()


def test_logits_of_minus_infinity_weigh_nothing(fx):
    """Rows whose logit is -inf (a bf16 key of -inf) come first, alone in their tiles and next to finite ones."""
    lens = [40, 17, 3, 200, 33]
    c = pr.Cache("bf16", lens, 2, 16, seed=4)
    dead = [np.arange(32), np.arange(16), np.arange(3), np.arange(0, 200, 2), np.arange(31, 33)]
    for G, Mq in ((1, 1), (5, 1), (3, 3)):
        q, _ = queries(c, G, Mq, 3)
        q[..., 5] = 1.5
        dev = c.device(fx)
        for b, at in enumerate(dead):
            pg, row = c.spot(b, at)
            dev.k[torch.from_numpy(pg).cuda(), :, torch.from_numpy(row).cuda(), 5] = -float("inf")
        out, lse = fx.fx_paged_decode(dev, torch.from_numpy(q).to(torch.bfloat16).cuda(), want_lse=True)
        alive = [np.setdiff1d(np.arange(n), at) for n, at in zip(lens, dead)]
        c2 = pr.Cache("bf16", lens, 2, 16, seed=4)
        c2.keys = lambda b, h, idx=None, tail_lo=None: alive[b]
        check_out(out, lse, pr.attend(c2, q, 128 ** -0.5))
        if Mq == 1:                                             # every logit of sequence 2
            assert not out[2].any() and (lse[2] == -float("inf")).all()


def test_decode_reports_bad_values(fx):
    c = pr.Cache("bf16", [50, 64], 1, 16, seed=3)
    q, qt = queries(c, 2, 1, 4)
    dev = c.device(fx)
    idx = np.array([[[3, -1, 50, 1 << 30, 7]], [[0, 1, 2, 64, 63]]])
    out, lse = fx.fx_paged_decode(dev, qt, cu(idx, torch.int32), cu([50, 64], torch.int32), want_lse=True)
    assert fx.fx_device_errors() == fx.FX_DEVERR_INDEX
    check_out(out, lse, pr.attend(c, q, 128 ** -0.5, idx, [50, 64]))
    out, lse = fx.fx_paged_decode(dev, qt, None, cu([-4, 10], torch.int32), want_lse=True)
    assert fx.fx_device_errors() == fx.FX_DEVERR_LEN
    check_out(out, lse, pr.attend(c, q, 128 ** -0.5, None, [0, 10]))
    dev.table[0, 1] = c.n_pages
    dev.table[1, 3] = -1
    out, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
    assert fx.fx_device_errors() == fx.FX_DEVERR_PAGE
    keep = [np.r_[0:16, 32:50], np.r_[0:48]]
    c.keys = lambda b, h, idx=None, tail_lo=None: keep[b]
    check_out(out, lse, pr.attend(c, q, 128 ** -0.5))
    s = fx.fx_paged_importance(dev, qt, lse)
    assert fx.fx_device_errors() == fx.FX_DEVERR_PAGE
    assert not s[0, 0, 16:32].any() and not s[1, 0, 48:].any()
    assert np.allclose(s.sum(-1).cpu().numpy(), 2.0, atol=1e-4)
    dev = c.device(fx)
    dev.length.copy_(cu([-1, 65], torch.int32))
    out = fx.fx_paged_decode(dev, qt)
    assert fx.fx_device_errors() == fx.FX_DEVERR_LEN and not out[0].any()


def test_decode_long_splits_and_repeats_bit_for_bit(fx):
    """Long rows over many CTAs, one and several sequences; the same call gives the same bits."""
    for fmt, lens, Hkv, G, Mq in (("e2m1", [5000], 1, 4, 1), ("e2m1", [9000, 3, 4097], 2, 1, 1), ("bf16", [5001], 1, 2, 1),
                                  ("bf16", [4800, 100, 2047], 1, 8, 2), ("e2m1", [6000, 10], 1, 2, 7)):
        c = pr.Cache(fmt, lens, Hkv, 64, seed=lens[0], garbage=False)
        q, qt = queries(c, G, Mq, 1)
        dev = c.device(fx)
        ws = fx.Workspace(nbytes=fx.fx_paged_decode_workspace_bytes(len(lens), Hkv, G * Hkv, Mq))
        out, lse = fx.fx_paged_decode(dev, qt, want_lse=True, ws=ws)
        check_out(out, lse, pr.attend(c, q, 128 ** -0.5), fmt)
        for _ in range(3):
            o2, l2 = fx.fx_paged_decode(dev, qt, want_lse=True, ws=ws)
            assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_decode_many_sequences(fx):
    g = np.random.default_rng(0)
    lens = [int(x) for x in g.integers(0, 40, 700)]
    c = pr.Cache("e2m1", lens, 1, 16, seed=11)
    q, qt = queries(c, 2, 1, 2)
    out, lse = fx.fx_paged_decode(c.device(fx), qt, want_lse=True)
    check_out(out, lse, pr.attend(c, q, 128 ** -0.5))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("B,Hkv,G,Mq", [(31, 2, 1, 1), (33, 1, 4, 1), (40, 2, 2, 4), (64, 1, 2, 7), (127, 1, 8, 1),
                                        (128, 2, 4, 1), (129, 1, 1, 3), (257, 2, 5, 2)])
def test_batches_around_the_sizes_of_the_scan(fx, fmt, B, Hkv, G, Mq):
    """Ragged batches, a few long sequences among short and empty ones: decode and importance."""
    g = np.random.default_rng(B)
    lens = [int(x) for x in g.integers(0, 70, B)]
    lens[B // 3], lens[-1], lens[0] = 900, 333, 0
    c = pr.Cache(fmt, lens, Hkv, 32, seed=B)
    q, qt = queries(c, G, Mq, 2)
    dev = c.device(fx)
    out, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
    check_out(out, lse, pr.attend(c, q, 128 ** -0.5))
    s = fx.fx_paged_importance(dev, qt, lse, cand=(3, 777))
    ref, dl = pr.importance(c, q, lse.double().cpu().numpy(), 128 ** -0.5, 3, 777)
    assert np.all(np.abs(s.double().cpu().numpy() - ref) <= 2.0 ** -19 * (dl + 1) * ref + 1e-37)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("page", [16, 1024])
def test_long_lists_and_tails_over_many_ctas(fx, fmt, page):
    lens = [6000, 40, 2999]
    c = pr.Cache(fmt, lens, 2, page, seed=3)
    g = np.random.default_rng(1)
    q, qt = queries(c, 4, 1, 2)
    k = 2501
    idx = np.stack([np.stack([g.integers(0, n, k) for _ in range(2)]) for n in lens])   # rows may come twice
    tail = [5211, 0, 2990]
    out, lse = fx.fx_paged_decode(c.device(fx), qt, cu(idx, torch.int32), cu(tail, torch.int32), want_lse=True)
    check_out(out, lse, pr.attend(c, q, 128 ** -0.5, idx, tail))


ROOM = 1 << 19   # rows a sequence may grow to: 4-bit attention then takes tiles in pairs


@pytest.mark.parametrize("G,Mq,Hkv,page,layout,ql", [
    (2, 1, 3, 32, "row", "token"), (3, 1, 1, 64, "gap", "head"), (4, 1, 2, 128, "head", "token"), (8, 1, 1, 256, "gap", "head"),
    (1, 4, 2, 32, "head", "head"), (2, 4, 1, 64, "row", "token"), (7, 1, 1, 1024, "head", "head"), (5, 1, 1, 16, "head", "token"),
])
def test_decode_with_room_to_grow(fx, G, Mq, Hkv, page, layout, ql):
    lens = LENS + [1000, 32, 31, 47]
    c = pr.Cache("e2m1", lens, Hkv, page, seed=G + Mq, layout=layout, exps=(1, -2), max_pages=ROOM // page)
    q, qt = queries(c, G, Mq, G + Mq, layout=ql)
    dev = c.device(fx)
    out, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
    check_out(out, lse, pr.attend(c, q, 128 ** -0.5))
    g = np.random.default_rng(page)
    for k, tail in ((5, 7), (33, 40), (0, 100), (16, 0)):
        idx = np.stack([g.integers(0, max(n, 1), (Hkv, k)) for n in lens])
        idx[0] = -1                                                    # (an empty sequence has no row to list)
        lo = np.array([max(0, n - tail) for n in lens])
        out, lse = fx.fx_paged_decode(dev, qt, cu(idx, torch.int32) if k else None, cu(lo, torch.int32), want_lse=True)
        assert fx.fx_device_errors() == (fx.FX_DEVERR_INDEX if k else 0)
        check_out(out, lse, pr.attend(c, q, 128 ** -0.5, idx if k else None, lo))


def test_decode_with_room_unseen_and_long_rows(fx):
    c = pr.Cache("e2m1", [40, 33, 700, 64], 1, 32, seed=2, max_pages=ROOM // 32)
    q, qt = queries(c, 2, 4, 3)
    ref = pr.attend(c, q, 128 ** -0.5)
    dev = c.device(fx)
    for b in range(4):                                                 # the row of query 2: NaN
        pg, row = c.spot(b, c.lens[b] - 2)
        dev.v_scale[pg, :, row] = 0x7f
    out, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
    check_out(out[:, :, :2], lse[:, :, :2], tuple(x[:, :, :2] for x in ref))
    assert torch.isnan(out[:, :, 2:]).all()
    g = np.random.default_rng(3)
    lens = [int(x) for x in g.integers(0, 90, 150)] + [5000, 2047]
    for Hkv, G, Mq in ((2, 4, 1), (1, 2, 3)):
        c = pr.Cache("e2m1", lens, Hkv, 64, seed=G, max_pages=ROOM // 64, garbage=False)
        q, qt = queries(c, G, Mq, 1)
        dev = c.device(fx)
        out, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
        check_out(out, lse, pr.attend(c, q, 128 ** -0.5))
        o2, l2 = fx.fx_paged_decode(dev, qt, want_lse=True)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


# ---------------------------------------------------------------------------------------- importance
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("G,Mq,Hkv,page,cand", [(2, 1, 2, 16, None), (4, 1, 1, 64, (5, 301)), (1, 8, 1, 32, (0, 1)),
                                                (4, 8, 2, 16, (100, 333)), (8, 8, 1, 128, (17, 340)), (3, 5, 1, 16, None)])
def test_importance(fx, fmt, G, Mq, Hkv, page, cand):
    exps = (0, 0) if fmt == "bf16" else (2, 0)
    c = pr.Cache(fmt, LENS, Hkv, page, seed=G + Mq, exps=exps)
    q, qt = queries(c, G, Mq, 5, layout="token")
    dev = c.device(fx)
    _, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
    s = fx.fx_paged_importance(dev, qt, lse, cand=cand)
    lo, hi = cand or (0, c.max_pages * page)
    ref, dl = pr.importance(c, q, lse.double().cpu().numpy(), 128 ** -0.5, lo, hi)
    got = s.double().cpu().numpy()
    assert got.shape == ref.shape
    assert np.all(np.abs(got - ref) <= 2.0 ** -19 * (dl + 1) * ref + 1e-37)
    if cand is None:
        want = [G * min(n, Mq) for n in LENS]
        assert np.allclose(got.sum(-1), np.array(want)[:, None], rtol=1e-3)


@pytest.mark.parametrize("fmt", FMT)
def test_importance_leaves_out_rows_without_lse(fx, fmt):
    """Query rows with an lse of -inf add nothing, whatever they hold (a padded batch); their neighbours stay exact."""
    c = pr.Cache(fmt, [70, 45, 16], 2, 16, seed=9)
    q, qt = queries(c, 3, 2, 5)
    dev = c.device(fx)
    _, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
    lse[0, 1] = lse[1, 0, 1] = lse[1, 5, 0] = lse[2] = -float("inf")
    qt[0, 1] = float("nan")
    qt[1, 0, 1] = float("inf")
    qt[2, :, :, ::2] = float("nan")
    s = fx.fx_paged_importance(dev, qt, lse)
    ref, dl = pr.importance(c, q, lse.double().cpu().numpy(), 128 ** -0.5, 0, c.max_pages * 16)
    assert np.all(np.abs(s.double().cpu().numpy() - ref) <= 2.0 ** -19 * (dl + 1) * ref + 1e-37)
    assert not s[2].any()


# ---------------------------------------------------------------------------------------- together
def test_matches_the_contiguous_calls(fx):
    """The same rows in a contiguous bf16 cache: focal attention, importance and sparse decode agree."""
    c = pr.Cache("e2m1", [300, 77, 512], 2, 32, seed=21)
    dev = c.device(fx)
    k, v = (torch.zeros(3, 2, 512, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fx.fx_paged_gather(dev, 512, k_out=k, v_out=v)
    q, qt = queries(c, 4, 1, 2)
    o1, s1 = fx.fx_focal_attn_scores(k, v, dev.length, qt)
    o2, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
    s2 = fx.fx_paged_importance(dev, qt, lse, cand=(0, 512))
    assert torch.allclose(o1, o2, atol=2e-3 * float(v.float().abs().max()))
    assert torch.allclose(s1, s2, rtol=2e-4, atol=1e-30)
    idx = fx.fx_topk_select(s2, 40)
    tail = torch.full((3,), 70, dtype=torch.int32, device="cuda")
    o1 = fx.fx_sparse_gqa_decode(k, v, dev.length, qt, idx, 70, ws=fx.Workspace())
    o2 = fx.fx_paged_decode(dev, qt, idx, tail)
    assert not (idx >= dev.length[:, None, None]).any()
    assert torch.allclose(o1, o2, atol=2e-3 * float(v.float().abs().max()))


class Model:
    """A decoding loop as a server runs it: prompt, then steps of append, dense attention, importance, selection and
    attention over the selection."""

    def __init__(self, fx, fmt, Mq=1):
        self.fx, self.B, self.H, self.G, self.page, self.Mq = fx, 3, 2, 4, 16, Mq
        self.lens0 = [70, 33, 50]
        B, H, page, P = self.B, self.H, self.page, 8
        z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        n = B * P
        table = torch.randperm(n, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, P).cuda()
        self.len = cu(self.lens0, torch.int32)
        if fmt == "bf16":
            self.c = fx.PagedKV(z(n, H, page, D, dt=torch.bfloat16), z(n, H, page, D, dt=torch.bfloat16), table, self.len)
        else:
            self.c = fx.PagedKV(z(n, H, page, 64), z(n, H, page, 64), table, self.len, k_scale=z(n, H, page, 8),
                                v_scale=z(n, H, page, 8))
        self.cs = cu(table_of(128, 256))
        self.tail = torch.zeros(B, dtype=torch.int32, device="cuda")
        g = torch.Generator().manual_seed(2)
        m = sum(self.lens0)
        self.prompt = torch.randn(m, (self.G + 2) * H, D, generator=g).to(torch.bfloat16).cuda()
        self.seq = torch.repeat_interleave(torch.arange(B), torch.tensor(self.lens0)).to(torch.int32).cuda()
        self.pos = torch.cat([torch.arange(n) for n in self.lens0]).to(torch.int32).cuda()
        self.qkv = torch.zeros(B * Mq, (self.G + 2) * H, D, dtype=torch.bfloat16, device="cuda")
        self.step_seq = torch.repeat_interleave(torch.arange(B), Mq).to(torch.int32).cuda()
        self.step_in = [torch.randn(self.qkv.shape, generator=g).to(torch.bfloat16).cuda() for _ in range(4)]

    def fill(self):
        Hq, H = self.G * self.H, self.H
        self.len.copy_(cu(self.lens0, torch.int32))
        self.fx.fx_paged_append(self.c, self.prompt[:, Hq:Hq + H], self.prompt[:, Hq + H:], self.seq, self.pos,
                                cos_sin=self.cs)

    def step(self, ws=None):
        fx, Hq, H, B, Mq = self.fx, self.G * self.H, self.H, self.B, self.Mq
        pos = (self.len[:, None] + torch.arange(Mq, device="cuda", dtype=torch.int32)).reshape(-1).to(torch.int32)
        x = self.qkv
        q = fx.fx_paged_append(self.c, x[:, Hq:Hq + H], x[:, Hq + H:], self.step_seq, pos, cos_sin=self.cs, q=x[:, :Hq])
        self.len.add_(Mq)
        q = q.view(B, Mq, Hq, D).transpose(1, 2)
        dense, lse = fx.fx_paged_decode(self.c, q, want_lse=True, ws=ws)
        scores = fx.fx_paged_importance(self.c, q, lse, cand=(0, 32))
        idx = fx.fx_topk_select(scores, 12)
        self.tail.copy_((self.len - 9).clamp(min=32))
        some = fx.fx_paged_decode(self.c, q, idx, self.tail, ws=ws)
        return dense, lse, scores, idx, some

    def run(self, do):
        self.fill()
        res = []
        for x in self.step_in:
            self.qkv.copy_(x)
            res.append([t.clone() for t in do()])
        return res


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("Mq", [1, 3])
@pytest.mark.parametrize("own_ws", [False, True])
def test_decoding_loop_eager_and_captured(fx, fmt, Mq, own_ws):
    m = Model(fx, fmt, Mq)
    ws = fx.Workspace(nbytes=fx.fx_paged_decode_workspace_bytes(m.B, m.H, m.G * m.H, Mq)) if own_ws else None
    eager = m.run(lambda: m.step(ws))
    # the first step against the plain statements, over the rows that the pages hold
    m.fill()
    m.qkv.copy_(m.step_in[0])
    dense, lse, scores, idx, some = m.step(ws)
    c = pr.Cache.__new__(pr.Cache)
    c.lens, c.B, c.Hkv = [n + Mq for n in m.lens0], m.B, m.H
    k, v = (t.double().cpu().numpy() for t in fx.fx_paged_gather(m.c, 128))
    c.rows = lambda w, b, h, at: (k, v)[w][b, h, at]
    qkv = m.step_in[0].double().cpu().numpy()
    at = np.concatenate([np.arange(n, n + Mq) for n in m.lens0])
    q, _ = pr.rotate(qkv[:, :m.G * m.H], m.cs.cpu().numpy()[at], False)
    q = q.reshape(m.B, Mq, -1, D).swapaxes(1, 2)
    check_out(dense, lse, pr.attend(c, q, 128 ** -0.5))
    s, dl = pr.importance(c, q, lse.double().cpu().numpy(), 128 ** -0.5, 0, 32)
    assert np.all(np.abs(scores.double().cpu().numpy() - s) <= 2.0 ** -19 * (dl + 1) * s + 1e-37)
    check_out(some, None, pr.attend(c, q, 128 ** -0.5, idx.cpu().numpy(), m.tail.cpu().numpy()))
    # captured once, replayed for every step: the same bits
    m.fill()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        outs = m.step(ws)
    got = m.run(lambda: (graph.replay(), outs)[1])
    for a, b in zip(eager, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_two_graphs_and_two_streams_at_once(fx):
    """Graphs captured without a workspace, and streams without one, do not share scratch: run at the same time they
    give what they give alone."""
    cs = [pr.Cache("e2m1", [6000], 1, 64, seed=s, garbage=False) for s in (1, 2)]
    devs = [c.device(fx) for c in cs]
    qs = [queries(c, 4, 1, 3)[1] for c in cs]
    alone = [fx.fx_paged_decode(d, q) for d, q in zip(devs, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for gr, d, q, s in zip(graphs, devs, qs, streams):
        with torch.cuda.graph(gr, stream=s):
            outs.append([fx.fx_paged_decode(d, q) for _ in range(8)])
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for a, os_ in zip(alone, outs):
        assert all(torch.equal(a, o) for o in os_)
    for _ in range(5):
        res = [[fx.fx_paged_decode(d, q, stream=s) for _ in range(8)] for d, q, s in zip(devs, qs, streams)]
        torch.cuda.synchronize()
        for a, os_ in zip(alone, res):
            assert all(torch.equal(a, o) for o in os_)


def test_views_whose_single_entries_have_any_stride(fx):
    """The stride of a dimension of one entry addresses nothing, whatever it is."""
    c = pr.Cache("e2m1", [20, 5], 1, 16, seed=1)
    q, qt = queries(c, 1, 1, 2)
    odd = torch.as_strided(qt, qt.shape, (128, 1, 1, 1))
    assert torch.equal(fx.fx_paged_decode(c.device(fx), odd), fx.fx_paged_decode(c.device(fx), qt))
    tok = qt[:1, 0]                                             # [1, 1, 128]
    one = torch.as_strided(tok, tok.shape, (3, 1, 1))
    dev = c.device(fx)
    fx.fx_paged_append(dev, one, one, cu([1], torch.int32), cu([4], torch.int32))
    k, v = fx.fx_paged_gather(dev, 1, lo=cu([0, 4], torch.int32))
    want = pr.dequantize(*pr.quantize(q[0, 0, 0][None]))
    assert np.array_equal(k[1, 0].double().cpu().numpy(), want) and torch.equal(k[1], v[1])


@pytest.mark.parametrize("fmt", FMT)
def test_chained_launches_and_other_streams_give_the_same_bits(fx, fmt):
    """A chain of programmatic launches, and the same on a stream that is given instead of the current one."""
    m = Model(fx, fmt)
    Hq, H = m.G * m.H, m.H
    zero = torch.zeros(m.B, dtype=torch.int32, device="cuda")

    def chain(flags, stream):
        kw = dict(flags=flags, stream=stream)
        fx.fx_paged_append(m.c, m.prompt[:, Hq:Hq + H], m.prompt[:, Hq + H:], m.seq, m.pos, cos_sin=m.cs, **kw)
        x, res = m.step_in[0], []
        for i in range(3):
            q = fx.fx_paged_append(m.c, x[:, Hq:Hq + H], x[:, Hq + H:], m.step_seq, m.len + (i - 3), cos_sin=m.cs,
                                   q=x[:, :Hq], **kw)
            q = q.view(m.B, 1, Hq, D).transpose(1, 2)
            out, lse = fx.fx_paged_decode(m.c, q, want_lse=True, **kw)
            s = fx.fx_paged_importance(m.c, q, lse, cand=(0, 60), **kw)
            k, v = fx.fx_paged_gather(m.c, 60, k_out=torch.zeros(m.B, H, 60, D, dtype=torch.bfloat16, device="cuda"),
                                      v_out=torch.zeros(m.B, H, 60, D, dtype=torch.bfloat16, device="cuda"), lo=zero, **kw)
            res += [q, out, lse, s, k, v]
        return res

    want = chain(0, None)
    torch.cuda.synchronize()
    got = chain(fx.FX_LAUNCH_PDL, None)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    side = torch.cuda.Stream()
    for flags in (0, fx.FX_LAUNCH_PDL):
        torch.cuda.synchronize()      # (the chain's inputs are made on the current stream)
        with torch.cuda.stream(side):
            got = chain(flags, None)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    q = want[0].contiguous()
    torch.cuda.synchronize()
    a = fx.fx_paged_decode(m.c, q)
    b = fx.fx_paged_decode(m.c, q, stream=side)
    c = fx.fx_paged_decode(m.c, q, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("heads_first", [False, True])
def test_pools_past_32_bits(fx, fmt, heads_first):
    """Pages, or heads, more than 4 GiB from the pool's start: the same bits as from a small pool."""
    c = pr.Cache(fmt, [150, 70, 333], 2, 64, seed=8, garbage=False)
    small = c.device(fx)
    N = 140000 if fmt == "bf16" else 560000
    n = c.n_pages

    def far(t):
        shape = (2, N) + t.shape[2:] if heads_first else (N, 2) + t.shape[2:]
        big = torch.empty(shape, dtype=t.dtype, device="cuda")
        big = big.transpose(0, 1) if heads_first else big
        big[N - n:] = t.flip(0)
        return big
    k = far(small.k)
    assert k[N - n, 1].data_ptr() - k.data_ptr() > 1 << 32             # the last head's rows
    kw = {} if fmt == "bf16" else dict(k_scale=far(small.k_scale), v_scale=far(small.v_scale), k_exp=c.exps[0], v_exp=c.exps[1])
    table = torch.where((small.table >= 0) & (small.table < n), N - 1 - small.table, small.table)
    dev = fx.PagedKV(k, far(small.v), table, small.length, **kw)
    g = np.random.default_rng(0)
    x = cu(pr.bf16(g.standard_normal((3, 4, D))), torch.bfloat16)
    q, qt = queries(c, 3, 2, 1)
    idx = cu(np.stack([np.stack([g.integers(0, m, 40) for _ in range(2)]) for m in c.lens]), torch.int32)
    got = []
    for cache in (small, dev):
        fx.fx_paged_append(cache, x[:, :2], x[:, 2:], cu([0, 1, 2], torch.int32), cu([140, 3, 332], torch.int32))
        out, lse = fx.fx_paged_decode(cache, qt, want_lse=True)
        some = fx.fx_paged_decode(cache, qt, idx, cu([120, 70, 300], torch.int32))
        rows = [torch.zeros(3, 2, 333, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        fx.fx_paged_gather(cache, 333, k_out=rows[0], v_out=rows[1])
        got.append([out, lse, some, fx.fx_paged_importance(cache, qt, lse), *fx.fx_paged_gather(cache, 40, idx=idx), *rows])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_binding_refusals(fx):
    c = pr.Cache("e2m1", [20], 2, 16, seed=1)
    dev = c.device(fx)
    q = torch.zeros(1, 4, 1, D, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fx.FxError):
        fx.PagedKV(dev.k, dev.v, dev.table, dev.length)                               # no scales
    with pytest.raises(fx.FxError):
        fx.PagedKV(dev.k, dev.v[:, :1], dev.table, dev.length, k_scale=dev.k_scale, v_scale=dev.v_scale)
    with pytest.raises(fx.FxError):
        fx.PagedKV(dev.k, dev.v, dev.table, dev.length.cpu(), k_scale=dev.k_scale, v_scale=dev.v_scale)
    for bad in (q.float(), q.cpu(), q[0], q.expand(2, 4, 1, D), q[:, :3], q[..., :64]):
        with pytest.raises(fx.FxError):
            fx.fx_paged_decode(dev, bad)
    with pytest.raises(fx.FxError):
        fx.fx_paged_decode(dev, q, torch.zeros(1, 2, 3, dtype=torch.int64, device="cuda"))
    with pytest.raises(fx.FxError):
        fx.fx_paged_decode(dev, q, out=torch.zeros(1, 4, 1, D, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(fx.FxError):
        fx.fx_paged_decode(dev, torch.zeros(1, 4, 33, D, dtype=torch.bfloat16, device="cuda"))   # 66 rows a head
    with pytest.raises(fx.FxError):
        fx.fx_paged_importance(dev, q, torch.zeros(1, 4, 1, device="cuda"), cand=(0, 33))
    with pytest.raises(fx.FxError):
        fx.fx_paged_append(dev, q[0], q[0], torch.zeros(4, dtype=torch.int32, device="cuda"),
                           torch.zeros(3, dtype=torch.int32, device="cuda"))
    ws = fx.Workspace(nbytes=512)
    assert fx.fx_paged_decode(dev, q, ws=ws).shape == (1, 4, 1, D)                    # grows the workspace it is given
