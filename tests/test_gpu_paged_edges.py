"""The paged-cache calls at the ends of their ranges, on a GPU: keys that are not finite, values near bf16's largest
and far below 1, logits of any size, scratch memory on streams that are not current."""
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


def queries(c, G, Mq, seed, scale=2.0):
    q = pr.bf16(scale * np.random.default_rng(seed).standard_normal((c.B, c.Hkv * G, Mq, D)))
    return q, bf16_cuda(q)


def bf16_cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).cuda()


def host(t):
    return t.double().cpu().numpy()


def poison(c, dev, b, at):
    """Makes the K rows `at` of sequence b NaN."""
    pg, row = (torch.from_numpy(np.atleast_1d(x)).long().cuda() for x in c.spot(b, np.asarray(at)))
    if c.fmt == "bf16":
        dev.k[pg, :, row] = float("nan")
    else:
        dev.k_scale[pg, :, row] = 0x7f


def importance_tolerance(ref, dl):
    """A logit is within 2^-19 dl (|lse| counted into dl), the exponential and the sums within 2^-20 of themselves."""
    return 2.0 ** -19 * (dl + 1) * ref + 1e-37


# ---------------------------------------------------------------------------------------- importance, not finite
@pytest.mark.parametrize("G,Mq", [(1, 1), (2, 1), (5, 1), (8, 1), (3, 3), (4, 4)])
def test_importance_of_rows_with_logits_of_minus_infinity(fx, G, Mq):
    """bf16 keys of -inf under queries that are positive there: their rows report 0, whatever the number of query rows
    is; a sequence of such rows alone has an lse of -inf and reports zeros."""
    lens = [40, 17, 3, 200, 33]
    c = pr.Cache("bf16", lens, 2, 16, seed=4)
    dead = [np.arange(32), np.arange(16), np.arange(3), np.arange(0, 200, 2), np.arange(31, 33)]
    q, _ = queries(c, G, Mq, 3)
    q[..., 5] = 1.5
    qt, dev = bf16_cuda(q), c.device(fx)
    for b, at in enumerate(dead):
        pg, row = c.spot(b, at)
        dev.k[torch.from_numpy(pg).cuda(), :, torch.from_numpy(row).cuda(), 5] = -float("inf")
    _, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
    ref, dl = pr.importance(c, q, host(lse), 128 ** -0.5, 0, c.max_pages * 16)
    for b, at in enumerate(dead):
        ref[b][:, at] = 0.0
    got = host(fx.fx_paged_importance(dev, qt, lse))
    assert np.all(np.abs(got - ref) <= importance_tolerance(ref, dl))
    assert not got[2].any()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("G,Mq", [(1, 2), (3, 2), (4, 2)])
def test_importance_leaves_out_queries_without_lse_under_keys_that_are_nan(fx, fmt, G, Mq):
    c = pr.Cache(fmt, [70, 45, 64], 2, 16, seed=9)
    q, qt = queries(c, G, Mq, 5)
    dev = c.device(fx)
    _, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
    lse[0] = -float("inf")            # nothing of sequence 0 counts
    lse[1, :, 1] = -float("inf")      # of sequence 1 the last query, which alone sees the last row
    ref, dl = pr.importance(c, q, host(lse), 128 ** -0.5, 0, c.max_pages * 16)
    poison(c, dev, 0, [3, 20, 69])
    poison(c, dev, 1, [44])
    poison(c, dev, 2, [5, 63])        # seen and counted: NaN
    got = host(fx.fx_paged_importance(dev, qt, lse))
    assert np.isnan(got[2][:, [5, 63]]).all()
    got[2][:, [5, 63]] = ref[2][:, [5, 63]]
    assert np.all(np.abs(got - ref) <= importance_tolerance(ref, dl))
    assert not got[0].any()


# ---------------------------------------------------------------------------------------- values and logits
def check_values(out, ref, floor):
    """|out - ref| <= (2^-18 dl + 2^-15) sum p|v|: the logits' error (2^-19 dl) in numerator and sum, the weights, sums
    and the quotient; and the floor."""
    r, _, mag, dl, _ = ref
    assert np.all(np.isfinite(out))
    assert np.all(np.abs(out - r) <= (2.0 ** -18 * dl[..., None] + 2.0 ** -15) * mag + floor)


@pytest.mark.parametrize("G,Mq", [(1, 1), (4, 1), (8, 1), (4, 4)])
@pytest.mark.parametrize("lens", [[1, 2, 40, 33, 16], [9000, 70]])
def test_values_near_the_largest_of_bf16(fx, lens, G, Mq):
    """Weighted means of values near 3.3e38 are finite: many equal weights, alternating signs, ordinary weights."""
    c = pr.Cache("bf16", lens, 1, 64, seed=2)
    g = np.random.default_rng(5)
    big = pr.bf16(3.3e38 * g.uniform(0.5, 1.0, c.pool[1].shape))
    for signs in (np.ones(big.shape), g.choice([-1.0, 1.0], big.shape)):
        c.pool[1] = big * signs
        dev = c.device(fx)
        for scale in (0.0, 2.0):
            q, qt = queries(c, G, Mq, 3, scale=scale)
            check_values(host(fx.fx_paged_decode(dev, qt)), pr.attend(c, q, 128 ** -0.5), 0.0)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("power", [-60, 60])
def test_values_far_from_one(fx, fmt, power):
    """No absolute error to speak of: values of 2^-60 come out as exactly as values of 2^60."""
    exps = (0, 0) if fmt == "bf16" else (0, power)
    for G, Mq, lens in ((1, 1, [1, 2, 40, 333]), (5, 1, [70, 9]), (3, 4, [500, 31])):
        c = pr.Cache(fmt, lens, 2, 32, seed=G, exps=exps)
        if fmt == "bf16":
            c.pool[1] = c.pool[1] * 2.0 ** power
        q, qt = queries(c, G, Mq, 4)
        # (4-bit rows: a weight's parts are off by up to 2^-36 of the largest)
        ref = pr.attend(c, q, 128 ** -0.5)
        check_values(host(fx.fx_paged_decode(c.device(fx), qt)), ref, 2.0 ** -36 * ref[4])


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("G,Mq", [(2, 1), (5, 1), (6, 2)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_of_any_size(fx, fmt, G, Mq, sign):
    """Logits up to 2^100 of either sign: the rows of the largest share the whole weight (the others' are at least a
    quarter of it away).

    Up to 2^20 they share it equally: exact weights, a sum of equal ones, one quotient; at most 2^-20 with the weights'
    parts.  Beyond, what fp32 may lose of a logit (2^-24 of it by one rounding) is no longer small beside 1: how they share
    is open, but the output lies between their values.  lse: 128 products, the scale times log2(e) and ln(2): within 2^-20
    of itself."""
    lens = [40, 3000, 17, 333]
    c = pr.Cache(fmt, lens, 2, 32, seed=3)
    g = np.random.default_rng(7)
    keys = np.zeros(c.pool[0].shape)
    keys[..., 0] = g.choice([0.0, 1.0, 2.0, 4.0] if sign > 0 else [2.0, 3.0, 4.0, 6.0], keys.shape[:-1])
    top = [[33], [2, 1500, 1501, 2999 - Mq], [0, 15 - Mq], [100, 101, 300]]
    for b, at in enumerate(top):
        pg, row = c.spot(b, np.asarray(at))
        keys[pg, :, row, 0] = 6.0 if sign > 0 else 1.0
    c.pool[0] = keys
    if fmt == "e2m1":
        c.packed[0] = pr.quantize(keys)
        c.pool[0] = pr.dequantize(*c.packed[0])
    best = c.rows(0, 0, 0, 33)[0]
    assert abs(np.sort(sign * np.unique(c.pool[0][..., 0]))[-2] - sign * best) > best / 4
    dev = c.device(fx)
    v = [np.stack([c.rows(1, b, h, at) for h in range(2)]).repeat(G, 0)[:, None] for b, at in enumerate(top)]
    mean, least, most, mag = (np.stack([f(x) for x in v]) for f in (
        lambda x: x.mean(2), lambda x: x.min(2), lambda x: x.max(2), lambda x: np.abs(x).max(2)))
    for power in (0, 10, 18, 20, 22, 23, 24, 26, 28, 30, 33, 40, 70, 97):
        q = np.zeros((len(lens), 2 * G, Mq, D))
        q[..., 0] = pr.bf16(g.uniform(1.0, 2.0, q.shape[:-1])) * 2.0 ** power
        s = sign * (3.0 if power < 10 else 0.7)
        if power < 10:                                   # (ordinary sizes: the others count)
            ref = pr.attend(c, q, s)
            check_values(host(fx.fx_paged_decode(dev, bf16_cuda(q), scale=s)), ref, 2.0 ** -36 * ref[4])
            continue
        out, lse = fx.fx_paged_decode(dev, bf16_cuda(q), scale=s, want_lse=True)
        out, lse = host(out), host(lse)
        lo, hi = (mean, mean) if power < 20 else (least, most)
        assert np.all(out >= lo - 2.0 ** -20 * mag) and np.all(out <= hi + 2.0 ** -20 * mag), power
        n = np.array([len(at) for at in top])[:, None, None]
        ref = np.float64(np.float32(s)) * best * q[..., 0] + np.log(n)
        assert np.all(np.abs(lse - ref) <= 2.0 ** -20 * np.abs(ref)), power


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("G,Mq", [(2, 1), (8, 1), (2, 7)])
def test_no_part_of_the_weights_is_lost_over_long_rows(fx, fmt, G, Mq):
    """Thousands of weights of two sizes, the smaller one no short binary fraction, over values that are all 1.

    The output is the sum of the weights' parts over the sum of the weights.  16 products of a tile are cut off at
    2^-24 of their sum each, for every part but the first: 2 * 2^-20.  A warp's additions (24 tiles at most here) and
    the sums over 4 warps and 16 CTAs at most round to 2^-24 each, in numerator and sum: 2 * 44 * 2^-24; quotient
    2^-24: less than 2^-17 in all.  (Half the weights without their second part would be 2^-11 off.)"""
    lens = [3000, 1501, 2222] * 8
    c = pr.Cache(fmt, lens, 2, 64, seed=6, garbage=False)
    keys = np.zeros(c.pool[0].shape)
    keys[:, :, ::2, 0] = 6.0
    c.pool = [keys, np.full(keys.shape, 6.0)]
    if fmt == "e2m1":
        c.packed = [pr.quantize(p) for p in c.pool]
        assert all(np.array_equal(pr.dequantize(*x), p) for x, p in zip(c.packed, c.pool))
    q = np.zeros((c.B, 2 * G, Mq, D))
    q[..., 0] = 1.0
    dev = c.device(fx)
    for drop in (0.2, 0.35, 0.61):
        out = host(fx.fx_paged_decode(dev, bf16_cuda(q), scale=drop / 6)) / 6
        assert np.all(np.abs(out - 1.0) <= 2.0 ** -17), (drop, np.abs(out - 1.0).max())


# ---------------------------------------------------------------------------------------- streams and scratch
def test_capture_on_a_stream_that_is_not_current(fx):
    """A call given a stream that is being captured takes its scratch from the graph, whatever the current stream does."""
    c = pr.Cache("e2m1", [3000], 1, 64, seed=1, garbage=False)
    dev = c.device(fx)
    _, qt = queries(c, 4, 1, 3)
    want = fx.fx_paged_decode(dev, qt)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    before = dict(fx._stream_ws)
    with torch.cuda.stream(side):
        graph.capture_begin()
    out = fx.fx_paged_decode(dev, qt, stream=side)
    with torch.cuda.stream(side):
        graph.capture_end()
    assert fx._stream_ws == before
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("own_ws", [False, True])
def test_programmatic_launches_are_captured(fx, own_ws):
    c = pr.Cache("e2m1", [3000, 64], 1, 64, seed=1, garbage=False)
    dev = c.device(fx)
    _, qt = queries(c, 4, 2, 3)
    ws = fx.Workspace(nbytes=fx.fx_paged_decode_workspace_bytes(2, 1, 4, 2)) if own_ws else None

    def chain():
        out, lse = fx.fx_paged_decode(dev, qt, want_lse=True, ws=ws, flags=fx.FX_LAUNCH_PDL)
        s = fx.fx_paged_importance(dev, qt, lse, flags=fx.FX_LAUNCH_PDL)
        again = fx.fx_paged_decode(dev, qt, ws=ws, flags=fx.FX_LAUNCH_PDL)
        return out, lse, s, again
    want = [t.clone() for t in chain()]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = chain()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_workspace_grows_beside_work_in_flight(fx):
    """The buffer that a workspace gives up stays reserved while calls on their stream still use it."""
    c = pr.Cache("e2m1", [3000], 1, 64, seed=1, garbage=False)
    dev = c.device(fx)
    small, large = queries(c, 4, 1, 3)[1], queries(c, 16, 1, 3)[1]
    want = [fx.fx_paged_decode(dev, q) for q in (small, large)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    ws = fx.Workspace(nbytes=fx.fx_paged_decode_workspace_bytes(1, 1, 4, 1))
    torch.cuda.synchronize()
    size, at = ws.buf.numel(), ws.buf.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1 << 30)
    first = fx.fx_paged_decode(dev, small, stream=side, ws=ws)
    assert ws.buf.data_ptr() == at
    second = fx.fx_paged_decode(dev, large, stream=side, ws=ws)
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    asleep = not side.query()
    torch.cuda.synchronize()
    assert asleep and ws.buf.numel() > size
    assert all(t.data_ptr() != at for t in others)
    assert torch.equal(first, want[0]) and torch.equal(second, want[1])


def test_a_workspace_of_another_device_is_refused(fx):
    c = pr.Cache("e2m1", [20], 1, 16, seed=1)
    _, qt = queries(c, 1, 1, 2)
    for device in ("cpu", "meta"):
        ws = fx.Workspace()
        ws.buf = torch.zeros(1 << 23, dtype=torch.uint8, device=device)     # as one made for that device holds it
        with pytest.raises(fx.FxError, match="ws must be"):
            fx.fx_paged_decode(c.device(fx), qt, ws=ws)


def test_ranges_of_rows_that_do_not_exist_are_refused(fx):
    c = pr.Cache("e2m1", [20], 2, 16, seed=1)
    dev = c.device(fx)
    _, qt = queries(c, 1, 1, 2)
    _, lse = fx.fx_paged_decode(dev, qt, want_lse=True)
    rows = c.max_pages * 16
    with pytest.raises(fx.FxError):
        fx.fx_paged_gather(dev, -1)
    for cand in ((5, 4), (-1, -1), (rows + 1, rows + 1), (0, rows + 1)):
        with pytest.raises(fx.FxError):
            fx.fx_paged_importance(dev, qt, lse, cand=cand)
    assert fx.fx_paged_importance(dev, qt, lse, cand=(rows, rows)).shape == (1, 2, 0)
    assert fx.fx_paged_gather(dev, 0)[0].shape == (1, 2, 0, D)


def test_memory_is_allocated_for_the_stream_of_a_handle(fx):
    """By number: the default stream's two handles, and another's.  What a call allocates belongs to its stream."""
    c = pr.Cache("e2m1", [300], 1, 16, seed=1)
    dev = c.device(fx)
    _, qt = queries(c, 2, 1, 2)
    want = fx.fx_paged_decode(dev, qt)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle, at in ((0, 0), (1, 0), (side.cuda_stream, side.cuda_stream)):
        with torch.cuda.stream(side), fx._on_stream(dev.device, handle):
            assert torch.cuda.current_stream().cuda_stream == at
        out = fx.fx_paged_decode(dev, qt, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
