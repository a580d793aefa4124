"""The paged-cache calls at the ends of their ranges, on a GPU: keys that are not finite."""
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
