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
