"""fx_paged_compact without a GPU: lengths that it would write over what it reads are refused before any device work."""
import ctypes

import pytest

from tests.test_paged_cpu import desc, lib  # noqa: F401


@pytest.mark.parametrize("what,at", [("src lengths", 0), ("src lengths", 4), ("src lengths", -4), ("tail_lo", 4), ("tail_lo", -4),
                                     ("src table", 0), ("src table", 12), ("dst table", 0), ("dst table", 8), ("dst table", 64 + 16), ("src table", 64 - 4), ("idx", 0), ("idx", 16)])
def test_lengths_that_overlap_what_is_read(lib, what, at):  # noqa: F811
    k, room = 3, dict(table_stride=16)               # 5 entries a row, 16 apart
    assert desc().B == 2 and desc().max_pages == 5
    reads = {"src lengths": 1 << 20, "tail_lo": 2 << 20, "src table": 3 << 20, "dst table": 4 << 20, "idx": 5 << 20}
    src = desc(table=reads["src table"], len=reads["src lengths"], **room)
    dst = desc(table=reads["dst table"], len=reads[what] + at, **room)
    assert lib.fx_paged_compact(ctypes.byref(src), ctypes.byref(dst), reads["idx"], k, reads["tail_lo"], 0, None) == 1
    assert b"of its own" in lib.fx_last_error()
