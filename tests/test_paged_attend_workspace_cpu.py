"""fx_paged_attend_workspace_bytes without a GPU: what suffices for a longest prompt suffices for its chunks."""
import pytest


@pytest.mark.parametrize("B,Hkv,Hq", [(1, 8, 32), (1, 1, 64), (2, 8, 24), (18, 8, 32), (19, 8, 8), (1, 152, 152), (200, 1, 3),
                                      (257, 1, 4)])
def test_workspace_suffices_for_fewer_tokens(B, Hkv, Hq):
    import kv_cache_token_fx_gb300 as fx
    last = 0
    for max_new in sorted({*range(1, 300), *range(300, 9000, 61), 1 << 20}):
        n = fx.fx_paged_attend_workspace_bytes(B, Hkv, Hq, max_new)
        assert n >= last > -1, max_new
        last = n


def test_workspace_of_a_long_prompt_holds_its_chunks():
    """A prompt of 8191 tokens is not cut, a chunk of 100 of them is: 152 or so parts of 256 rows of 130 numbers."""
    import kv_cache_token_fx_gb300 as fx
    w = fx.fx_paged_attend_workspace_bytes
    assert w(1, 8, 32, 8191) == w(1, 8, 32, 100) >= 100 * 256 * 130 * 4
