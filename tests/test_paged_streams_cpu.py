"""Scratch and output memory of the paged calls by stream, without a GPU."""
import pytest
import torch

import kv_cache_token_fx_gb300 as fx


class OneDevice:
    device, _index = torch.device("cuda", 0), 0


class PerThread:
    cuda_stream = 2


def test_the_per_thread_default_stream_gets_no_memory_by_its_handle():
    """Handle 2 is another stream in every thread: a workspace kept for it, or memory of an allocator that knows streams
    by their handles, would be shared by streams that run at the same time."""
    kept = dict(fx._stream_ws)
    for stream in (None, 2, PerThread()):                      # (None: it is the current stream)
        with pytest.raises(fx.FxError, match="per-thread"):
            fx._paged_workspace(OneDevice, 256, stream, 2)
    for stream in (2, PerThread()):
        with pytest.raises(fx.FxError, match="per-thread"):
            fx._paged_alloc(OneDevice, stream, (1,), torch.float32)
    assert fx._stream_ws == kept
