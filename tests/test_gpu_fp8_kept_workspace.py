"""A workspace that goes by the cache's size is not kept: chunk attention over the 8-bit cache, given none, leaves no more
memory allocated than it found, and calls in a row, on two streams and in two threads find the memory again."""
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from test_fp8_least_workspace import long_case
from test_gpu_fp8_calls import on_a_thread

pytestmark = pytest.mark.gpu


def test_large_ones_are_not_kept():
    case, _ = long_case()
    assert case.need > 64 << 20
    want = case.call(unpack=False)
    outs = [torch.empty_like(want) for _ in range(6)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()

    def calls(outs, stream):
        for out in outs:
            pkv.paged_fp8_prefill_attention(case.dq, *case.caches, case.dstart, case.most, 0.09, out, stream=stream)

    calls(outs[:2], streams[0])
    assert torch.cuda.memory_allocated() == before
    assert torch.cuda.max_memory_allocated() >= before + case.need  # (it did take one)
    threads = [on_a_thread(lambda x=x: calls(outs[2 + 2 * x:4 + 2 * x], streams[x])) for x in range(2)]
    for thread, raised in threads:
        thread.join()
        assert not raised, raised
    assert torch.cuda.memory_allocated() == before
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs) and device_errors() == 0


def test_what_follows_on_the_stream_may_use_the_memory():
    """Tensors that are made right behind a call take its memory, and the call's result is whole."""
    case, _ = long_case()
    want = case.call(unpack=False)
    torch.cuda.synchronize()
    for _ in range(4):
        out = case.call()
        over = [torch.full((case.need // 2,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(bool((x == 0x7F).all()) for x in over)
        del over
    assert device_errors() == 0
