"""Chunk attention over the 8-bit cache without the workspace that holds its blocks as bf16: asked for, or because there is no
memory for it.  It converts the blocks as it goes then, to the same bits where it is not split."""
import ctypes

import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from plain64 import BLOCK


def test_the_query_checks_its_arguments():
    from paged_kv_cache_275_gb300 import build
    build.build(quiet=True)
    lib, n = pkv.load(), ctypes.c_size_t(7)
    size = lib.pkv_fp8_prefill_least_workspace_size
    assert size(4, 1, 4, 32, 8, 128, 8, None) == 1
    assert size(-1, 1, 4, 32, 8, 128, 8, ctypes.byref(n)) == 1
    assert size(4, -1, 4, 32, 8, 128, 8, ctypes.byref(n)) == 1
    assert size(4, 1, 4, 30, 8, 128, 8, ctypes.byref(n)) == 1
    assert size(4, 1, 4, 32, 8, 96, 8, ctypes.byref(n)) == 2
    assert size(0, 1, 4, 32, 8, 128, 8, ctypes.byref(n)) == 0 and n.value == 0


def long_case(width=2000):
    from test_gpu_fp8_unpacked import Case

    case = Case((0, 100, 0), (1500, 1600, 1700), 16, 2, 128, seed=8, width=width)
    sizes = len(case.q), case.most, 3, 16, 2, 128, width
    assert case.need == pkv.fp8_prefill_workspace_size(*sizes) >= case.unpacked == 4 * 3 * width * BLOCK * 2 * 128
    return case, sizes


def on_a_thread_without_memory(f, piece):
    """f() on a thread of its own (which has kept no workspace), while this process can have no more than what it has and no
    piece of that as large as `piece` is free."""
    from test_gpu_fp8_calls import on_a_thread

    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction(torch.cuda.memory_reserved() / total)
    held = []
    try:
        while True:
            try:
                held.append(torch.empty(piece, dtype=torch.uint8, device="cuda"))
            except torch.OutOfMemoryError:
                break
        thread, raised = on_a_thread(f)
        thread.join()
        torch.cuda.synchronize()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    if raised:
        raise raised[0]


@pytest.mark.gpu
def test_asked_for():
    case, sizes = long_case()
    assert pkv.fp8_prefill_workspace_size(*sizes, unpack=False) == 0
    want = case.call()
    torch.cuda.synchronize()
    got = torch.empty_like(want)
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    pkv.paged_fp8_prefill_attention(case.dq, *case.caches, case.dstart, case.most, 0.09, got, unpack=False)
    assert torch.cuda.max_memory_allocated() == before
    assert torch.equal(got, want)
    launches = pkv.kernel_launch_count()
    case.call(unpack=False)
    assert pkv.kernel_launch_count() - launches == 1
    # A large workspace does not choose the form.
    case.call(unpack=False, workspace=torch.empty(case.need, dtype=torch.uint8, device="cuda"))
    assert pkv.kernel_launch_count() - launches == 2
    assert device_errors() == 0


@pytest.mark.gpu
def test_asked_for_and_split():
    from test_gpu_fp8_unpacked import Case

    case = Case((4096,), (1024,), 16, 2, 128, seed=9)
    sizes = 1024, 1024, 1, 16, 2, 128, case.caches[3].shape[1]
    least = pkv.fp8_prefill_workspace_size(*sizes, unpack=False)
    assert 0 < least <= case.need - case.unpacked
    case.check(case.call(unpack=False), rows=30)
    case.check(case.call(unpack=False, workspace=torch.full((least,), 0xFF, dtype=torch.uint8, device="cuda")), rows=30)
    with pytest.raises(ValueError, match="workspace"):
        case.call(unpack=False, workspace=torch.empty(least - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="workspace"):
        case.call(workspace=torch.empty(least, dtype=torch.uint8, device="cuda"))
    assert device_errors() == 0


@pytest.mark.gpu
def test_no_memory_for_the_blocks():
    case, _ = long_case()
    want, got = case.call(), torch.empty_like(case.dq)
    piece = 30 << 20
    assert case.need > piece
    on_a_thread_without_memory(
        lambda: pkv.paged_fp8_prefill_attention(case.dq, *case.caches, case.dstart, case.most, 0.09, got), piece)
    assert torch.equal(got, want) and device_errors() == 0


@pytest.mark.gpu
def test_no_memory_for_a_split_call_s_states():
    """A call that cannot do without says so, and the next one is served."""
    from test_gpu_fp8_unpacked import Case

    case = Case((4096,), (1024,), 16, 2, 128, seed=9)
    want, got = case.call(), torch.empty_like(case.dq)
    with pytest.raises(torch.OutOfMemoryError):
        on_a_thread_without_memory(
            lambda: pkv.paged_fp8_prefill_attention(case.dq, *case.caches, case.dstart, case.most, 0.09, got), 4 << 20)
    assert torch.equal(case.call(), want) and device_errors() == 0
