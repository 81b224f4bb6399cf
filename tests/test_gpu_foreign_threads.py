"""Calls from OS threads that Python did not start (an embedding program's worker, a ctypes callback): such a thread
gets a new Python thread state, and with it new thread-local storage, each time it enters the interpreter, while what the
binding remembers of the thread lives as long as the OS thread.  A workspace must not outlive its owner."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from plain64 import Pages, assert_within, attend, f64, sees

pytestmark = pytest.mark.gpu

SOURCE = """
#include <pthread.h>
struct job { void (*enter)(int); int times; };
static void* body(void* x) {
  struct job* j = x;
  for (int i = 0; i < j->times; ++i) j->enter(i);
  return 0;
}
int run_on_a_thread(void (*enter)(int), int times) {
  struct job j = {enter, times};
  pthread_t t;
  return pthread_create(&t, 0, body, &j) || pthread_join(t, 0);
}
"""


@pytest.fixture(scope="module")
def run_on_a_thread(tmp_path_factory):
    """run_on_a_thread(f, n): one new OS thread enters Python n times, calling f(0) .. f(n - 1)."""
    d = tmp_path_factory.mktemp("thread")
    (d / "thread.c").write_text(SOURCE)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(d / "thread.so"), str(d / "thread.c"), "-lpthread"], check=True)
    lib = ctypes.CDLL(str(d / "thread.so"))
    kind = ctypes.CFUNCTYPE(None, ctypes.c_int)

    def run(f, times):
        raised = []

        def enter(i):
            try:
                f(i)
            except BaseException as e:  # (ctypes would print and drop it)
                raised.append(e)

        assert lib.run_on_a_thread(kind(enter), times) == 0
        if raised:
            raise raised[0]

    return run


def _window_decode():
    lens = (500, 40, 300)
    pages = Pages(lens, 2, 64, 40)
    q = pages.randn(3, 8, 64)
    kc, vc, table, cl = pages.cuda()
    dq = q.cuda()
    need = pkv.window_decode_workspace_size(3, 8, 2, 64, table.shape[1], 200, 4, 30)
    keys, extra = [sees(n - 1, 200, 4) for n in lens], 0.0
    return pages, q, keys, extra, need, lambda out: pkv.paged_window_decode_attention(
        dq, kc, vc, table, cl, 0.09, out, 200, 4, num_partitions=30)


def _window_prefill():
    lens = (500, 40, 300)  # one row a sequence
    pages = Pages(lens, 2, 64, 41)
    q = pages.randn(3, 8, 64)
    kc, vc, table, cl = pages.cuda()
    dq, start = q.cuda(), torch.arange(4, dtype=torch.int32, device="cuda")
    need = pkv.window_prefill_workspace_size(64, 4)
    keys, extra = [sees(n - 1, 200, 4) for n in lens], 2.0**-8
    return pages, q, keys, extra, need, lambda out: pkv.paged_window_prefill_attention(
        dq, kc, vc, table, cl, start, 1, 0.09, out, 200, 4, num_splits=4)


def _prefix_decode():
    lens = (500, 40, 300)
    pages = Pages(lens, 2, 64, 42, width=4000)
    q = pages.randn(3, 8, 64)
    kc, vc, table, cl = pages.cuda()
    dq, start = q.cuda(), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    prefix = torch.tensor([160], dtype=torch.int32, device="cuda")
    need = pkv.prefix_decode_workspace_size(3, 8, 2, 64, table.shape[1], 1)
    keys, extra = [sees(n - 1) for n in lens], 2.0**-8
    return pages, q, keys, extra, need, lambda out: pkv.paged_prefix_decode_attention(
        dq, kc, vc, table, cl, start, prefix, 0.09, out)


@pytest.mark.parametrize("make", [_window_decode, _window_prefill, _prefix_decode])
def test_a_foreign_thread_keeps_its_workspace_between_its_entries(make, run_on_a_thread):
    """Between two entries of one thread other tensors are allocated; the second call must not write to them."""
    pages, q, keys, extra, need, call = make()
    assert need > 0
    qf, kf, vf = f64(q), f64(pages.k), f64(pages.v)
    rows = [attend(qf[b], kf, vf, pages.table[b], keys[b], 0.09, extra) for b in range(len(keys))]
    ref, allowed = np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])
    outs = [torch.zeros(q.shape, dtype=q.dtype, device="cuda") for _ in range(3)]
    others = []
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()

    def enter(i):
        call(outs[i])
        torch.cuda.synchronize()
        # As large as the workspace (the allocator's best fit for memory that was given back), and smaller ones.
        others.extend(torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (need, need, need // 2, 4096))
        torch.cuda.synchronize()

    run_on_a_thread(enter, 3)
    for out in outs:
        assert_within(out, ref, allowed, "foreign thread")
    assert all(bool((t == 0x5A).all()) for t in others), "a call wrote to another tensor's memory"
    others.clear()
    assert torch.cuda.memory_allocated() == before, "the thread's workspace goes with the thread"
    assert device_errors() == 0
