"""How the 8-bit cache's calls are made: first in a thread or captured first in a process, from threads that Python did not
start, two at a time, and as graphs that are replayed in turns and at once."""
import subprocess
import sys
import threading
from pathlib import Path

import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from fp8_plain import Fp8Pages, attend_fp8
from gpu_util import device_errors
from plain64 import assert_within, f64
from test_gpu_foreign_threads import run_on_a_thread  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

SCALE = 0.09
# Decode in clusters and in the stream form; chunks of a few rows (both forms), of one CTA's rows, and in splits.
FORMS = ["clusters", "stream", "few rows in clusters", "few rows in the stream", "chunks", "chunks in splits"]


class Call:
    """An attention call over a cache of its own, and what it must give."""

    def __init__(self, form, seed=0):
        stream, few = "stream" in form, "few rows" in form
        lens = [40 + 7 * (b % 9) for b in range(50)] if stream else [3000] if "splits" in form else [300, 40, 700]
        if form == "chunks":
            lens = lens * 20  # more than the GPU has SMs: no splits
        self.hq, self.hkv, self.d, chunk = 16, 8 if stream else 4, 128, 3 if few else 20 if "chunks" in form else 1
        self.pages = Fp8Pages(lens, self.hkv, self.d, seed)
        self.chunks = [1 if form in ("clusters", "stream") else chunk - b % 3 for b in range(len(lens))]
        self.q = self.pages.randn(sum(self.chunks), self.hq, self.d)
        self.starts = np.concatenate([[0], np.cumsum(self.chunks)])
        self.kc, self.vc, self.sc, self.table, self.cl = self.pages.cuda()
        self.dq = self.q.cuda()
        self.start = torch.from_numpy(self.starts.astype(np.int32)).cuda()
        self.decode, self.chunk = form in ("clusters", "stream"), chunk
        n, w = len(lens), self.table.shape[1]
        self.need = (pkv.fp8_decode_workspace_size(n, self.hq, self.hkv, self.d, w) if self.decode
                     else pkv.fp8_prefill_workspace_size(len(self.q), chunk, n, self.hq, self.hkv, self.d, w))

    def zeros(self):
        return torch.zeros_like(self.dq)

    def __call__(self, out, **kw):
        args = self.dq, self.kc, self.vc, self.sc, self.table, self.cl
        if self.decode:
            return pkv.paged_fp8_decode_attention(*args, SCALE, out, **kw)
        return pkv.paged_fp8_prefill_attention(*args, self.start, self.chunk, SCALE, out, **kw)

    def check(self, out):
        for b, n in enumerate(self.pages.lens):
            for i in range(self.chunks[b]):
                ref, allowed = attend_fp8(self.pages, b, f64(self.q[self.starts[b] + i]), n - self.chunks[b] + i + 1, SCALE,
                                          2.0**-8)
                assert_within(out[self.starts[b] + i], ref, allowed, f"sequence {b}, row {i}")


def test_the_forms_are_those_that_are_meant():
    for form in FORMS:
        assert (Call(form).need > 0) == (form in ("stream", "few rows in the stream", "chunks in splits")), form


def on_a_thread(f):
    raised = []

    def body():
        try:
            f()
        except Exception as e:
            raised.append(e)

    thread = threading.Thread(target=body)
    thread.start()
    return thread, raised


@pytest.mark.parametrize("form", FORMS)
def test_a_threads_first_cuda_call(form):
    call = Call(form, 1)
    want, got = call.zeros(), call.zeros()
    call(want)  # (what a process looks up once is looked up here)
    torch.cuda.synchronize()
    thread, raised = on_a_thread(lambda: call(got))
    thread.join()
    if raised:
        raise raised[0]
    torch.cuda.synchronize()
    assert torch.equal(want, got)
    call.check(got)
    assert device_errors() == 0


def test_rows_calls_are_a_threads_first():
    pages = Fp8Pages((40, 60), 2, 64, 3)
    caches = pages.cuda()[:3]
    k, v, q = pages.randn(5, 2, 64).cuda(), pages.randn(5, 2, 64).cuda(), pages.randn(5, 4, 64).cuda()
    slots, pos, cs = torch.tensor([0, 17, 33, -1, 5], device="cuda"), torch.arange(5, device="cuda"), torch.ones(8, 64, device="cuda")
    pairs = torch.tensor([[0, 3], [1, 4]], device="cuda")

    def steps(caches):
        rk, rv, turned = torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(q)
        for f in (lambda: pkv.kv_append_fp8(k, v, slots, *caches),
                  lambda: pkv.rope_append_fp8(q, k, v, pos, slots + 64, cs, *caches, turned),
                  lambda: pkv.copy_blocks_fp8(*caches, pairs), lambda: pkv.kv_gather_fp8(*caches, slots, rk, rv)):
            yield f
        yield rk, rv, turned, *caches

    here, there = [x.clone() for x in caches], [x.clone() for x in caches]
    *fs, want = steps(here)
    for f in fs:
        f()
    *fs, got = steps(there)
    torch.cuda.synchronize()
    for f in fs:
        thread, raised = on_a_thread(f)
        thread.join()
        assert not raised, raised
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got))
    assert device_errors() == 0


PROGRAM = """
import sys
sys.path[:0] = ["tests", "."]
import torch
import paged_kv_cache_275_gb300 as pkv
from test_gpu_fp8_calls import FORMS, Call

calls = [Call.__new__(Call) for _ in FORMS]
real = pkv.fp8_decode_workspace_size, pkv.fp8_prefill_workspace_size
pkv.fp8_decode_workspace_size = pkv.fp8_prefill_workspace_size = lambda *a: 0  # (nothing may be looked up early)
for c, f in zip(calls, FORMS):
    c.__init__(f)
pkv.fp8_decode_workspace_size, pkv.fp8_prefill_workspace_size = real
outs = [c.zeros() for c in calls]
c = calls[0]
k, v = c.pages.randn(3, 4, 128).cuda(), c.pages.randn(3, 4, 128).cuda()
rk, rv, turned = torch.zeros_like(k), torch.zeros_like(v), torch.zeros(3, 16, 128, dtype=torch.bfloat16, device="cuda")
slots, pos, cs = torch.tensor([0, -1, 20], device="cuda"), torch.arange(3, device="cuda"), torch.ones(8, 128, device="cuda")
pairs = torch.zeros(0, 2, dtype=torch.int64, device="cuda")

def steps():
    pkv.rope_append_fp8(c.dq, k, v, pos, slots, cs, c.kc, c.vc, c.sc, turned)
    pkv.kv_append_fp8(k, v, slots, c.kc, c.vc, c.sc)
    pkv.kv_gather_fp8(c.kc, c.vc, c.sc, slots, rk, rv)
    pkv.copy_blocks_fp8(c.kc, c.vc, c.sc, pairs)
    for call, out in zip(calls, outs):
        call(out)

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    steps()
g.replay()
torch.cuda.synchronize()
results = [*outs, rk, rv, turned]
captured = [o.clone() for o in results]
for o in results:
    o.zero_()
steps()
torch.cuda.synchronize()
assert pkv.get_and_clear_device_error() == 0
assert all(torch.equal(a, b) for a, b in zip(captured, results)), "captured and eager results differ"
print("same")
"""


def test_first_calls_may_be_captured():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=Path(__file__).resolve().parents[1], capture_output=True,
                       text=True, timeout=240)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout[-500:] + r.stderr[-1500:]


@pytest.mark.parametrize("form", ["stream", "few rows in the stream", "chunks in splits"])
def test_a_foreign_thread_keeps_its_workspace_between_its_entries(form, run_on_a_thread):  # noqa: F811
    call = Call(form, 2)
    outs, others = [call.zeros() for _ in range(3)], []
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()

    def enter(i):
        call(outs[i])
        torch.cuda.synchronize()
        others.extend(torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (call.need, call.need, 4096))
        torch.cuda.synchronize()

    run_on_a_thread(enter, 3)
    for out in outs:
        call.check(out)
    assert all(bool((t == 0x5A).all()) for t in others), "a call wrote to another tensor's memory"
    others.clear()
    assert torch.cuda.memory_allocated() == before, "the thread's workspace goes with the thread"
    assert device_errors() == 0


@pytest.mark.parametrize("form", FORMS)
def test_two_threads_on_two_streams(form):
    calls = [Call(form, 3), Call(form, 4)]
    outs = [[c.zeros() for _ in range(8)] for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()

    def body(x):
        for out in outs[x]:
            calls[x](out, stream=streams[x])
        streams[x].synchronize()

    threads = [on_a_thread(lambda x=x: body(x)) for x in range(2)]
    for thread, raised in threads:
        thread.join()
        assert not raised, raised
    for call, made in zip(calls, outs):
        assert all(torch.equal(made[0], o) for o in made)
        call.check(made[0])
    assert device_errors() == 0


@pytest.mark.parametrize("form", FORMS)
def test_two_graphs_in_turns_and_at_once(form):
    """Each graph's workspace is its own; eager calls between the replays take another."""
    calls = [Call(form, 5), Call(form, 6)]
    outs, graphs, streams = [c.zeros() for c in calls], [], [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for call, out in zip(calls, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(out)
        graphs.append(graph)
    want = [c(c.zeros()) for c in calls]
    torch.cuda.synchronize()
    for _ in range(4):
        for out in outs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        eager = calls[0](calls[0].zeros())
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(eager, want[0])
    for call, out in zip(calls, outs):
        call.check(out)
    assert device_errors() == 0
