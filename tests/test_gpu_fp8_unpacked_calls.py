"""How chunk attention over the 8-bit cache is called where its blocks are turned into bf16 ahead of it, with one split and with
several: the cases of test_gpu_fp8_calls for the calls that have most workspace and launches."""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
import test_gpu_fp8_calls as calls
from fp8_plain import Fp8Pages, attend_fp8
from plain64 import BLOCK, assert_within, f64
from test_gpu_foreign_threads import run_on_a_thread  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

FORMS = ["unpacked", "unpacked in splits"]


class Long(calls.Call):
    def __init__(self, form, seed=0):
        split = "splits" in form
        self.hq, self.hkv, self.d, self.decode = 16, 2, 128, False
        lens, self.chunks = ([4500], [1024]) if split else ([1500, 1600, 1000], [1500, 1400, 1000])
        self.pages = Fp8Pages(lens, self.hkv, self.d, seed)
        self.q = self.pages.randn(sum(self.chunks), self.hq, self.d)
        self.starts, self.chunk = np.concatenate([[0], np.cumsum(self.chunks)]), max(self.chunks)
        self.kc, self.vc, self.sc, self.table, self.cl = self.pages.cuda()
        self.dq = self.q.cuda()
        self.start = torch.from_numpy(self.starts.astype(np.int32)).cuda()
        n, w = len(lens), self.table.shape[1]
        self.need = pkv.fp8_prefill_workspace_size(len(self.q), self.chunk, n, self.hq, self.hkv, self.d, w)
        blocks = 4 * n * w * BLOCK * self.hkv * self.d
        if self.need:  # (0: the query is not to be made)
            assert self.need >= blocks + (2 * self.chunk * self.hq * (self.d + 2) * 4 if split else 0)

    def check(self, out):
        for row in {*np.random.RandomState(1).randint(0, len(self.q), 25).tolist(), 0, len(self.q) - 1}:
            b = int(np.searchsorted(self.starts, row, side="right")) - 1
            n = self.pages.lens[b] - self.chunks[b] + row - int(self.starts[b]) + 1
            assert_within(out[row], *attend_fp8(self.pages, b, f64(self.q[row]), n, calls.SCALE, 2.0**-8), f"row {row}")


@pytest.fixture(autouse=True)
def long_calls(monkeypatch):
    monkeypatch.setattr(calls, "Call", Long)


@pytest.mark.parametrize("form", FORMS)
def test_a_threads_first_cuda_call(form):
    calls.test_a_threads_first_cuda_call(form)


@pytest.mark.parametrize("form", FORMS)
def test_two_threads_on_two_streams(form):
    calls.test_two_threads_on_two_streams(form)


@pytest.mark.parametrize("form", FORMS)
def test_two_graphs_in_turns_and_at_once(form):
    calls.test_two_graphs_in_turns_and_at_once(form)


@pytest.mark.parametrize("form", FORMS)
def test_a_foreign_threads_calls(form, run_on_a_thread):  # noqa: F811
    calls.test_a_foreign_thread_keeps_its_workspace_between_its_entries(form, run_on_a_thread)


def test_first_calls_may_be_captured():
    program = calls.PROGRAM.replace("from test_gpu_fp8_calls import FORMS, Call",
                                    "from test_gpu_fp8_unpacked_calls import FORMS, Long as Call")
    program = program.replace("c.pages.randn(3, 4, 128)", "c.pages.randn(3, 2, 128)").replace("c.dq, k, v", "c.dq[:3], k, v")
    r = subprocess.run([sys.executable, "-c", program], cwd=Path(__file__).resolve().parents[1], capture_output=True,
                       text=True, timeout=240)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout[-500:] + r.stderr[-1500:]
