"""Which windowed prefill calls take a workspace: only those that are split.  (Each call here runs on a host thread of its
own, which has no buffer yet and keeps the one it takes until it ends.)"""
import threading

import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from plain64 import Pages, assert_within, attend, f64, sees

pytestmark = pytest.mark.gpu


def taken(chunk, hq, hkv, splits, **kw):
    """Bytes of device memory that a call with one chunk and a window of 1000 takes, after checking some of its rows."""
    pages = Pages((chunk,), hkv, 64, chunk)
    q = pages.randn(chunk, hq, 64)
    kc, vc, table, cl = pages.cuda()
    qg, start = q.cuda(), torch.tensor([0, chunk], dtype=torch.int32, device="cuda")
    out = torch.empty_like(qg)
    torch.cuda.synchronize()
    before, took, raised = torch.cuda.memory_allocated(), [], []

    def call():
        try:
            pkv.paged_window_prefill_attention(qg, kc, vc, table, cl, start, chunk, 0.1, out, 1000, 0, num_splits=splits, **kw)
            torch.cuda.synchronize()
            took.append(torch.cuda.memory_allocated() - before)
        except Exception as e:
            raised.append(e)

    thread = threading.Thread(target=call)
    thread.start()
    thread.join()
    if raised:
        raise raised[0]
    qf, kf, vf = f64(q), f64(pages.k), f64(pages.v)
    for i in (0, chunk // 2, chunk - 1):
        ref, allowed = attend(qf[i], kf, vf, pages.table[0], sees(i, 1000), 0.1, 2.0**-8)
        assert_within(out[i:i + 1], ref[None], allowed[None], f"row {i}")
    assert device_errors() == 0
    return took[0]


@pytest.mark.parametrize("splits", [0, 2, 32])
def test_calls_that_are_not_split_take_none(splits):
    """2500 rows of 8 kv heads, four q heads each: 40 tile pairs, 320 units."""
    assert pkv.window_prefill_splits(2500, 2500, 1, 32, 8, 32) == 1
    assert taken(2500, 32, 8, splits) == 0


def test_a_given_workspace_is_not_looked_at_by_a_call_that_is_not_split():
    assert taken(2500, 32, 8, 4, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")) == 0


def test_calls_that_are_split_take_one():
    assert pkv.window_prefill_splits(300, 300, 1, 8, 2, 5) == 5
    need = pkv.window_prefill_workspace_size(64, 5)
    assert need <= taken(300, 8, 2, 5) < need + (1 << 21)
    with pytest.raises(ValueError, match="workspace"):
        taken(300, 8, 2, 5, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("rows,most,seqs", [(512, 512, 1), (600, 512, 3), (1, 1, 1), (1200, 64, 19), (1216, 64, 19),
                                            (1217, 64, 20), (5000, 64, 320)])
def test_the_count_goes_by_the_units(rows, most, seqs):
    """Eight kv heads, four q heads each, 64 tokens a tile pair: split if twice the most units fit the SMs."""
    sms = min(160, torch.cuda.get_device_properties(0).multi_processor_count)
    units = 8 * min(seqs * -(-most // 64), rows // 64 + seqs)
    assert pkv.window_prefill_splits(rows, most, seqs, 32, 8, 7) == (7 if 2 * units <= sms else 1)
