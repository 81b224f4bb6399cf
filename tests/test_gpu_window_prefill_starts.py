"""Windowed prefill with query starts that fall: chunks over earlier ones are flagged and skipped, and nothing is written
outside the workspace.  (The host tells from the number of rows whether a call's units are split, and sizes the workspace
for that; chunks that overlap could be more units.)"""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from plain64 import Pages, assert_within, attend, f64, sees

pytestmark = pytest.mark.gpu
WINDOW, SINKS, SCALE = 24, 2, 0.1


def call(starts, length, rows, hq, hkv, d, splits, most):
    """Every sequence has the same `length` tokens.  The workspace is exactly as large as asked for, in front of bytes that
    must stay as they are."""
    pages = Pages((length,), hkv, d, 7)
    q = pages.randn(rows, hq, d)
    kc, vc, table, cl = pages.cuda()
    seqs = len(starts) - 1
    need = pkv.window_prefill_workspace_size(d, splits)
    whole = torch.full((need + (1 << 16),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    assert device_errors() == 0
    pkv.paged_window_prefill_attention(q.cuda(), kc, vc, table.repeat(seqs, 1), cl.repeat(seqs),
                                       torch.tensor(starts, dtype=torch.int32, device="cuda"), most, SCALE, out, WINDOW,
                                       SINKS, num_splits=splits, workspace=whole[:need] if splits > 1 else None)
    assert device_errors() == pkv.DEVERR_CONTEXT_LEN_TOO_LONG
    assert bool((whole[need:] == 0xA5).all()), "written behind the workspace"
    return pages, q, out


def check(pages, q, out, first, chunk):
    """Rows first .. first + chunk - 1 of out are a chunk's."""
    qf, kf, vf = f64(q), f64(pages.k), f64(pages.v)
    n = pages.lens[0]
    rows = [attend(qf[first + i], kf, vf, pages.table[0], sees(n - chunk + i, WINDOW, SINKS), SCALE, 2.0**-8)
            for i in range(chunk)]
    assert_within(out[first:first + chunk], np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows]),
                  f"rows from {first}")


@pytest.mark.parametrize("splits", [1, 2, 32])
@pytest.mark.parametrize("seqs,rows,hq,hkv,d", [
    (4, 1000, 16, 2, 64),   # 128 units where the rows bound 70: more than the workspace has records for
    (15, 1024, 4, 4, 64),   # 128 where they bound 76
    (68, 2048, 1, 1, 64),   # 272 where they bound 76: more units than SMs
    (68, 2048, 1, 1, 128),
    (330, 700, 2, 1, 64),   # two launches, not split
])
def test_starts_that_go_back_and_forth(seqs, rows, hq, hkv, d, splits):
    """Starts 0, rows, 0, rows, ...: the first chunk stands; the falling ones and those over the first are skipped."""
    pages, q, out = call([0 if i % 2 == 0 else rows for i in range(seqs + 1)], rows, rows, hq, hkv, d, splits, rows)
    check(pages, q, out, 0, rows)


@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("starts,stand", [
    ([0, 60, 30, 90], [(0, 60)]),             # the third chunk starts inside the first
    ([0, 60, 60, 40, 100], [(0, 60)]),        # an empty one in between
    ([0, 10, 500, 20, 60], [(0, 10), (20, 40)]),  # one that ends behind the rows is skipped and hides nothing
    ([50, 80, 10, 40, 90], [(50, 30)]),       # below an earlier one: skipped as well
    ([70, 40, 70, 100], [(40, 30), (70, 30)]),  # a falling start alone hides nothing
])
def test_which_chunks_stand(starts, stand, splits):
    pages, q, out = call(starts, 200, 100, 8, 2, 128, splits, 100)
    untouched = np.ones(100, dtype=bool)
    for first, chunk in stand:
        check(pages, q, out, first, chunk)
        untouched[first:first + chunk] = False
    assert bool((out.cpu()[torch.from_numpy(untouched)] == 5.0).all())
