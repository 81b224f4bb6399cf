"""The workspace of chunk attention over the 8-bit cache: what is enough for a batch of drafted tokens is enough for smaller
ones and for narrower tables."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from fp8_plain import Fp8Pages, attend_fp8
from gpu_util import device_errors
from plain64 import assert_within, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,most", [(1, 1, 128, 3), (8, 1, 128, 3), (2, 2, 64, 8), (32, 8, 128, 6), (32, 8, 128, 2), (16, 2, 64, 1)])
def test_sizes_of_drafted_tokens_do_not_fall(hq, hkv, d, most):
    sizes = [[pkv.fp8_prefill_workspace_size(n * most, most, n, hq, hkv, d, width)
              for n in (1, 2, 3, 4, 5, 8, 12, 16, 19, 20, 37, 38, 64, 75, 76, 77, 152, 153, 304, 305, 1024, 1025)]
             for width in (1, 8, 60, 100, 300, 410, 512, 700, 800, 1000, 2000, 4000, 20000)]
    assert (np.diff(sizes, axis=0) >= 0).all() and (np.diff(sizes, axis=1) >= 0).all()
    assert sizes[0][0] == 0 and sizes[-1][0] > 0  # (both forms)


def test_one_workspace_for_all_batches_of_drafts():
    """Lengths that one sequence takes in the stream and more in clusters: every batch with the largest one's workspace."""
    lens, width, most = (6000, 9000), 800, 2
    pages = Fp8Pages(lens, 1, 128, 3, width=width)
    sizes = [pkv.fp8_prefill_workspace_size(n * most, most, n, 1, 1, 128, width) for n in range(1, 9)]
    space = torch.empty(max(16, sizes[-1]), dtype=torch.uint8, device="cuda")
    q = pages.randn(8 * most, 1, 128)
    kc, vc, sc, table, cl = pages.cuda()
    for n in range(1, 9):
        start = torch.arange(n + 1, dtype=torch.int32, device="cuda") * most
        out = torch.empty(n * most, 1, 128, dtype=torch.bfloat16, device="cuda")
        pkv.paged_fp8_prefill_attention(q[:n * most].cuda(), kc, vc, sc, table.repeat(4, 1)[:n], cl.repeat(4)[:n], start, most, 0.1,
                                        out, workspace=space)
        for row in range(n * most):
            b = row // most
            seen = lens[b % 2] - most + row % most + 1
            assert_within(out[row], *attend_fp8(pages, b % 2, f64(q[row]), seen, 0.1, 2.0**-11), f"{n} sequences, row {row}")
    assert device_errors() == 0
