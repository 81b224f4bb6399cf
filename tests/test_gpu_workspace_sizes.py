"""A workspace sized for a caller's largest batch serves its smaller ones, whichever form they take: the sizes of the
windowed and the shared-prefix decode do not fall with the number of sequences or the width of the table."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from plain64 import Pages, assert_within, attend, f64, sees

pytestmark = pytest.mark.gpu
SEQS = [1, 2, 3, 5, 7, 8, 9, 12, 16, 18, 19, 20, 24, 36, 37, 38, 40, 64, 75, 76, 77, 100, 151, 152, 153, 200, 303, 304, 305,
        400, 600, 1000, 1500, 2000, 2500, 3000, 3500, 4000, 4095, 4096]


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 128), (8, 1, 128), (2, 2, 64), (32, 8, 128), (64, 8, 64)])
def test_window_decode_sizes_do_not_fall(hq, hkv, d):
    for window in (1, 500, 4000, 17000, 18000, 20000):
        sizes = [[pkv.window_decode_workspace_size(n, hq, hkv, d, width, window, 4) for n in SEQS + [4097, 9000]]
                 for width in (1, 30, 100, 300, 900, 1080, 1100, 1200, 1300, 2000, 4000)]
        assert (np.diff(sizes, axis=0) >= 0).all() and (np.diff(sizes, axis=1) >= 0).all(), window


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 128), (8, 1, 128), (2, 2, 64), (32, 8, 128), (64, 8, 64)])
def test_prefix_decode_sizes_do_not_fall(hq, hkv, d):
    sizes = np.array([[[pkv.prefix_decode_workspace_size(n, hq, hkv, d, width, groups) for n in SEQS]
                       for width in (1, 30, 100, 300, 900, 2000)] for groups in (0, 1, 4, 100, 4096)])
    for axis in range(3):
        assert (np.diff(sizes, axis=axis) >= 0).all()


@pytest.mark.parametrize("width", [1000, 1100, 1200, 1400])
def test_one_workspace_for_all_batches(width):
    """Windows that a few sequences take in pieces and more in clusters: every batch with the largest one's workspace."""
    lens = [16 * width - 3 * b for b in range(2)]
    pages = Pages(lens, 1, 128, width)
    kc, vc, table, cl = pages.cuda()
    q = pages.randn(8, 1, 128)
    qf, kf, vf = f64(q), f64(pages.k), f64(pages.v)
    rows = [attend(qf[b], kf, vf, pages.table[b % 2], sees(lens[b % 2] - 1), 0.1, 0.0) for b in range(8)]
    ref, allowed = np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])
    need = pkv.window_decode_workspace_size(8, 1, 1, 128, width, 16 * width, 0)
    space = torch.empty(need, dtype=torch.uint8, device="cuda")
    for n in range(1, 9):
        out = torch.empty(n, 1, 128, dtype=torch.bfloat16, device="cuda")
        pkv.paged_window_decode_attention(q[:n].cuda(), kc, vc, table.repeat(4, 1)[:n], cl.repeat(4)[:n], 0.1, out,
                                          16 * width, 0, workspace=space)
        assert_within(out, ref[:n], allowed[:n], f"{n} sequences")
    assert device_errors() == 0
