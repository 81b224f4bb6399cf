"""Shared-prefix decode attention carries its weights to 16 bits in both of its forms, as the other decode calls do: the
bound of plain64.attend without the term for weights in one bf16 part.  So what a sequence gets does not depend, beyond
the output's own rounding, on the table's width or on the other sequences of the batch, which choose the form and the
splits.  Prefixes are short here: the fewer keys, the less the weights' roundings cancel."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from plain64 import BLOCK, Pages, assert_within, attend, f64, sees

pytestmark = pytest.mark.gpu


def bound(pages, q, lens, scale):
    qf, kf, vf = f64(q), f64(pages.k), f64(pages.v)
    rows = [attend(qf[b], kf, vf, pages.table[b], sees(n - 1), scale, 0.0) for b, n in enumerate(lens)]
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


def call(pages, q, starts, prefixes, scale):
    kc, vc, table, cl = pages.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.paged_prefix_decode_attention(q.cuda(), kc, vc, table, cl, torch.tensor(starts, **i32),
                                      torch.tensor(prefixes, **i32), scale, out)
    assert device_errors() == 0
    return out


def shared(pages, groups):
    for first, rows, prefix in groups:
        pages.table[first:first + rows, :prefix // BLOCK] = pages.table[first, :prefix // BLOCK]


@pytest.mark.parametrize("width", [None, 4000], ids=["narrow", "wide"])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (4, 2, 128), (8, 2, 128), (16, 2, 128), (2, 2, 64), (16, 2, 64)])
@pytest.mark.parametrize("prefix", [16, 48, 128, 400])
def test_weights_in_two_parts(prefix, hq, hkv, d, width):
    rows = 40
    lens = [prefix + b % 3 for b in range(rows)]
    pages = Pages(lens, hkv, d, prefix + hq, width=width)
    shared(pages, [(0, rows, prefix)])
    q = pages.randn(rows, hq, d)
    out = call(pages, q, [0, rows], [prefix], d ** -0.5)
    assert_within(out, *bound(pages, q, lens, d ** -0.5), f"prefix {prefix} {hq}/{hkv} D{d}")


def test_a_sequence_in_other_batches():
    """Four sequences behind 304 tokens: alone, in a wide table, and before and between groups with longer prefixes (other
    split lengths)."""
    mine, prefix, scale = [305, 310, 304, 333], 304, 128 ** -0.5
    for others, width in (([], None), ([], 4000), ([2000] * 30, 4000), ([9000] * 3, 4000)):
        lens = mine + [n + b for b, n in enumerate(others)]
        pages = Pages(lens, 2, 128, 5, width=width)
        groups = [(0, 4, prefix)] + ([(4, len(others), others[0])] if others else [])
        shared(pages, groups)
        q = pages.randn(len(lens), 16, 128)
        out = call(pages, q, [g[0] for g in groups] + [len(lens)], [g[2] for g in groups], scale)
        ref, allowed = bound(pages, q[:4], mine, scale)
        assert_within(out[:4], ref, allowed, f"with {len(others)} others")
