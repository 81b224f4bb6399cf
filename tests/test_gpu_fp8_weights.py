"""What a sequence gets from the few-row attention over the 8-bit cache does not depend, beyond 32-bit arithmetic and the
output's own rounding, on how its batch is cut into pieces: alone in a cluster, alone in the stream, in the middle of a batch,
and as a chunk's one row beside sequences with more of them.

Softmax weights enter the product with V as fp16.  Against references that are whole numbers (base 2) a weight's eleven bits are
the same whatever the reference, so that two cuts differ where 32-bit arithmetic does, by about 2^-22 of sum p |v|.  With n
keys of independent values that is 2^-22 sqrt(n) of a result, against steps of 2^-8 of it and more: 0.1 % of the results round
to the other side with 300 keys.  A weight whose 32 bits differ so may round to the other eleven, one in 2^11, which moves a
result by 2^-10 / sqrt(n) of itself: less than another 0.1 %.  Ten times that is allowed.  References that are not whole
numbers round every weight anew: 2^-11 of itself at most, 4e-4 of a result between two cuts, and 5 % of the results differ.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from fp8_plain import Fp8Pages, attend_fp8
from gpu_util import device_errors
from plain64 import assert_within, f64

pytestmark = pytest.mark.gpu

MINE = (300, 77, 513, 160)


def in_a_batch(caches, q, order, table, lens, scale):
    """The rows of q in the given order, and then back in their own."""
    at = torch.from_numpy(order).cuda()
    out = torch.empty_like(q)
    pkv.paged_fp8_decode_attention(q[at].contiguous(), *caches, table[at].contiguous(), lens[at].contiguous(), scale, out)
    back = torch.empty_like(out)
    back[at] = out
    return back


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (16, 2, 128), (16, 4, 64), (3, 3, 64)])
def test_a_sequence_in_other_batches(hq, hkv, d):
    r = np.random.RandomState(hq)
    lens = list(MINE) + list(r.randint(1, 700, 200))
    pages = Fp8Pages(lens, hkv, d, hq)
    q, scale, n = pages.randn(len(lens), hq, d).cuda(), d ** -0.5, len(MINE)
    kc, vc, sc, table, cl = pages.cuda()
    caches = kc, vc, sc
    wide = torch.full((1, 20000), -1, dtype=torch.int32, device="cuda")
    outs = {"alone": [], "in the stream": [], "beside longer chunks": []}
    for b in range(n):
        out = torch.empty_like(q[:1])
        pkv.paged_fp8_decode_attention(q[b:b + 1], *caches, table[b:b + 1], cl[b:b + 1], scale, out)
        outs["alone"].append(out)
        wide[0, :table.shape[1]] = table[b]
        outs["in the stream"].append(pkv.paged_fp8_decode_attention(q[b:b + 1], *caches, wide, cl[b:b + 1], scale, torch.empty_like(out)))
        # The query of a chunk of one token, in a call whose chunks may have up to 24 rows.
        start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        outs["beside longer chunks"].append(pkv.paged_fp8_prefill_attention(
            q[b:b + 1], *caches, table[b:b + 1], cl[b:b + 1], start, 24 // (hq // hkv), scale, torch.empty_like(out)))
    outs = {k: torch.cat(v) for k, v in outs.items()}
    outs["first of a batch"] = in_a_batch(caches, q, np.arange(len(lens)), table, cl, scale)[:n]
    outs["amid a batch"] = in_a_batch(caches, q, r.permutation(len(lens)), table, cl, scale)[:n]
    assert device_errors() == 0
    for b in range(n):
        ref, allowed = attend_fp8(pages, b, f64(q[b]), MINE[b], scale, 2.0**-11)
        for what, out in outs.items():
            assert_within(out[b], ref, allowed, f"{what}, sequence {b}")
    differ = {what: float((out.view(torch.int16) != outs["alone"].view(torch.int16)).float().mean()) for what, out in outs.items()}
    print(hq, hkv, d, differ)
    assert max(differ.values()) <= 0.02, differ


@pytest.mark.parametrize("spread", [1.0, 4.0])
def test_rows_of_different_sizes(spread):
    """Weights that take V's exponents with them, over many powers of two."""
    lens = list(MINE) * 60
    pages = Fp8Pages(lens, 4, 128, 7, spread=spread)
    pages.table[:] = np.concatenate([pages.table[:4]] * 60)
    q = pages.randn(4, 16, 128).repeat(60, 1, 1).cuda()
    kc, vc, sc, table, cl = pages.cuda()
    out = pkv.paged_fp8_decode_attention(q, kc, vc, sc, table, cl, 2.0**-6, torch.empty_like(q))
    assert device_errors() == 0
    bits = out.view(torch.int16).view(60, 4, 16, 128)
    differ = float((bits != bits[:1]).float().mean())
    print(spread, differ)
    assert differ <= 0.02
