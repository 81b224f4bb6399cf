"""Softmax weights of the few-row attention over the 8-bit cache.

Decode carries them to 16 bits and more, as the other decode calls do: the bound of fp8_plain.attend_fp8 without a term for
weights that were rounded (its 2^-16 is the second part's).

Chunks of more rows have eleven bits, half a step 2^-11 of a weight; the normaliser sums the same ones, so that both the
product and its normaliser may be off by that.

And what a sequence gets does not depend, beyond 32-bit arithmetic and the output's own rounding, on how its batch is cut into
pieces: alone in a cluster, alone in the stream, first or in the middle of a batch.  Against references that are whole numbers
(base 2) a weight's bits are the same whatever the reference, so that two cuts differ where 32-bit arithmetic does, by about
2^-22 of sum p |v|.  With n keys of independent values that is 2^-22 sqrt(n) of a result, against steps of 2^-8 of it and more:
0.1 % of the results round to the other side with 300 keys.  A weight whose 32 bits differ so may round to other eleven, one in
2^11, which moves a result by 2^-10 / sqrt(n) of itself: less than another 0.1 %.  Ten times that is allowed.  References that
are not whole numbers round every weight anew: 2^-11 of itself at most, 4e-4 of a result between two cuts, and 5 % of the
results differ.
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


class Batch:
    """Sequences of which the first are looked at; one query token each, as decode or as chunks of a call that allows more."""

    def __init__(self, hq, hkv, d, drafts):
        r = np.random.RandomState(hq)
        self.lens = list(MINE) + list(r.randint(1, 700, 200))
        self.pages = Fp8Pages(self.lens, hkv, d, hq)
        self.q = self.pages.randn(len(self.lens), hq, d).cuda()
        *self.caches, self.table, self.cl = self.pages.cuda()
        self.scale, self.most = d ** -0.5, 24 // (hq // hkv) if drafts else 0
        self.shuffled = torch.from_numpy(r.permutation(len(self.lens))).cuda()

    def call(self, rows, wide=False):
        q, table, cl = (x[rows].contiguous() for x in (self.q, self.table, self.cl))
        if wide:
            table = torch.nn.functional.pad(table, (0, 20000 - table.shape[1]), value=-1)
        out = torch.empty_like(q)
        if not self.most:
            return pkv.paged_fp8_decode_attention(q, *self.caches, table, cl, self.scale, out)
        start = torch.arange(len(q) + 1, dtype=torch.int32, device="cuda")
        return pkv.paged_fp8_prefill_attention(q, *self.caches, table, cl, start, self.most, self.scale, out)


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (16, 2, 128), (16, 4, 64), (3, 3, 64)])
@pytest.mark.parametrize("drafts", [False, True], ids=["decode", "drafts"])
def test_a_sequence_in_other_batches(hq, hkv, d, drafts):
    batch, n = Batch(hq, hkv, d, drafts), len(MINE)
    outs = {"alone": torch.cat([batch.call(slice(b, b + 1)) for b in range(n)]),
            "in the stream": torch.cat([batch.call(slice(b, b + 1), wide=True) for b in range(n)]),
            "first of a batch": batch.call(slice(None))[:n]}
    back = torch.empty_like(batch.q)
    back[batch.shuffled] = batch.call(batch.shuffled)
    outs["amid a batch"] = back[:n]
    assert device_errors() == 0
    for b in range(n):
        ref, allowed = attend_fp8(batch.pages, b, f64(batch.q[b]), MINE[b], batch.scale, 2.0**-10 if drafts else 0.0)
        for what, out in outs.items():
            assert_within(out[b], ref, allowed, f"{what}, sequence {b}")
    differ = {what: float((out.view(torch.int16) != outs["alone"].view(torch.int16)).float().mean()) for what, out in outs.items()}
    print(hq, hkv, d, differ)
    assert max(differ.values()) <= 0.02, differ


@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (4, 2, 128), (16, 2, 128), (2, 2, 64), (16, 2, 64)])
@pytest.mark.parametrize("seqs", [3, 400])  # in clusters and in the stream
def test_weights_of_decode(hq, hkv, d, seqs):
    """Few keys, whose weights' roundings cancel least, and a few more."""
    lens = [2 + b % 61 for b in range(seqs)]
    pages = Fp8Pages(lens, hkv, d, hq + seqs)
    q = pages.randn(seqs, hq, d)
    kc, vc, sc, table, cl = pages.cuda()
    out = pkv.paged_fp8_decode_attention(q.cuda(), kc, vc, sc, table, cl, d ** -0.5, torch.empty(q.shape, dtype=q.dtype, device="cuda"))
    assert device_errors() == 0
    for b, n in enumerate(lens):
        assert_within(out[b], *attend_fp8(pages, b, f64(q[b]), n, d ** -0.5, 0.0), f"sequence {b}")


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
