"""Chunk attention over the 8-bit cache at sizes that take its rarer paths: unpacked and split over keys, more sequences than a
CTA ranks, batches in slices, and caches whose rows lie behind 2^32 bytes."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from fp8_plain import FP8, Fp8Pages, attend_fp8
from gpu_util import device_errors
from plain64 import BLOCK, assert_within, f64

pytestmark = pytest.mark.gpu

SCALE = 0.09


class Case:
    def __init__(self, pasts, chunks, hq, hkv, d, seed=0):
        self.chunks, self.most, self.hq, self.hkv, self.d = list(chunks), max(chunks), hq, hkv, d
        self.pages = Fp8Pages([p + c for p, c in zip(pasts, chunks)], hkv, d, seed)
        self.start = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
        self.q = self.pages.randn(int(self.start[-1]), hq, d)
        self.caches = list(self.pages.cuda())
        n, width = len(chunks), self.pages.width
        sizes = len(self.q), self.most, n, hq, hkv, d, width
        self.states = pkv.fp8_prefill_workspace_size(*sizes, unpack=False)  # of splits, or pieces
        self.unpacks = pkv.fp8_prefill_workspace_size(*sizes) >= self.states + 4 * n * width * BLOCK * hkv * d

    def call(self):
        out = torch.full_like(self.q, float("nan"), device="cuda")
        pkv.paged_fp8_prefill_attention(self.q.cuda(), *self.caches, torch.from_numpy(self.start).cuda(), self.most, SCALE, out)
        assert device_errors() == 0
        return out

    def check(self, out, rows, weight):
        assert not torch.isnan(out.float()).any()
        picked = set(np.random.RandomState(1).randint(0, len(self.q), rows)) | {0, len(self.q) - 1}
        for row in sorted(picked):
            b = int(np.searchsorted(self.start, row, side="right")) - 1
            n = self.pages.lens[b] - self.chunks[b] + row - int(self.start[b]) + 1
            assert_within(out[row], *attend_fp8(self.pages, b, f64(self.q[row]), n, SCALE, weight), f"row {row}")


@pytest.mark.parametrize("past,chunk,hq,hkv,d", [(4096, 1024, 16, 2, 128), (4001, 1027, 16, 2, 128), (5012, 1100, 16, 2, 64)])
def test_unpacked_and_split(past, chunk, hq, hkv, d):
    case = Case((past,), (chunk,), hq, hkv, d, chunk)
    assert case.unpacks and case.states >= 2 * chunk * hq * (d + 2) * 4  # (of two splits)
    out = case.call()
    case.check(out, 60, 2.0**-8)
    assert torch.equal(out, case.call())


def test_more_sequences_than_a_cta_ranks():
    r = np.random.RandomState(3)
    chunks = r.randint(0, 17, 600)
    chunks[5] = 16  # 32 rows of two heads: more than the few-row kernel takes
    case = Case(r.randint(0, 150, 600), chunks, 2, 1, 64, 3)
    assert case.most * 2 > 24 and not case.unpacks
    case.check(case.call(), 300, 2.0**-8)


@pytest.mark.parametrize("most,hq", [(3, 2), (3, 8)])
def test_drafted_tokens_of_a_batch_in_slices(most, hq):
    r = np.random.RandomState(most + hq)
    chunks = r.randint(0, most + 1, 2100)
    case = Case(r.randint(0, 60, 2100), chunks, hq, 1, 64, 4)
    assert case.most * hq <= 24
    before = pkv.kernel_launch_count()
    out = case.call()
    assert pkv.kernel_launch_count() - before == 2 * 3  # slices of 1024 sequences, two kernels each
    case.check(out, 300, 2.0**-11)


@pytest.mark.parametrize("past,chunk,form", [(300, 3, "few rows"), (300, 40, "converts"), (0, 2500, "unpacks")])
def test_a_large_cache(past, chunk, form):
    """Blocks whose rows lie behind 2^32 bytes."""
    nb = 270_000
    case = Case((past,) * 2, (chunk,) * 2, 16, 8, 128, chunk)
    assert case.unpacks == (form == "unpacks")
    shift, pages = nb - case.pages.pool, case.pages
    big = [torch.zeros(nb, *x.shape[1:], dtype=torch.uint8, device="cuda") for x in (pages.k8, pages.v8, pages.scales)]
    assert big[0].numel() > 1 << 32
    for dst, src in zip(big, (pages.k8, pages.v8, pages.scales)):
        dst[shift:] = src.view(torch.uint8).cuda()
    case.caches[:4] = big[0].view(FP8), big[1].view(FP8), big[2], torch.from_numpy(pages.table + shift).cuda()
    case.check(case.call(), 40, 2.0**-8)
