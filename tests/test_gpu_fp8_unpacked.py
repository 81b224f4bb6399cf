"""Chunk attention over the 8-bit cache where the cache is turned into bf16 ahead of it (long chunks): rows against the
definition in 64 bits, and all of them against the kernel that converts as it goes, bit for bit.  A call with more rows of q
than its chunks could hold takes the latter."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from fp8_plain import Fp8Pages, attend_fp8
from gpu_util import device_errors
from plain64 import BLOCK, assert_within, f64

pytestmark = pytest.mark.gpu

SCALE = 0.09


class Case:
    def __init__(self, pasts, chunks, hq, hkv, d, seed=0, width=None):
        self.chunks, self.most, self.hq, self.hkv, self.d = list(chunks), max(chunks), hq, hkv, d
        self.pages = Fp8Pages([p + c for p, c in zip(pasts, chunks)], hkv, d, seed, width=width)
        self.start = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
        self.q = self.pages.randn(int(self.start[-1]), hq, d)
        self.dq, self.dstart = self.q.cuda(), torch.from_numpy(self.start).cuda()
        self.caches = list(self.pages.cuda())
        n = len(chunks)
        self.unpacked = 4 * n * self.caches[3].shape[1] * BLOCK * hkv * d
        self.need = pkv.fp8_prefill_workspace_size(len(self.q), self.most, n, hq, hkv, d, self.caches[3].shape[1])
        self.padded = n * self.most + 1  # rows of q with which a call does not unpack

    def call(self, **kw):
        out = torch.full_like(self.dq, float("nan"))
        return pkv.paged_fp8_prefill_attention(self.dq, *self.caches, self.dstart, self.most, SCALE, out, **kw)

    def without(self):
        q = torch.zeros(self.padded, self.hq, self.d, dtype=torch.bfloat16, device="cuda")
        q[:len(self.q)] = self.dq
        need = pkv.fp8_prefill_workspace_size(len(q), self.most, len(self.chunks), self.hq, self.hkv, self.d,
                                              self.caches[3].shape[1])
        assert need < self.unpacked
        out = torch.full_like(q, float("nan"))
        pkv.paged_fp8_prefill_attention(q, *self.caches, self.dstart, self.most, SCALE, out)
        assert torch.isnan(out[len(self.q):].float()).all()
        return out[:len(self.q)]

    def check(self, out, seed=0, rows=60):
        r = np.random.RandomState(seed)
        picked = set(r.randint(0, len(self.q), rows)) | {0, len(self.q) - 1} | {int(x) for x in self.start[:-1] if x < len(self.q)}
        for row in sorted(picked):
            b = int(np.searchsorted(self.start, row, side="right")) - 1
            n = self.pages.lens[b] - self.chunks[b] + row - int(self.start[b]) + 1
            ref, allowed = attend_fp8(self.pages, b, f64(self.q[row]), n, SCALE, 2.0**-8)
            assert_within(out[row], ref, allowed, f"row {row}")


CASES = [((0, 0, 0, 0), (1500, 1500, 1500, 1500), 16, 2, 128), ((0, 5, 300, 0, 77), (2000, 1, 1333, 0, 1900), 16, 2, 64),
         ((0,) * 6, (1000, 900, 1001, 17, 999, 1000), 32, 8, 128), ((100, 0), (4000, 3333), 8, 2, 128), ((0, 40), (3000, 2900), 6, 6, 64),
         ((3000, 2000), (1025, 1024), 16, 4, 128), ((0,), (5000,), 8, 1, 128)]


@pytest.mark.parametrize("pasts,chunks,hq,hkv,d", CASES)
def test_rows(pasts, chunks, hq, hkv, d):
    case = Case(pasts, chunks, hq, hkv, d, seed=len(chunks))
    takes = case.need >= case.unpacked
    out = case.call()
    assert not torch.isnan(out.float()).any() and device_errors() == 0
    case.check(out)
    assert torch.equal(out, case.without()) or not takes
    assert device_errors() == 0
    assert takes == ((hq, hkv) not in ((32, 8), (6, 6)))  # (these have too few rows, and convert as they go)


def test_what_no_row_sees_does_not_matter():
    case = Case((0, 30, 0), (1999, 1500, 1777), 16, 2, 128, seed=3, width=140)
    assert case.need >= case.unpacked
    a = case.call()
    table = case.caches[3]
    table[table < 0] = 1 << 30
    space = torch.full((case.need,), 0xFF, dtype=torch.uint8, device="cuda")
    b = case.call(workspace=space)
    assert torch.equal(a, b) and device_errors() == 0
    with pytest.raises(ValueError, match="workspace"):
        case.call(workspace=space[:-1])


def test_a_row_that_is_not_a_number_spoils_its_sequence():
    case = Case((0, 0, 0), (1500, 1600, 1700), 16, 2, 128, seed=4)
    assert case.need >= case.unpacked
    a = case.call()
    case.caches[1].view(torch.uint8)[case.pages.table[1, 0], :, 3] = 0x7F
    b = case.call()
    assert torch.isnan(b[1500 + 3:3100].float()).all()
    assert torch.equal(a[:1500], b[:1500]) and torch.equal(a[3100:], b[3100:])
    assert device_errors() == 0


def test_bad_chunks_and_blocks_are_flagged_and_skipped():
    case = Case((0, 0, 0), (1500, 1600, 1700), 16, 2, 128, seed=5)
    assert case.need >= case.unpacked
    whole = case.call()
    lens, start = case.caches[4], case.dstart
    for bad in (-3, 1599, case.caches[3].shape[1] * BLOCK + 1):  # negative, shorter than its chunk, longer than its table
        case.caches[4] = lens.clone()
        case.caches[4][1] = bad
        out = case.call()
        assert device_errors() == pkv.DEVERR_CONTEXT_LEN_TOO_LONG
        assert torch.equal(out[:1500], whole[:1500]) and torch.equal(out[3100:], whole[3100:])
        assert torch.isnan(out[1500:3100].float()).all()
    case.caches[4] = lens
    for starts in ([0, 1500, 3100, 4801], [-1, 1500, 3100, 4800], [0, 1500, 1400, 2800], [0, -2**31, 2**31 - 1, 4800]):
        case.dstart = torch.tensor(starts, dtype=torch.int32, device="cuda")
        case.call()
        assert device_errors() == pkv.DEVERR_CONTEXT_LEN_TOO_LONG
    case.dstart = start
    table = case.caches[3].clone()
    table[2, 5] = 1 << 20
    case.caches[3] = table
    case.call()
    assert device_errors() == pkv.DEVERR_BLOCK_ID_OUT_OF_RANGE


def test_same_bits_again_and_in_a_graph():
    case = Case((0, 100, 0), (1500, 1600, 1700), 16, 2, 128, seed=6)
    assert case.need >= case.unpacked
    first, out = case.call(), torch.empty_like(case.dq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_fp8_prefill_attention(case.dq, *case.caches, case.dstart, case.most, SCALE, out)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    # Other lengths and rows of the cache in the same graph (the last sequence then sees two rows that are not numbers).
    case.caches[4].copy_(torch.tensor([1500, 1650, 1702], dtype=torch.int32))
    case.caches[0].view(torch.uint8)[:, :, ::3] ^= 0x80
    want = case.call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert not torch.equal(out[:3100], first[:3100]) and not torch.isnan(out[:3100].float()).any()
    assert device_errors() == 0
