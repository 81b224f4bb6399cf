"""Chunk attention over the 8-bit cache with tables that are wider than their sequences (as wide as the longest context that is
served): short prompts are not unpacked because their table could hold long ones, and long ones are whatever it could hold."""
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors

pytestmark = pytest.mark.gpu


def unpacks(chunk, width, seqs=1, hq=32, hkv=8, d=128):
    sizes = seqs * chunk, chunk, seqs, hq, hkv, d, width
    blocks = 4 * seqs * width * 16 * hkv * d
    more = pkv.fp8_prefill_workspace_size(*sizes) - pkv.fp8_prefill_workspace_size(*sizes, unpack=False)
    assert more == 0 or more >= blocks
    return more > 0


@pytest.mark.parametrize("width", [32, 64, 257, 2048, 8192])
@pytest.mark.parametrize("chunk,seqs,d", [(512, 1, 128), (300, 3, 128), (700, 1, 64), (512, 8, 128)])
def test_a_short_prompt(width, chunk, seqs, d):
    # (Eight of 512 tokens behind up to 3584 are unpacked if the table was made for that; these tables are narrower or wider.)
    assert not unpacks(chunk, width, seqs, d=d)


@pytest.mark.parametrize("chunk,width,seqs", [(8192, 512, 2), (8192, 8192, 2), (2048, 128, 1), (2048, 8192, 1), (1024, 64, 8),
                                              (1024, 2000, 8), (2048, 640, 2), (512, 256, 8)])
def test_long_ones(chunk, width, seqs):
    assert unpacks(chunk, width, seqs)


def test_results_do_not_go_by_the_width():
    from test_gpu_fp8_unpacked import Case

    narrow = Case((100,), (600,), 32, 8, 128, seed=2)
    wide = Case((100,), (600,), 32, 8, 128, seed=2, width=8192)
    assert torch.equal(narrow.dq, wide.dq)
    a, b = narrow.call(), wide.call()
    narrow.check(a)
    wide.check(b)
    assert device_errors() == 0
