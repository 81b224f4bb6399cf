"""Chunk attention over the 8-bit cache on the GPU against the definition in 64 bits (bounds: fp8_plain.attend_fp8; a weight
may be rounded to bf16 before the product with V, half a step 2^-8, while the denominator sums the weights in 32 bits)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from fp8_plain import Fp8Pages, attend_fp8
from gpu_util import device_errors
from plain64 import assert_within, f64

pytestmark = pytest.mark.gpu

WEIGHT = 2.0**-8


def exact_rows(pages, q, chunks, scale):
    qf = f64(q)
    out, allowed, at = [], [], 0
    for b, c in enumerate(chunks):
        for i in range(c):
            o, a = attend_fp8(pages, b, qf[at], pages.lens[b] - c + i + 1, scale, WEIGHT)
            out.append(o)
            allowed.append(a)
            at += 1
    return np.stack(out), np.stack(allowed)


def starts(chunks):
    return torch.tensor(np.concatenate([[0], np.cumsum(chunks)]), dtype=torch.int32, device="cuda")


def run(pasts, chunks, hq, hkv, d, seed=0, scale=None, most=None, pages=None, spread=1.0, behind=3, **kw):
    lens = [p + c for p, c in zip(pasts, chunks)]
    pages = pages or Fp8Pages(lens, hkv, d, seed, spread=spread)
    scale = d ** -0.5 if scale is None else scale
    rows = int(sum(chunks))
    q = pages.randn(rows + behind, hq, d)
    kc, vc, sc, table, cl = pages.cuda()
    out = torch.full((rows + behind, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = pkv.paged_fp8_prefill_attention(q.cuda(), kc, vc, sc, table, cl, starts(chunks), most or max(chunks), scale, out, **kw)
    assert got is out
    assert (out[rows:] == 7.0).all(), "rows behind the last sequence"
    ref, allowed = exact_rows(pages, q, chunks, scale)
    assert_within(out[:rows], ref, allowed, f"{hq}/{hkv} D{d} {pasts} {chunks}")
    assert device_errors() == 0
    return out[:rows]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (4, 1), (8, 1), (4, 2), (16, 2), (3, 3), (24, 3), (10, 5), (8, 8), (12, 12)])
def test_layouts(hq, hkv, d):
    run((0, 1, 17, 40, 130), (5, 33, 1, 20, 64), hq, hkv, d, seed=hq)


@pytest.mark.parametrize("chunk", list(range(1, 20)) + [31, 32, 33, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (8, 1)])
def test_every_chunk_length(chunk, hq, hkv):
    run((0, 100), (chunk, max(1, chunk // 2)), hq, hkv, 64, seed=chunk)


@pytest.mark.parametrize("chunk", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (4, 1), (8, 1), (12, 3), (16, 2), (32, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_drafted_tokens(chunk, hq, hkv, d):
    """A few rows a sequence over caches of very different lengths, among them sequences without rows."""
    pasts = (0, 1, 7, 12, 16, 250, 1111, 3000, 0)
    chunks = [max(0, chunk - i % 4) for i in range(len(pasts) - 1)] + [0]
    chunks[2] = chunk
    run(pasts, chunks, hq, hkv, d, seed=chunk, most=chunk)


@pytest.mark.parametrize("past,chunk", [(0, 1), (4000, 1), (4000, 40), (9000, 130), (0, 1500), (127, 129), (128, 128)])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (16, 2)])
def test_one_sequence(past, chunk, hq, hkv):
    run((past,), (chunk,), hq, hkv, 128, seed=past + chunk)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,most", [(8, 8, 9), (8, 8, 17), (8, 8, 24), (32, 8, 4), (32, 8, 6), (12, 6, 12), (16, 2, 3), (8, 4, 8),
                                         (2, 1, 12)])
def test_more_pairs_than_clusters(hq, hkv, most, d):
    """Chunks of up to 24 rows, more (sequence, kv head) pairs than the GPU holds clusters for, some of them long."""
    r = np.random.RandomState(most)
    n = 310 // hkv + 1
    run(r.randint(0, 90, n) + (r.rand(n) < 0.1) * 1500, np.append(r.randint(0, most + 1, n - 1), most), hq, hkv, d, most=most)


def test_many_sequences():
    r = np.random.RandomState(1)
    chunks = r.randint(0, 9, 700)
    run(r.randint(0, 60, 700), chunks, 2, 1, 64, most=9)


@pytest.mark.parametrize("seed", range(6))
def test_random_shapes(seed):
    r = np.random.RandomState(seed)
    hkv = int(r.choice([1, 2, 3, 4]))
    n = r.randint(1, 7)
    run(r.randint(0, 400, n), r.randint(1, 200, n), hkv * int(r.choice([1, 2, 4, 8])), hkv, int(r.choice([64, 128])), seed=seed)


@pytest.mark.parametrize("chunks", [(3, 2, 1), (30, 20, 70)])
def test_rows_of_very_different_sizes(chunks):
    run((5, 100, 40), chunks, 8, 2, 128, seed=5, spread=8.0, scale=2.0**-7)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 3.0])
@pytest.mark.parametrize("chunks", [(2, 4), (70, 33)])
def test_scales(scale, chunks):
    run((40, 90), chunks, 8, 2, 64, seed=4, scale=scale)


@pytest.mark.parametrize("chunk", [1, 3, 40, 200])
def test_a_chunk_of_one_and_decode_agree(chunk):
    """A chunk's last row sees what a decode call's query sees; both are within their bounds of the exact result."""
    pages = Fp8Pages((300 + chunk,), 2, 128, 8)
    q = pages.randn(chunk, 8, 128)
    kc, vc, sc, table, cl = pages.cuda()
    out, one = torch.empty_like(q).cuda(), torch.empty(1, 8, 128, dtype=torch.bfloat16, device="cuda")
    pkv.paged_fp8_prefill_attention(q.cuda(), kc, vc, sc, table, cl, starts([chunk]), chunk, 0.09, out)
    pkv.paged_fp8_decode_attention(q[-1:].cuda(), kc, vc, sc, table, cl, 0.09, one)
    ref, allowed = attend_fp8(pages, 0, f64(q)[-1], 300 + chunk, 0.09, WEIGHT)
    assert_within(out[-1], ref, allowed, "chunk")
    assert_within(one[0], ref, allowed, "decode")
    assert device_errors() == 0


@pytest.mark.parametrize("chunk", [2, 90])
def test_what_no_row_sees_does_not_matter(chunk):
    pages = Fp8Pages((5 + chunk, chunk), 2, 128, 7, width=20)
    kw = dict(pages=pages)
    a = run((5, 0), (chunk, chunk), 8, 2, 128, **kw)
    pages.g.manual_seed(0)
    b = run((5, 0), (chunk, chunk), 8, 2, 128, **kw)
    pages.table[pages.table < 0] = -(1 << 30)
    pages.g.manual_seed(0)
    c = run((5, 0), (chunk, chunk), 8, 2, 128, **kw)
    assert a.shape == b.shape and torch.equal(b, c)


@pytest.mark.parametrize("chunk", [2, 40])
def test_a_row_that_is_not_a_number_spoils_the_sequence_that_sees_it(chunk):
    pages = Fp8Pages((200 + chunk, 40 + chunk), 1, 128, 9)
    q = pages.randn(2 * chunk, 8, 128)
    ref, allowed = exact_rows(pages, q, (chunk, chunk), 0.09)
    pages.k8.view(torch.uint8)[pages.table[0, 5], :, 3] = 0x7F
    kc, vc, sc, table, cl = pages.cuda()
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.paged_fp8_prefill_attention(q.cuda(), kc, vc, sc, table, cl, starts([chunk, chunk]), chunk, 0.09, out)
    assert torch.isnan(out[:chunk].float()).all()
    assert_within(out[chunk:], ref[chunk:], allowed[chunk:], "the other")
    assert device_errors() == 0


@pytest.mark.parametrize("chunk", [3, 70])
def test_bad_chunks_and_blocks_are_flagged(chunk):
    """A sequence whose chunk is longer than its context, or reaches outside the rows, is skipped; the other is computed."""
    pages = Fp8Pages((chunk + 9, chunk + 20), 2, 64, 3)
    q = pages.randn(2 * chunk, 4, 64)
    kc, vc, sc, table, cl = pages.cuda()
    ref, allowed = exact_rows(pages, q, (chunk, chunk), 0.1)

    def call(lens, qs, most=chunk, tab=table):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        pkv.paged_fp8_prefill_attention(q.cuda(), kc, vc, sc, tab, lens, torch.tensor(qs, dtype=torch.int32, device="cuda"),
                                        most, 0.1, out)
        return out, device_errors()

    assert device_errors() == 0
    for lens, qs in ((torch.tensor([chunk - 1, chunk + 20]), [0, chunk, 2 * chunk]),
                     (torch.tensor([1 << 20, chunk + 20]), [0, chunk, 2 * chunk])):
        out, bits = call(lens.int().cuda(), qs)
        assert bits == pkv.DEVERR_CONTEXT_LEN_TOO_LONG
        assert (out[:chunk] == 7.0).all()
        assert_within(out[chunk:], ref[chunk:], allowed[chunk:], "the other")
    for qs in ([-chunk, chunk, 2 * chunk], [0, chunk, 2 * chunk + 5], [chunk + 1, chunk, 2 * chunk]):
        out, bits = call(cl, qs)
        assert bits == pkv.DEVERR_CONTEXT_LEN_TOO_LONG
    out, bits = call(cl, [0, chunk, 2 * chunk], most=chunk - 1)
    assert bits == pkv.DEVERR_CONTEXT_LEN_TOO_LONG and (out[chunk - 1] == 7.0).all()
    bad = table.clone()
    bad[1, 0] = -7
    out, bits = call(cl, [0, chunk, 2 * chunk], tab=bad)
    assert bits == pkv.DEVERR_BLOCK_ID_OUT_OF_RANGE
    assert_within(out[:chunk], ref[:chunk], allowed[:chunk], "the first")


@pytest.mark.parametrize("pasts,chunks", [((3000,), (5,)), ((2000, 40), (60, 3)), ((500, 0, 3), (300, 200, 1))])
def test_same_bits_again_and_in_a_graph(pasts, chunks):
    pages = Fp8Pages([p + c for p, c in zip(pasts, chunks)], 4, 128, 11)
    q = pages.randn(sum(chunks), 16, 128).cuda()
    kc, vc, sc, table, cl = pages.cuda()
    qs, out = starts(chunks), torch.empty_like(q)
    call = lambda: pkv.paged_fp8_prefill_attention(q, kc, vc, sc, table, cl, qs, max(chunks), 0.09, out)  # noqa: E731
    call()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(out, first)
    assert device_errors() == 0


@pytest.mark.parametrize("past,chunk", [(3000, 5), (3000, 200)])
def test_a_given_workspace_and_one_that_is_too_small(past, chunk):
    pages = Fp8Pages((past + chunk,), 2, 128, 12)
    need = pkv.fp8_prefill_workspace_size(chunk + 3, chunk, 1, 8, 2, 128, pages.width)
    pages.g.manual_seed(1)
    a = run((past,), (chunk,), 8, 2, 128, pages=pages)
    pages.g.manual_seed(1)
    b = run((past,), (chunk,), 8, 2, 128, pages=pages,
            workspace=torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a, b)
    if need > 0:
        with pytest.raises(ValueError, match="workspace"):
            run((past,), (chunk,), 8, 2, 128, pages=pages, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


def test_no_rows():
    pages = Fp8Pages((5, 9), 2, 64, 1)
    kc, vc, sc, table, cl = pages.cuda()
    none = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert pkv.paged_fp8_prefill_attention(none, kc, vc, sc, table, cl, starts([0, 0]), 0, 0.1, none) is none
    assert device_errors() == 0


def test_refusals_of_the_tensors():
    pages = Fp8Pages((20, 40), 1, 64, 3)
    q = pages.randn(4, 2, 64).cuda()
    kc, vc, sc, table, cl = pages.cuda()
    with pytest.raises(ValueError, match="query_start"):
        pkv.paged_fp8_prefill_attention(q, kc, vc, sc, table, cl, starts([4]), 4, 0.1, q.clone())
    with pytest.raises(pkv.PagedKVError, match="scale"):
        pkv.paged_fp8_prefill_attention(q, kc, vc, sc, table, cl, starts([2, 2]), 2, 0.0, q.clone())
    with pytest.raises(TypeError, match="bfloat16"):
        pkv.paged_fp8_prefill_attention(q.half(), kc, vc, sc, table, cl, starts([2, 2]), 2, 0.1, q.half())
