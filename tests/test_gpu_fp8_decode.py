"""Decode attention over the 8-bit cache on the GPU against the definition in 64 bits (bounds: fp8_plain.attend_fp8; weights
enter the product with V in 16 bits of eleven significant ones, half a step 2^-11)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from fp8_plain import FP8, Fp8Pages, attend_fp8
from gpu_util import device_errors
from plain64 import BLOCK, assert_within, f64

pytestmark = pytest.mark.gpu

WEIGHT = 2.0**-11


def exact(pages, q, lens, scale):
    qf = f64(q)
    rows = [attend_fp8(pages, b, qf[b], int(n), scale, WEIGHT) for b, n in enumerate(lens)]
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


def run(lens, hq, hkv, d, seed=0, scale=None, spread=1.0, q=None, pages=None, **kw):
    pages = pages or Fp8Pages(lens, hkv, d, seed, spread=spread)
    q = pages.randn(len(lens), hq, d) if q is None else q
    scale = d ** -0.5 if scale is None else scale
    kc, vc, sc, table, cl = pages.cuda()
    out = torch.full((len(lens), hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = pkv.paged_fp8_decode_attention(q.cuda(), kc, vc, sc, table, cl, scale, out, **kw)
    assert got is out
    ref, allowed = exact(pages, q, lens, scale)
    assert_within(out, ref, allowed, f"{hq}/{hkv} D{d}")
    assert device_errors() == 0
    return out


LENS = (0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257, 700)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (4, 1), (8, 1), (2, 2), (16, 2), (3, 3), (12, 3), (4, 4), (10, 5), (6, 6),
                                    (48, 6), (8, 8), (32, 8), (64, 8), (24, 12), (16, 16)])
def test_layouts(hq, hkv, d):
    run(LENS, hq, hkv, d, seed=hq)


@pytest.mark.parametrize("seqs,most", [(1, 1), (1, 5000), (2, 3000), (9, 100), (33, 1000), (200, 300), (1, 20000)])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (8, 1), (12, 3), (32, 4)])
def test_batches(seqs, most, hq, hkv):
    lens = np.random.RandomState(seqs + most).randint(0, most + 1, seqs)
    lens[0] = most
    run(lens, hq, hkv, 64, seed=seqs)


@pytest.mark.parametrize("n", range(1, 52))
def test_every_short_length(n):
    run((n, n + 51), 8, 2, 128, seed=n)


def test_many_sequences():
    lens = np.random.RandomState(0).randint(0, 40, 4096 + 200)
    run(lens, 2, 1, 64, seed=6)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0, 3.0])
@pytest.mark.parametrize("hq", [2, 16])
def test_scales(hq, scale):
    run((40, 90, 1), hq, 2, 64, seed=4, scale=scale)


@pytest.mark.parametrize("spread", [6.0, 12.0])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_very_different_sizes(spread, d):
    """Sizes over many powers of two: rows of large values outweigh, in V those of small ones still count."""
    run((1, 7, 40, 300, 1000), 8, 2, d, seed=5, spread=spread, scale=2.0**-8)


def test_queries_of_very_different_sizes():
    pages = Fp8Pages((50, 60, 70, 80), 2, 128, 3)
    q = pages.randn(4, 8, 128) * (2.0 ** torch.arange(-24, 8).reshape(4, 8, 1)).to(torch.bfloat16)
    q[1, :, 5] = 3e4
    run(pages.lens, 8, 2, 128, pages=pages, q=q, scale=0.01)


def test_values_of_zero():
    pages = Fp8Pages((33, 100), 2, 64, 3)
    pages.v[pages.table[0, :3]] = 0.0  # a sequence whose values are all zero, and one with half of them
    pages.v[pages.table[1, :7], :, ::2] = 0.0
    pages.quantise()
    out = run((33, 100), 4, 2, 64, pages=pages)
    assert (out[0] == 0).all()


def test_what_is_not_seen_does_not_matter():
    """NaN codes and exponents of 255 behind each sequence's last token (as Fp8Pages leaves them), and table entries behind the
    last block that point anywhere."""
    pages = Fp8Pages((5, 0, 16, 47), 2, 128, 7, width=9)
    q = pages.randn(4, 8, 128)
    a = run(pages.lens, 8, 2, 128, pages=pages, q=q)
    pages.table[pages.table < 0] = 1 << 30
    b = run(pages.lens, 8, 2, 128, pages=pages, q=q)
    assert torch.equal(a, b)


@pytest.mark.parametrize("hq", [1, 4, 8])
@pytest.mark.parametrize("which", ["k8", "v8"])
def test_a_row_that_is_not_a_number_spoils_the_sequence_that_sees_it(hq, which):
    pages = Fp8Pages((200, 40, 300), 1, 128, 9)
    q = pages.randn(3, hq, 128)
    ref, allowed = exact(pages, q, pages.lens, 0.09)
    getattr(pages, which).view(torch.uint8)[pages.table[0, 5], :, 3] = 0x7F
    kc, vc, sc, table, cl = pages.cuda()
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.paged_fp8_decode_attention(q.cuda(), kc, vc, sc, table, cl, 0.09, out)
    assert torch.isnan(out[0].float()).all()
    assert_within(out[1:], ref[1:], allowed[1:], "the others")
    assert device_errors() == 0


def test_bad_lengths_and_blocks_are_flagged():
    pages = Fp8Pages((20, 40), 1, 64, 3)
    q = pages.randn(2, 2, 64).cuda()
    kc, vc, sc, table, cl = pages.cuda()
    out = torch.empty_like(q)
    assert device_errors() == 0
    for bad, bit in ((-5, pkv.DEVERR_CONTEXT_LEN_NEGATIVE), (49, pkv.DEVERR_CONTEXT_LEN_TOO_LONG)):
        lens = cl.clone()
        lens[0] = bad
        pkv.paged_fp8_decode_attention(q, kc, vc, sc, table, lens, 0.1, out)
        assert device_errors() & bit
    table[1, 2] = 1 << 20
    pkv.paged_fp8_decode_attention(q, kc, vc, sc, table, cl, 0.1, out)
    assert device_errors() == pkv.DEVERR_BLOCK_ID_OUT_OF_RANGE


def test_empty_sequences_only():
    pages = Fp8Pages((0, 0, 0), 2, 64, 3)
    assert (run((0, 0, 0), 4, 2, 64, pages=pages) == 0).all()
    kc, vc, sc, table, cl = pages.cuda()
    none = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert pkv.paged_fp8_decode_attention(none, kc, vc, sc, table[:0], cl[:0], 0.1, none) is none
    assert device_errors() == 0


def test_same_bits_again_in_a_graph_and_on_another_stream():
    """Every run of a call gives the same bits; a graph replayed over other inputs of the same sizes gives theirs."""
    lens = (900, 3, 0, 77, 2000, 16, 1)
    pages = Fp8Pages(lens, 4, 128, 11)
    q = pages.randn(7, 16, 128).cuda()
    kc, vc, sc, table, cl = pages.cuda()
    out = torch.empty_like(q)
    pkv.paged_fp8_decode_attention(q, kc, vc, sc, table, cl, 0.09, out)
    first = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.paged_fp8_decode_attention(q, kc, vc, sc, table, cl, 0.09, out)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    shorter = torch.tensor([1, 900, 33, 0, 500, 16, 2], dtype=torch.int32, device="cuda").minimum(cl.clamp(min=0))
    eager = torch.empty_like(q)
    pkv.paged_fp8_decode_attention(q, kc, vc, sc, table, shorter, 0.09, eager, stream=torch.cuda.current_stream())
    cl.copy_(shorter)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    with torch.cuda.stream(side):
        pkv.paged_fp8_decode_attention(q, kc, vc, sc, table, cl, 0.09, out)
    side.synchronize()
    assert torch.equal(out, eager)
    assert device_errors() == 0


def test_a_given_workspace_and_one_that_is_too_small():
    pages = Fp8Pages((3000, 40), 2, 128, 12)
    q = pages.randn(2, 8, 128)
    need = pkv.fp8_decode_workspace_size(2, 8, 2, 128, pages.width)
    assert pkv.fp8_decode_workspace_size(1, 8, 2, 128, pages.width) <= need
    a = run(pages.lens, 8, 2, 128, pages=pages, q=q)
    b = run(pages.lens, 8, 2, 128, pages=pages, q=q, workspace=torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a, b)
    if need > 0:
        with pytest.raises(ValueError, match="workspace"):
            run(pages.lens, 8, 2, 128, pages=pages, q=q, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


SEQS = [1, 2, 3, 4, 5, 8, 9, 12, 16, 18, 19, 20, 24, 36, 37, 38, 40, 64, 75, 76, 77, 100, 151, 152, 153, 200, 303, 304, 305, 600,
        1023, 1024, 1025, 4000]


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 128), (8, 1, 128), (2, 2, 64), (32, 8, 128), (64, 8, 64), (12, 3, 128)])
def test_workspace_sizes_do_not_fall(hq, hkv, d):
    sizes = [[pkv.fp8_decode_workspace_size(n, hq, hkv, d, width) for n in SEQS]
             for width in (1, 8, 9, 60, 100, 300, 410, 500, 512, 521, 600, 700, 1000, 1024, 2000, 2048, 4000, 20000)]
    assert (np.diff(sizes, axis=0) >= 0).all() and (np.diff(sizes, axis=1) >= 0).all()
    assert sizes[0][0] == 0 and sizes[-1][0] > 0  # (both forms)


@pytest.mark.parametrize("hkv", [1, 8])
def test_one_workspace_for_all_batches(hkv):
    """Lengths that a few sequences take in the stream and more in clusters: every batch with the largest one's workspace."""
    lens = [6000, 9000]
    pages = Fp8Pages(lens, hkv, 128, hkv, width=1500)
    q = pages.randn(8, hkv, 128)
    rows = [attend_fp8(pages, b % 2, f64(q)[b], lens[b % 2], 0.1, WEIGHT) for b in range(8)]
    ref, allowed = np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])
    kc, vc, sc, table, cl = pages.cuda()
    space = torch.empty(max(16, pkv.fp8_decode_workspace_size(8, hkv, hkv, 128, 1500)), dtype=torch.uint8, device="cuda")
    for n in range(1, 9):
        out = torch.empty(n, hkv, 128, dtype=torch.bfloat16, device="cuda")
        pkv.paged_fp8_decode_attention(q[:n].cuda(), kc, vc, sc, table.repeat(4, 1)[:n], cl.repeat(4)[:n], 0.1, out, workspace=space)
        assert_within(out, ref[:n], allowed[:n], f"{n} sequences")
    assert device_errors() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (8, 8), (16, 4), (12, 6), (5, 5), (8, 1)])
def test_more_pairs_than_clusters(hq, hkv, d):
    """Long and short sequences, more than the GPU holds clusters for: pieces that begin and end inside of pairs."""
    r = np.random.RandomState(hq)
    lens = r.randint(0, 90, 310 // hkv + 1) + (r.rand(310 // hkv + 1) < 0.1) * 1500
    run(lens, hq, hkv, d, seed=hq)


def test_a_large_cache():
    """Blocks whose rows lie behind 2^32 bytes."""
    hkv, d, nb = 8, 128, 270_000
    pages = Fp8Pages((100,), hkv, d, 13)
    q = pages.randn(1, 16, 128)
    ref, allowed = exact(pages, q, pages.lens, 0.09)
    shift = nb - pages.pool
    big = [torch.zeros(nb, *x.shape[1:], dtype=torch.uint8, device="cuda") for x in (pages.k8, pages.v8, pages.scales)]
    assert big[0].numel() > 1 << 32
    for dst, src in zip(big, (pages.k8, pages.v8, pages.scales)):
        dst[shift:] = src.view(torch.uint8).cuda()
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.paged_fp8_decode_attention(q.cuda(), big[0].view(FP8), big[1].view(FP8), big[2],
                                   torch.from_numpy(pages.table + shift).cuda(), torch.tensor(pages.lens, dtype=torch.int32).cuda(), 0.09, out)
    assert_within(out, ref, allowed, "large cache")
    assert device_errors() == 0


def test_refusals_of_the_tensors():
    pages = Fp8Pages((20, 40), 1, 64, 3)
    q = pages.randn(2, 2, 64).cuda()
    kc, vc, sc, table, cl = pages.cuda()
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        pkv.paged_fp8_decode_attention(q, kc.view(torch.uint8), vc, sc, table, cl, 0.1, q.clone())
    with pytest.raises(ValueError, match="kv_scales"):
        pkv.paged_fp8_decode_attention(q, kc, vc, sc[:, :, :1].contiguous(), table, cl, 0.1, q.clone())
    with pytest.raises(ValueError, match="batch"):
        pkv.paged_fp8_decode_attention(q, kc, vc, sc, table, cl[:1], 0.1, q.clone())
    with pytest.raises(ValueError, match="contiguous"):
        pkv.paged_fp8_decode_attention(q.transpose(0, 1), kc, vc, sc, table, cl, 0.1, q.clone())
    with pytest.raises(pkv.PagedKVError, match="group"):
        bad = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
        pkv.paged_fp8_decode_attention(bad, kc, vc, sc, table, cl, 0.1, bad.clone())
