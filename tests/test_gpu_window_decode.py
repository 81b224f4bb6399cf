"""Windowed decode attention on the GPU against the definition in 64 bits (tolerances: plain64.attend).

A call with few (sequence, kv head) pairs and no partition count given joins through shared memory; others, and all with
a count, through the workspace.  Most tests run both."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from plain64 import BLOCK, Pages, assert_within, attend, f64, sees

pytestmark = pytest.mark.gpu


def exact(pages, q, lens, window, sinks, scale):
    qf, kf, vf = f64(q), f64(pages.k), f64(pages.v)
    rows = [attend(qf[b], kf, vf, pages.table[b], sees(n - 1, window, sinks) if n > 0 else [], scale, 0.0)
            for b, n in enumerate(lens)]
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


def hide(pages, window, sinks):
    """NaN in every token that is not seen, and -1 for every block that holds none that is."""
    for b, n in enumerate(pages.lens):
        seen = set(sees(n - 1, window, sinks).tolist()) if n else set()
        pages.poison(b, [t for t in range(-(-n // BLOCK) * BLOCK) if t not in seen])
        for blk in range(-(-n // BLOCK)):
            if not any(t in seen for t in range(blk * BLOCK, blk * BLOCK + BLOCK)):
                pages.table[b, blk] = -1


def run(lens, hq, hkv, d, window, sinks, seed=0, scale=None, **kw):
    pages = Pages(lens, hkv, d, seed)
    hide(pages, window, sinks)
    q = pages.randn(len(lens), hq, d)
    scale = d ** -0.5 if scale is None else scale
    kc, vc, table, cl = pages.cuda()
    out = torch.full((len(lens), hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = pkv.paged_window_decode_attention(q.cuda(), kc, vc, table, cl, scale, out, window, sinks, **kw)
    assert got is out
    ref, allowed = exact(pages, q, lens, window, sinks, scale)
    assert_within(out, ref, allowed, f"{hq}/{hkv} D{d} window {window} sinks {sinks} {kw}")
    assert device_errors() == 0
    return out


LENS = (0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257, 700)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (16, 2), (8, 8), (3, 3)])
@pytest.mark.parametrize("parts", [0, 37])
def test_layouts(hq, hkv, d, parts):
    run(LENS, hq, hkv, d, 50, 4, seed=hq, num_partitions=parts)


@pytest.mark.parametrize("seqs,window", [(1, 1000), (1, 40), (2, 1000), (9, 1000), (9, 100), (19, 200), (70, 300), (160, 60)])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (8, 1), (32, 4)])
def test_either_side_of_the_forms(seqs, window, hq, hkv):
    """Clusters of one to eight CTAs a pair, from one block a warp to several, and calls too large for them."""
    lens = np.random.RandomState(seqs + window).randint(0, 1500, seqs)
    run(lens, hq, hkv, 64, window, 5, seed=seqs)


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 700, 5000, 0x7fffffff])
@pytest.mark.parametrize("sinks", [0, 1, 16, 20])
@pytest.mark.parametrize("parts", [0, 37])
def test_windows(hq, window, sinks, parts):
    run(LENS, hq, 2, 64, window, sinks, seed=window % 1000 + sinks, num_partitions=parts)


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("sinks", [99, 690, 0x7fffffff])
def test_many_sinks(hq, sinks):
    run(LENS, hq, 2, 128, 3, sinks, seed=1)


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("parts", [1, 2, 7, 64, 1000])
def test_partition_counts(hq, parts):
    run((300, 0, 1, 77, 1000), hq, 2, 128, 130, 5, seed=2, num_partitions=parts)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("parts", [0, 5])
def test_scales(hq, scale, parts):
    run((40, 90), hq, 2, 64, 30, 3, seed=4, scale=scale, num_partitions=parts)


def test_window_as_long_as_the_sequences_is_plain_decode():
    """Both within their bound of the exact result (their weights enter the product differently)."""
    lens = (5, 16, 40, 333)
    pages = Pages(lens, 2, 128, 8)
    q = pages.randn(4, 8, 128)
    ref, allowed = exact(pages, q, lens, None, 0, 0.1)
    kc, vc, table, cl = pages.cuda()
    a, b = (torch.empty(q.shape, dtype=q.dtype, device="cuda") for _ in range(2))
    pkv.paged_window_decode_attention(q.cuda(), kc, vc, table, cl, 0.1, a, 400, 0, num_partitions=9)
    pkv.paged_decode_attention(q.cuda(), kc, vc, table, cl, 0.1, b, num_partitions=9)
    assert_within(a, ref, allowed, "window")
    assert_within(b, ref, allowed, "whole sequences")
    assert device_errors() == 0


@pytest.mark.parametrize("hq", [1, 4, 8])
@pytest.mark.parametrize("parts", [0, 1, 9])
def test_a_key_that_is_not_a_number_spoils_the_row_that_sees_it(hq, parts):
    pages = Pages((200, 40, 300), 1, 128, 9)
    q = pages.randn(3, hq, 128)
    pages.poison(0, [190])
    ref, allowed = exact(pages, q, (200, 40, 300), 64, 2, 0.09)
    kc, vc, table, cl = pages.cuda()
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.paged_window_decode_attention(q.cuda(), kc, vc, table, cl, 0.09, out, 64, 2, num_partitions=parts)
    assert torch.isnan(out[0].float()).all()
    assert_within(out[1:], ref[1:], allowed[1:], "the others")
    assert device_errors() == 0


def test_more_sequences_than_one_launch():
    lens = np.random.RandomState(0).randint(0, 40, 4096 + 200)
    run(lens, 2, 1, 64, 9, 2, seed=6)


@pytest.mark.parametrize("parts", [0, 3])
def test_bad_lengths_and_blocks_are_flagged(parts):
    pages = Pages((20, 40), 1, 64, 3)
    q = pages.randn(2, 2, 64).cuda()
    kc, vc, table, cl = pages.cuda()
    out = torch.empty_like(q)
    assert device_errors() == 0
    for bad, bit in ((-5, pkv.DEVERR_CONTEXT_LEN_NEGATIVE), (49, pkv.DEVERR_CONTEXT_LEN_TOO_LONG)):
        lens = cl.clone()
        lens[0] = bad
        pkv.paged_window_decode_attention(q, kc, vc, table, lens, 0.1, out, 10, 1, num_partitions=parts)
        assert device_errors() & bit
    table[1, 2] = 1 << 20
    pkv.paged_window_decode_attention(q, kc, vc, table, cl, 0.1, out, 10, 1, num_partitions=parts)
    assert device_errors() == pkv.DEVERR_BLOCK_ID_OUT_OF_RANGE


@pytest.mark.parametrize("parts", [0, 40])
def test_graphs_without_a_given_workspace_do_not_share_it(parts):
    """Two captured calls of different sizes, then eager ones that make the eager workspace grow."""
    cases = []
    for lens, hq in (((40, 300), 4), ((700,) * 9, 16)):
        pages = Pages(lens, 2, 128, len(lens))
        q = pages.randn(len(lens), hq, 128)
        ref = exact(pages, q, lens, 64, 4, 0.09)
        cases.append((pages.cuda(), q.cuda(), torch.empty(len(lens), hq, 128, dtype=torch.bfloat16, device="cuda"), ref))

    def call(c):
        (kc, vc, table, cl), q, out, _ = c
        pkv.paged_window_decode_attention(q, kc, vc, table, cl, 0.09, out, 64, 4, num_partitions=parts)

    for c in cases:
        call(c)
    torch.cuda.synchronize()
    graphs = []
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(c)
    run(LENS * 20, 16, 2, 128, 2000, 4, seed=11, num_partitions=parts and 5000)
    for _ in range(2):
        for g, c in zip(graphs, cases):
            c[2].zero_()
            g.replay()
        torch.cuda.synchronize()
        for _, _, out, (ref, allowed) in cases:
            assert_within(out, ref, allowed, "replayed")
    assert device_errors() == 0


@pytest.mark.parametrize("parts", [0, 40])
def test_two_streams_at_once(parts):
    lens = (900, 20, 400)
    pages = Pages(lens, 4, 128, 21)
    q = pages.randn(3, 16, 128)
    ref, allowed = exact(pages, q, lens, 200, 4, 0.09)
    kc, vc, table, cl = pages.cuda()
    qg = q.cuda()
    outs = [torch.zeros_like(qg) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, out in zip(streams, outs):
            pkv.paged_window_decode_attention(qg, kc, vc, table, cl, 0.09, out, 200, 4, stream=s, num_partitions=parts)
    torch.cuda.synchronize()
    for out in outs:
        assert_within(out, ref, allowed, "two streams")
    assert device_errors() == 0


@pytest.mark.parametrize("parts", [0, 20])
@pytest.mark.parametrize("hq", [8, 32])
def test_blocks_at_the_end_of_a_large_cache(parts, hq):
    """Element offsets past 32 bits: 2.3e9 elements a cache."""
    lens = (300, 20)
    pages = Pages(lens, 8, 128, 23)
    q = pages.randn(2, hq, 128)
    ref, allowed = exact(pages, q, lens, 100, 4, 0.09)
    kc, vc, table, cl = pages.cuda()
    blocks = 140_000
    big = [torch.empty(blocks, 8, BLOCK, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for b, c in zip(big, (kc, vc)):
        b[blocks - pages.pool:] = c
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    pkv.paged_window_decode_attention(q.cuda(), *big, torch.where(table >= 0, table + (blocks - pages.pool), table), cl,
                                      0.09, out, 100, 4, num_partitions=parts)
    assert_within(out, ref, allowed, "large cache")
    assert device_errors() == 0


def test_threads_on_one_stream_keep_their_workspaces_apart():
    """Host threads whose calls interleave on one stream: each has a workspace of its own."""
    import threading
    cases = []
    for k in range(3):
        lens = (500 + k, 40, 300 - k)
        pages = Pages(lens, 2, 64, 40 + k)
        q = pages.randn(3, 8, 64)
        cases.append((exact(pages, q, lens, 200, 4, 0.09), q.cuda(), pages.cuda(),
                      torch.zeros(q.shape, dtype=q.dtype, device="cuda")))

    def work(case):
        _, q, (kc, vc, table, cl), out = case
        for _ in range(50):
            pkv.paged_window_decode_attention(q, kc, vc, table, cl, 0.09, out, 200, 4, num_partitions=30)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for (ref, allowed), _, _, out in cases:
        assert_within(out, ref, allowed, "threads")
    assert device_errors() == 0


def test_refusals():
    pages = Pages((20, 40), 1, 64, 3)
    q = pages.randn(2, 2, 64).cuda()
    kc, vc, table, cl = pages.cuda()
    out = torch.empty_like(q)
    call = pkv.paged_window_decode_attention
    with pytest.raises(pkv.PagedKVError, match="window"):
        call(q, kc, vc, table, cl, 0.1, out, 0)
    with pytest.raises(pkv.PagedKVError, match="num_sink_tokens"):
        call(q, kc, vc, table, cl, 0.1, out, 5, -1)
    with pytest.raises(ValueError, match="32 bits"):
        call(q, kc, vc, table, cl, 0.1, out, (1 << 32) + 5)
    with pytest.raises(ValueError, match="batch"):
        call(q, kc, vc, table[:1], cl, 0.1, out, 5)
    with pytest.raises(ValueError, match="workspace"):
        call(q, kc, vc, table, cl, 0.1, out, 5, num_partitions=2,
             workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="bfloat16"):
        call(q.float(), kc, vc, table, cl, 0.1, out, 5)
    with pytest.raises(ValueError, match="contiguous"):
        call(q, kc, vc, table.t().contiguous().t(), cl, 0.1, out, 5)
    assert device_errors() == 0
