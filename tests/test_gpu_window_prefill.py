"""Windowed prefill attention on the GPU against the definition in 64 bits (tolerances: plain64.attend; the weights
enter the product as bf16, 2^-8 each)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from plain64 import BLOCK, Pages, assert_within, attend, f64, sees

pytestmark = pytest.mark.gpu


def exact(pages, q, start, lens, window, sinks, scale):
    qf = f64(q)
    kf, vf = f64(pages.k), f64(pages.v)
    out, allowed = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(lens):
        chunk = start[b + 1] - start[b]
        for i in range(chunk):
            keys = sees(n - chunk + i, window, sinks)
            out[start[b] + i], allowed[start[b] + i] = attend(qf[start[b] + i], kf, vf, pages.table[b], keys, scale,
                                                              2.0**-8)
    return out, allowed


def make(chunks, pasts, hq, hkv, d, window, sinks, seed, hidden=True):
    lens = [p + c for p, c in zip(pasts, chunks)]
    pages = Pages(lens, hkv, d, seed)
    if hidden:  # what no row of a chunk sees: NaN, and -1 for blocks that hold nothing else
        for b, (p, c) in enumerate(zip(pasts, chunks)):
            n = p + c
            seen = set(range(max(0, p + 1 - window), n)) | set(range(min(sinks, n)))
            if c == 0:
                seen = set()
            pages.poison(b, [t for t in range(-(-n // BLOCK) * BLOCK) if t not in seen])
            for blk in range(-(-n // BLOCK)):
                if not any(t in seen for t in range(blk * BLOCK, blk * BLOCK + BLOCK)):
                    pages.table[b, blk] = -1
    start = np.concatenate([[0], np.cumsum(chunks)]).astype(int)
    return pages, lens, start, pages.randn(int(start[-1]), hq, d)


def run(chunks, pasts, hq, hkv, d, window, sinks, seed=0, **kw):
    pages, lens, start, q = make(chunks, pasts, hq, hkv, d, window, sinks, seed)
    scale = d ** -0.5
    kc, vc, table, cl = pages.cuda()
    qs = torch.tensor(start, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    got = pkv.paged_window_prefill_attention(q.cuda(), kc, vc, table, cl, qs, max(chunks), scale, out, window, sinks, **kw)
    assert got is out
    ref, allowed = exact(pages, q, start, lens, window, sinks, scale)
    assert_within(out, ref, allowed, f"{hq}/{hkv} D{d} chunks {chunks} after {pasts} window {window} sinks {sinks} {kw}")
    assert device_errors() == 0


CHUNKS, PASTS = (1, 7, 37, 130, 16, 0, 1), (0, 3, 100, 500, 64, 20, 333)


@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (4, 2, 128), (8, 2, 128), (16, 2, 128), (2, 2, 64), (4, 2, 64),
                                      (8, 2, 64), (16, 2, 64)])
@pytest.mark.parametrize("splits", [1, 3])
def test_layouts(hq, hkv, d, splits):
    run(CHUNKS, PASTS, hq, hkv, d, 50, 4, seed=hq + d, num_splits=splits)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 127, 128, 129, 400, 100000, 0x7fffffff])
@pytest.mark.parametrize("sinks", [0, 1, 16, 20])
def test_windows(window, sinks):
    run((300, 5), (200, 700), 8, 2, 64, window, sinks, seed=window % 1000 + sinks, num_splits=1)


@pytest.mark.parametrize("sinks", [100, 119, 128, 250, 0x7fffffff])
@pytest.mark.parametrize("window", [1, 30])
@pytest.mark.parametrize("splits", [1, 2])
def test_many_sinks(sinks, window, splits):
    """The gap between sinks and window lies inside a step, on its border and over it."""
    run((200, 33), (400, 255), 8, 1, 64, window, sinks, seed=sinks % 1000, num_splits=splits)


@pytest.mark.parametrize("splits", [0, 2, 3, 7, 32])
def test_splits(splits):
    run((70, 1, 300), (900, 40, 0), 4, 1, 128, 333, 9, seed=splits, num_splits=splits)


@pytest.mark.parametrize("splits", [0, 1, 5])
@pytest.mark.parametrize("tiles", [19, 20, 28, 29, 38])
def test_last_waves(tiles, splits):
    """Eight kv heads and chunks of `tiles` tile pairs (32 tokens each) in all, the first and last rows of them ragged:
    152 SMs are full, have 8, 72 and 80 units in a second wave, and are full twice."""
    a = tiles // 3
    run((32 * a - 5, 3, 32 * (tiles - a - 1) - 31), (100, 700, 0), 64, 8, 64, 300, 4, seed=tiles, num_splits=splits)


@pytest.mark.parametrize("d,window,sinks", [(64, 20, 3), (128, 140, 30), (64, 1, 0), (128, 500, 200)])
def test_many_rounds_of_short_units(d, window, sinks):
    """100 chunks of one to five tokens and eight kv heads: 800 units, one to six key steps each, five or six a CTA, with keys
    past the end and between sinks and window in most."""
    run([1 + i % 5 for i in range(100)], [(37 * i) % 700 for i in range(100)], 8, 8, d, window, sinks, seed=d + window)


@pytest.mark.parametrize("splits", [0, 3])
def test_more_sequences_than_are_ranked(splits):
    for n in (320, 321):
        run([1 + i % 3 for i in range(n)], [(7 * i) % 60 for i in range(n)], 2, 1, 64, 20, 2, seed=n, num_splits=splits)


@pytest.mark.parametrize("seed", range(6))
def test_random_shapes(seed):
    import random
    rng = random.Random(seed)
    b = rng.randint(1, 6)
    chunks = [rng.choice([1, rng.randint(1, 40), rng.randint(40, 200)]) for _ in range(b)]
    pasts = [rng.choice([0, rng.randint(0, 64), rng.randint(64, 1500)]) for _ in range(b)]
    hkv = rng.choice([1, 2, 3])
    run(chunks, pasts, hkv * rng.choice([1, 2, 4, 8]), hkv, rng.choice([64, 128]), rng.randint(1, 600),
        rng.choice([0, 1, 4, 33, 130]), seed=seed, num_splits=rng.choice([0, 1, 2]))


def test_long_past_is_not_read():
    """20000 cached tokens, of which a chunk sees a few hundred: the block-id window slides within the stream."""
    run((40,), (20000,), 4, 2, 128, 700, 70, seed=3, num_splits=1)
    run((3,), (20000,), 4, 2, 128, 5000, 70, seed=3, num_splits=1)


def test_window_longer_than_everything_is_plain_prefill():
    """Both within their bound of the exact result (their exponentials are computed differently)."""
    pages, lens, start, q = make(CHUNKS[:5], PASTS[:5], 8, 2, 128, 10000, 0, 5, hidden=False)
    ref, allowed = exact(pages, q, start, lens, None, 0, 0.09)
    kc, vc, table, cl = pages.cuda()
    qs, qg = torch.tensor(start, dtype=torch.int32, device="cuda"), q.cuda()
    a, b = torch.empty_like(qg), torch.empty_like(qg)
    pkv.paged_window_prefill_attention(qg, kc, vc, table, cl, qs, 130, 0.09, a, 10000, 0, num_splits=1)
    pkv.paged_prefill_attention(qg, kc, vc, table, cl, qs, 130, 0.09, b)
    assert_within(a, ref, allowed, "window")
    assert_within(b, ref, allowed, "plain")
    assert device_errors() == 0


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_key_that_is_not_finite_spoils_the_rows_that_see_it(value, splits):
    """Row i of the chunk is at position 300 + i; key 280 is in the windows of the rows up to 280 + 63."""
    pages, lens, start, q = make((100,), (300,), 4, 1, 128, 64, 0, 6, hidden=False)
    pages.k[int(pages.table[0, 280 // BLOCK]), 0, 280 % BLOCK] = value
    kc, vc, table, cl = pages.cuda()
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.paged_window_prefill_attention(q.cuda(), kc, vc, table, cl, torch.tensor(start, dtype=torch.int32, device="cuda"),
                                       100, 0.09, out, 64, 0, num_splits=splits)
    finite = torch.isfinite(out.float()).all(-1).cpu()
    if value != value:
        assert not finite[:44].any()
    assert finite[44:].all()
    pages.k[int(pages.table[0, 280 // BLOCK]), 0, 280 % BLOCK] = 0.0
    ref, allowed = exact(pages, q, start, lens, 64, 0, 0.09)
    assert_within(out[44:], ref[44:], allowed[44:], "rows that do not see it")
    assert device_errors() == 0


def test_rows_behind_the_last_sequence_are_left_alone():
    pages, lens, start, q = make((20, 30), (0, 50), 4, 2, 64, 16, 2, 9)
    kc, vc, table, cl = pages.cuda()
    qg = torch.cat([q, q[:11]]).cuda()
    for splits in (1, 2):
        out = torch.full_like(qg, 5.0)
        pkv.paged_window_prefill_attention(qg, kc, vc, table, cl, torch.tensor(start, dtype=torch.int32, device="cuda"),
                                           30, 0.1, out, 16, 2, num_splits=splits)
        assert (out[50:] == 5.0).all() and torch.isfinite(out.float()).all()
    assert device_errors() == 0


def test_bad_lengths_and_blocks_are_flagged():
    pages, lens, start, q = make((20,), (50,), 4, 2, 64, 16, 2, 9)
    kc, vc, table, cl = pages.cuda()
    qg, qs = q.cuda(), torch.tensor(start, dtype=torch.int32, device="cuda")
    out = torch.empty_like(qg)
    assert device_errors() == 0
    for bad in (10, 81):  # shorter than the chunk, longer than the table
        pkv.paged_window_prefill_attention(qg, kc, vc, table, torch.full_like(cl, bad), qs, 20, 0.1, out, 16, 2)
        assert device_errors() == pkv.DEVERR_CONTEXT_LEN_TOO_LONG
    table[0, 4] = 1 << 20
    pkv.paged_window_prefill_attention(qg, kc, vc, table, cl, qs, 20, 0.1, out, 16, 2)
    assert device_errors() == pkv.DEVERR_BLOCK_ID_OUT_OF_RANGE


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("start", [[0, 20, 41], [0, 41, 20], [-1, 20, 40], [20, 40, 60]])
def test_chunks_outside_the_query_rows_are_flagged_and_skipped(start, splits):
    pages, lens, _, q = make((20, 20), (50, 60), 4, 2, 64, 16, 2, 9, hidden=False)
    kc, vc, table, cl = pages.cuda()
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    assert device_errors() == 0
    pkv.paged_window_prefill_attention(q.cuda(), kc, vc, table, cl, torch.tensor(start, dtype=torch.int32, device="cuda"),
                                       41, 0.1, out, 16, 2, num_splits=splits)
    assert device_errors() == pkv.DEVERR_CONTEXT_LEN_TOO_LONG
    if start == [0, 20, 41]:  # the first chunk is in order
        ref, allowed = exact(pages, q, [0, 20, 40], lens, 16, 2, 0.1)
        assert_within(out[:20], ref[:20], allowed[:20], "the other chunk")
        assert (out[20:] == 5.0).all()


@pytest.mark.parametrize("splits", [1, 3])
def test_blocks_at_the_end_of_a_large_cache(splits):
    """Element offsets past 32 bits: 2.3e9 elements a cache."""
    pages, lens, start, q = make((40,), (150,), 16, 8, 128, 100, 4, 17)
    ref, allowed = exact(pages, q, start, lens, 100, 4, 0.1)
    kc, vc, table, cl = pages.cuda()
    blocks = 140_000
    big = [torch.empty(blocks, 8, BLOCK, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for b, c in zip(big, (kc, vc)):
        b[blocks - pages.pool:] = c
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    pkv.paged_window_prefill_attention(q.cuda(), *big, torch.where(table >= 0, table + (blocks - pages.pool), table), cl,
                                       torch.tensor(start, dtype=torch.int32, device="cuda"), 40, 0.1, out, 100, 4,
                                       num_splits=splits)
    assert_within(out, ref, allowed, "large cache")
    assert device_errors() == 0


@pytest.mark.parametrize("splits", [1, 0])
def test_graph_and_stream(splits):
    pages, lens, start, q = make((64, 9), (300, 80), 8, 2, 128, 100, 4, 13)
    ref, allowed = exact(pages, q, start, lens, 100, 4, 0.09)
    kc, vc, table, cl = pages.cuda()
    qg, qs = q.cuda(), torch.tensor(start, dtype=torch.int32, device="cuda")
    out = torch.empty_like(qg)

    def call(stream=None):
        pkv.paged_window_prefill_attention(qg, kc, vc, table, cl, qs, 64, 0.09, out, 100, 4, num_splits=splits, stream=stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    s.synchronize()
    assert_within(out, ref, allowed, "another stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for _ in range(2):
        out.zero_()
        g.replay()
        assert_within(out, ref, allowed, "replayed")
    assert device_errors() == 0


def test_refusals():
    pages, lens, start, q = make((20,), (50,), 4, 2, 64, 16, 2, 9)
    kc, vc, table, cl = pages.cuda()
    qg, qs = q.cuda(), torch.tensor(start, dtype=torch.int32, device="cuda")
    out = torch.empty_like(qg)
    call = pkv.paged_window_prefill_attention
    with pytest.raises(pkv.PagedKVError, match="window"):
        call(qg, kc, vc, table, cl, qs, 20, 0.1, out, 0)
    with pytest.raises(pkv.PagedKVError, match="scale"):
        call(qg, kc, vc, table, cl, qs, 20, 0.0, out, 5)
    with pytest.raises(ValueError, match="query_start"):
        call(qg, kc, vc, table, cl, qs[:1], 20, 0.1, out, 5)
    with pytest.raises(pkv.PagedKVError, match="num_splits"):
        call(qg, kc, vc, table, cl, qs, 20, 0.1, out, 5, num_splits=33)
    with pytest.raises(ValueError, match="workspace"):
        call(qg, kc, vc, table, cl, qs, 20, 0.1, out, 5, num_splits=2,
             workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert device_errors() == 0
