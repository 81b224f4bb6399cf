"""Shared-prefix decode attention on the GPU against the definition in 64 bits (tolerances: plain64.attend; the
shared part's weights enter their product as bf16, 2^-8 each).

A call with few (sequence, kv head) pairs and a narrow table runs as one kernel in which each pair reads the shared blocks
for itself; others share them.  WIDE tables make small calls take the second form."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from plain64 import BLOCK, Pages, assert_within, attend, f64, sees

pytestmark = pytest.mark.gpu
WIDE = 4000
both_forms = pytest.mark.parametrize("width", [None, WIDE], ids=["narrow", "wide"])


def make(groups, lens, hkv, d, seed, width=None):
    """groups: (first row, rows, prefix length).  Each group's whole prefix blocks are its first row's; the other
    rows' own entries there are -1 (they are not read)."""
    pages = Pages(lens, hkv, d, seed, width=width)
    real = pages.table.copy()
    for first, rows, prefix in groups:
        blocks = prefix // BLOCK
        for b in range(first + 1, first + rows):
            real[b, :blocks] = real[first, :blocks]
            pages.table[b, :blocks] = -1
    return pages, real


def exact(pages, real, q, lens, scale):
    qf, kf, vf = f64(q), f64(pages.k), f64(pages.v)
    rows = [attend(qf[b], kf, vf, real[b], sees(n - 1) if n > 0 else [], scale, 2.0**-8) for b, n in enumerate(lens)]
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


def bounds(groups):
    return [g[0] for g in groups] + [groups[-1][0] + groups[-1][1]] if groups else [0]


def run(groups, lens, hq, hkv, d, width=None, seed=0, **kw):
    pages, real = make(groups, lens, hkv, d, seed, width)
    q = pages.randn(len(lens), hq, d)
    ref, allowed = exact(pages, real, q, lens, d ** -0.5)
    kc, vc, table, cl = pages.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    got = pkv.paged_prefix_decode_attention(q.cuda(), kc, vc, table, cl, torch.tensor(bounds(groups), **i32),
                                            torch.tensor([g[2] for g in groups], **i32), d ** -0.5, out, **kw)
    assert got is out
    assert_within(out, ref, allowed, f"{hq}/{hkv} D{d} groups {groups}")
    assert device_errors() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (16, 2), (8, 8), (3, 3)])
@both_forms
def test_layouts(hq, hkv, d, width):
    run([(0, 3, 200), (3, 2, 64)], (201, 333, 217, 65, 300), hq, hkv, d, width, seed=hq)


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 112, 128, 129, 144, 1000])
@pytest.mark.parametrize("hq", [4, 16])
@both_forms
def test_prefix_lengths(prefix, hq, width):
    """Whole blocks only are shared; the sequences' tails start inside one, on its border, or are empty."""
    lens = [prefix + t for t in (0, 1, 15, 16, 17, 90)]
    lens[0] += prefix == 0
    run([(0, 6, prefix)], lens, hq, 2, 128, width, seed=prefix)


@pytest.mark.parametrize("rows", [1, 2, 16, 31, 32, 33, 63, 64, 65, 128, 200])
@pytest.mark.parametrize("hq", [2, 8])
@both_forms
def test_group_sizes(rows, hq, width):
    """One, two and more tiles of 128 rows, full, by one short and by one over."""
    lens = 200 + np.random.RandomState(rows).randint(0, 40, rows)
    run([(0, rows, 200)], lens, hq, 1, 64, width, seed=rows)


@both_forms
def test_sequences_shorter_than_the_prefix_see_their_own_length(width):
    run([(0, 5, 320)], (330, 0, 1, 100, 319), 8, 2, 128, width, seed=3)


@both_forms
def test_empty_groups_single_sequences_and_sequences_outside(width):
    run([(1, 0, 500), (1, 3, 100), (4, 1, 64), (5, 0, 7), (5, 2, 33)], (50, 120, 100, 140, 90, 40, 60, 5), 8, 2, 128,
        width, seed=4)


@both_forms
def test_no_groups_is_plain_decode(width):
    run([], (50, 0, 140), 8, 2, 64, width, seed=5)


@pytest.mark.parametrize("count", [31, 32, 33, 70, 400])
@both_forms
def test_many_groups(count, width):
    """More groups than a warp has lanes, of all lengths."""
    rng = np.random.RandomState(count)
    rows = rng.randint(0, 4, count)
    prefix = rng.randint(0, 700, count)
    first = np.concatenate([[0], np.cumsum(rows)])
    groups = [(int(first[g]), int(rows[g]), int(prefix[g])) for g in range(count)]
    lens = np.concatenate([prefix[g] + rng.randint(1, 50, rows[g]) for g in range(count)])
    run(groups, lens, 4, 1, 64, width, seed=count)


def test_more_units_than_sms():
    """40 groups of 8 kv heads: whole waves of CTAs."""
    groups = [(2 * g, 2, 300 + 10 * g) for g in range(40)]
    lens = [groups[b // 2][2] + 1 + b % 7 for b in range(80)]
    run(groups, lens, 8, 8, 64, WIDE, seed=7)


def test_long_prefix():
    run([(0, 4, 20000)], (20001, 20010, 20100, 20016), 8, 2, 128, seed=8)


@both_forms
def test_what_the_tables_hold_behind_a_sequence_does_not_matter(width):
    groups, lens = [(0, 3, 100)], (130, 101, 97 + 16)
    pages, real = make(groups, lens, 2, 128, 9, width)
    q = pages.randn(3, 8, 128)
    ref, allowed = exact(pages, real, q, lens, 0.1)
    for b, n in enumerate(lens):  # rows behind the end of the last block
        pages.table, real = real, pages.table
        pages.poison(b, range(n, -(-n // BLOCK) * BLOCK))
        pages.table, real = real, pages.table
    kc, vc, table, cl = pages.cuda()
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    pkv.paged_prefix_decode_attention(q.cuda(), kc, vc, table, cl, torch.tensor([0, 3], **i32),
                                      torch.tensor([100], **i32), 0.1, out)
    assert_within(out, ref, allowed, "poisoned ends")
    assert device_errors() == 0


@pytest.mark.parametrize("start", [[0, 3, 2], [-1, 1, 3], [0, 2, 9], [3, 0, 3]])
@both_forms
def test_groups_out_of_order_are_flagged(start, width):
    pages = Pages((100, 120, 90), 2, 64, 1, width=width)
    q = pages.randn(3, 4, 64).cuda()
    kc, vc, table, cl = pages.cuda()
    out, i32 = torch.empty_like(q), dict(dtype=torch.int32, device="cuda")
    assert device_errors() == 0
    pkv.paged_prefix_decode_attention(q, kc, vc, table, cl, torch.tensor(start, **i32), torch.tensor([64, 64], **i32),
                                      0.1, out)
    assert device_errors() == pkv.DEVERR_CONTEXT_LEN_TOO_LONG


@both_forms
def test_bad_prefixes_and_blocks_are_flagged(width):
    pages = Pages((100, 120, 90), 2, 64, 1, width=width)
    q = pages.randn(3, 4, 64).cuda()
    kc, vc, table, cl = pages.cuda()
    out, i32 = torch.empty_like(q), dict(dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 3], **i32)
    ref, allowed = exact(pages, pages.table, q.cpu(), pages.lens, 0.1)
    assert device_errors() == 0
    pkv.paged_prefix_decode_attention(q, kc, vc, table, cl, start, torch.tensor([-7], **i32), 0.1, out)
    assert device_errors() == pkv.DEVERR_CONTEXT_LEN_NEGATIVE
    assert_within(out, ref, allowed, "negative prefix: nothing shared")
    pkv.paged_prefix_decode_attention(q, kc, vc, table, cl, start, torch.tensor([10**6], **i32), 0.1, out)
    assert device_errors() & pkv.DEVERR_CONTEXT_LEN_TOO_LONG
    table[0, 1] = 1 << 20
    pkv.paged_prefix_decode_attention(q, kc, vc, table, cl, start, torch.tensor([64], **i32), 0.1, out)
    assert device_errors() == pkv.DEVERR_BLOCK_ID_OUT_OF_RANGE


@both_forms
def test_back_to_back_calls_graphs_and_streams(width):
    """Calls that reuse one workspace with other groups in between, two streams at once, and graphs."""
    cases = []
    for k, (groups, lens) in enumerate([([(0, 4, 500)], (501, 600, 510, 700)),
                                        ([(0, 2, 100), (2, 30, 900)], [110, 150] + list(range(901, 931)))]):
        pages, real = make(groups, lens, 2, 128, 20 + k, width)
        q = pages.randn(len(lens), 8, 128)
        i32 = dict(dtype=torch.int32, device="cuda")
        cases.append((exact(pages, real, q, lens, 0.09), q.cuda(), pages.cuda(), torch.tensor(bounds(groups), **i32),
                      torch.tensor([g[2] for g in groups], **i32), torch.empty(q.shape, dtype=q.dtype, device="cuda")))

    def call(c, **kw):
        _, q, (kc, vc, table, cl), start, prefix, out = c
        pkv.paged_prefix_decode_attention(q, kc, vc, table, cl, start, prefix, 0.09, out, **kw)

    def check(what):
        torch.cuda.synchronize()
        for (ref, allowed), *_, out in cases:
            assert_within(out, ref, allowed, what)
            out.zero_()

    for _ in range(10):
        for c in cases:
            call(c)
    check("in turn")
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(cases, streams):
            call(c, stream=s)
    check("two streams")
    graphs = [torch.cuda.CUDAGraph() for _ in cases]
    for g, c in zip(graphs, cases):
        with torch.cuda.graph(g):
            call(c)
    for _ in range(3):
        for g in graphs:
            g.replay()
    check("replayed")
    assert device_errors() == 0


@both_forms
def test_blocks_at_the_end_of_a_large_cache(width):
    """Element offsets past 32 bits: 2.3e9 elements a cache, every block used near its end."""
    groups, lens = [(0, 3, 100)], (130, 101, 115)
    pages, real = make(groups, lens, 8, 128, 31, width)
    q = pages.randn(3, 16, 128)
    ref, allowed = exact(pages, real, q, lens, 0.1)
    kc, vc, table, cl = pages.cuda()
    blocks = 140_000
    big = [torch.empty(blocks, 8, BLOCK, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    shift = blocks - pages.pool
    for b, c in zip(big, (kc, vc)):
        b[shift:] = c
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    moved = torch.where(table >= 0, table + shift, table)
    pkv.paged_prefix_decode_attention(q.cuda(), *big, moved, cl, torch.tensor([0, 3], **i32), torch.tensor([100], **i32),
                                      0.1, out)
    assert_within(out, ref, allowed, "large cache")
    assert device_errors() == 0


def test_refusals():
    pages = Pages((100, 120, 90), 2, 64, 1, width=WIDE)
    q = pages.randn(3, 4, 64).cuda()
    kc, vc, table, cl = pages.cuda()
    out, i32 = torch.empty_like(q), dict(dtype=torch.int32, device="cuda")
    start, prefix = torch.tensor([0, 3], **i32), torch.tensor([64], **i32)
    call = pkv.paged_prefix_decode_attention
    with pytest.raises(ValueError, match="group_start"):
        call(q, kc, vc, table, cl, start[:1], prefix, 0.1, out)
    with pytest.raises(TypeError, match="prefix_lens"):
        call(q, kc, vc, table, cl, start, prefix.long(), 0.1, out)
    with pytest.raises(pkv.PagedKVError, match="scale"):
        call(q, kc, vc, table, cl, start, prefix, -0.1, out)
    with pytest.raises(ValueError, match="workspace"):
        call(q, kc, vc, table, cl, start, prefix, 0.1, out, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert device_errors() == 0
