"""Quantising append, reading back and block copies of the 8-bit cache on the GPU: bit for bit against the format's
definition (fp8_plain)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from fp8_plain import FP8, quantise, values
from gpu_util import device_errors
from plain64 import BLOCK, f64, rotated_bits

pytestmark = pytest.mark.gpu


def rows(g, *shape, spread=2.0):
    size = torch.exp2(torch.randn(*shape[:-1], 1, generator=g) * spread)
    return (torch.randn(*shape, generator=g) * size).to(torch.bfloat16)


def empty_cache(nb, hkv, d):
    """A cache whose every byte is set, to see what is left alone."""
    return (torch.full((nb, hkv, BLOCK, d), 0x55, dtype=torch.uint8).view(FP8).cuda(),
            torch.full((nb, hkv, BLOCK, d), 0xAA, dtype=torch.uint8).view(FP8).cuda(),
            torch.full((nb, hkv, 2, BLOCK), 0x33, dtype=torch.uint8).cuda())


def expect(cache, k, v, slots, nb):
    """The caches' bytes after an append of k, v at slots."""
    want = [x.cpu().view(torch.uint8).clone() for x in cache]
    for i, x in enumerate((k, v)):
        codes, e = quantise(x)
        bits = torch.from_numpy(codes).float().to(FP8).view(torch.uint8)
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < nb * BLOCK:
                want[i][s // BLOCK, :, s % BLOCK] = bits[t]
                want[2][s // BLOCK, :, i, s % BLOCK] = torch.from_numpy(e[t]).to(torch.uint8)
    return want


def same(cache, want):
    for got, w in zip(cache, want):
        assert torch.equal(got.cpu().view(torch.uint8), w)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 2, 3, 5, 8, 12])
@pytest.mark.parametrize("n", [1, 2, 17, 333])
def test_append(n, hkv, d):
    g = torch.Generator().manual_seed(n + hkv)
    nb = -(-n // BLOCK) + 3
    slots = torch.randperm(nb * BLOCK, generator=g)[:n]
    k, v = rows(g, n, hkv, d), rows(g, n, hkv, d)
    cache = empty_cache(nb, hkv, d)
    want = expect(cache, k, v, slots, nb)
    pkv.kv_append_fp8(k.cuda(), v.cuda(), slots.cuda(), *cache)
    same(cache, want)
    assert device_errors() == 0


def test_append_of_many_tokens():
    g = torch.Generator().manual_seed(1)
    nb = 1200
    slots = torch.randperm(nb * BLOCK, generator=g)[:19000]
    k, v = rows(g, 19000, 2, 64), rows(g, 19000, 2, 64)
    cache = empty_cache(nb, 2, 64)
    pkv.kv_append_fp8(k.cuda(), v.cuda(), slots.cuda(), *cache)
    at = slots.cuda()
    for i, x in enumerate((k, v)):
        codes, e = quantise(x)
        got = cache[i].view(torch.uint8)[at // BLOCK, :, at % BLOCK].cpu()
        assert torch.equal(got, torch.from_numpy(codes).float().to(FP8).view(torch.uint8))
        assert np.array_equal(cache[2][at // BLOCK, :, i, at % BLOCK].cpu().numpy(), e)
    assert device_errors() == 0


def test_append_of_views_with_padding_and_a_slot_outside():
    g = torch.Generator().manual_seed(2)
    n, hq, hkv, d, nb = 40, 4, 2, 128, 5
    fused = rows(g, n, hq + 2 * hkv, d).cuda()
    k, v = fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    slots = torch.randperm(nb * BLOCK, generator=g)[:n]
    slots[3] = slots[39] = -1
    slots[7] = nb * BLOCK
    slots[8] = 1 << 40
    cache = empty_cache(nb, hkv, d)
    want = expect(cache, k.cpu(), v.cpu(), slots, nb)
    pkv.kv_append_fp8(k, v, slots.cuda(), *cache)
    same(cache, want)
    assert device_errors() == pkv.DEVERR_SLOT_OUT_OF_RANGE


def test_append_borders_and_values_that_are_no_numbers():
    d = 64
    special = torch.zeros(14, 1, d, dtype=torch.float64)
    special[0] = 0.0
    special[1, 0, :3] = torch.tensor([448.0, 17.0, 19.0])            # ties to even
    special[2, 0, :3] = torch.tensor([450.0, 1.0, -450.0])
    special[3, 0, 5] = float("nan")
    special[4, 0, :2] = torch.tensor([float("inf"), 3.0])
    special[5, 0, :3] = torch.tensor([-float("inf"), float("nan"), -7.0])
    special[6] = float("nan")
    special[7, 0, 63] = 3.3e38
    special[8, 0, 1] = 2.0**-133                                     # the least bf16 value
    special[9, 0, :2] = torch.tensor([2.0**-119 * 1.75, 2.0**-126])
    special[10, 0, :4] = torch.tensor([448.0, 2.0**-9, 2.0**-10, 1.5 * 2.0**-9])
    special[11, 0, :2] = torch.tensor([-447.0, -2.0**-7])
    special[12] = -0.0
    special[13, 0, :2] = torch.tensor([3.0e38, 3.0e30])
    x = special.to(torch.bfloat16)
    slots = torch.arange(14)
    cache = empty_cache(1, 1, d)
    pkv.kv_append_fp8(x.cuda(), x.flip(0).contiguous().cuda(), slots.cuda(), *cache)
    for i, y in enumerate((x, x.flip(0))):
        codes, e = quantise(y)
        got = cache[i][0, 0, :14].cpu().double().numpy()
        assert np.array_equal(got, codes[:, 0], equal_nan=True)
        assert np.array_equal(cache[2][0, 0, i, :14].cpu().numpy(), e[:, 0])
    assert device_errors() == 0


def table(max_position, d):
    inverse = 1e4 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))
    angle = torch.arange(max_position, dtype=torch.float64)[:, None] * inverse
    return torch.cat([angle.cos(), angle.sin()], 1).float()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (9, 3), (32, 8), (8, 1)])
@pytest.mark.parametrize("axes,n", [(1, 1), (1, 70), (3, 37)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_append(d, hq, hkv, axes, n, in_place):
    g = torch.Generator().manual_seed(hq + n)
    nb = -(-n // BLOCK) + 2
    fused = rows(g, n, hq + 2 * hkv, d)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    pos = torch.randint(0, 500, (axes, n), generator=g)
    freq = pkv.rope_freq_axes([d // 2 - 16, 9, 7]) if axes == 3 else bytes(d // 2)
    slots = torch.randperm(nb * BLOCK, generator=g)[:n]
    if n > 4:
        slots[2] = -1
    cs = table(500, d)
    cache = empty_cache(nb, hkv, d)
    want_q, want_k = rotated_bits(q, pos.numpy(), list(freq), cs), rotated_bits(k, pos.numpy(), list(freq), cs)
    want = expect(cache, want_k, v, slots, nb)
    on = fused.cuda()
    q_on = on[:, :hq]
    out = q_on if in_place else torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    left = out[2].clone() if n > 4 else None
    got = pkv.rope_append_fp8(q_on, on[:, hq:hq + hkv], on[:, hq + hkv:], pos.cuda() if axes > 1 else pos[0].cuda(),
                              slots.cuda(), cs.cuda(), *cache, out, freq_axes=freq if axes > 1 else None)
    assert got is out
    same(cache, want)
    if n > 4:
        assert torch.equal(out[2], left)
        want_q[2] = left.cpu()
    assert torch.equal(out.cpu().view(torch.int16), want_q.view(torch.int16))
    assert device_errors() == 0


def test_rope_append_positions_outside_the_table():
    g = torch.Generator().manual_seed(4)
    q, k, v = (rows(g, 3, 2, 64) for _ in range(3))
    cs = table(10, 64)
    cache = empty_cache(2, 2, 64)
    out = torch.empty_like(q).cuda()
    pkv.rope_append_fp8(q.cuda(), k.cuda(), v.cuda(), torch.tensor([-3, 4, 10]).cuda(), torch.arange(3).cuda(), cs.cuda(), *cache, out)
    assert torch.equal(out.cpu(), rotated_bits(q, np.array([[0, 4, 9]]), [0] * 32, cs))
    assert device_errors() == pkv.DEVERR_POSITION_OUT_OF_TABLE


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("n", [1, 33, 5000])
def test_gather(d, hkv, n):
    g = torch.Generator().manual_seed(n)
    nb = -(-n // BLOCK) + 2
    cache = (torch.randint(0, 256, (nb, hkv, BLOCK, d), generator=g, dtype=torch.uint8),
             torch.randint(0, 256, (nb, hkv, BLOCK, d), generator=g, dtype=torch.uint8),
             torch.randint(0, 248, (nb, hkv, 2, BLOCK), generator=g, dtype=torch.uint8))
    slots = torch.randint(0, nb * BLOCK, (n,), generator=g)  # some twice
    if n > 4:
        slots[1] = -5
        slots[4] = nb * BLOCK
    wide = torch.full((n, 2 * hkv + 1, d), 3.0, dtype=torch.bfloat16, device="cuda")
    k, v = wide[:, :hkv], wide[:, hkv + 1:]
    on = [x.cuda() for x in cache]
    pkv.kv_gather_fp8(on[0].view(FP8), on[1].view(FP8), on[2], slots.cuda(), k, v)
    ok = (slots >= 0) & (slots < nb * BLOCK)
    at = slots[ok]
    for i, got in enumerate((k, v)):
        want = torch.full((n, hkv, d), 3.0, dtype=torch.float64)
        want[ok] = torch.from_numpy(values(cache[i][at // BLOCK, :, at % BLOCK], cache[2][at // BLOCK, :, i, at % BLOCK]))
        with np.errstate(over="ignore"):
            want = want.to(torch.bfloat16)
        assert np.array_equal(f64(got), f64(want), equal_nan=True)
    assert (wide[:, hkv] == 3.0).all()
    assert device_errors() == (pkv.DEVERR_SLOT_OUT_OF_RANGE if n > 4 else 0)


def test_gather_gives_back_what_was_appended():
    g = torch.Generator().manual_seed(6)
    n, hkv, d = 100, 4, 128
    # Rows that the format holds exactly: four significant bits, and magnitudes within 2^9 of each other.
    x = (torch.randint(8, 16, (2, n, hkv, d), generator=g) * 2.0 ** torch.randint(-4, 4, (2, n, hkv, d), generator=g)
         * torch.where(torch.rand(2, n, hkv, d, generator=g) < 0.5, -1.0, 1.0)).to(torch.bfloat16).cuda()
    cache = empty_cache(8, hkv, d)
    slots = torch.randperm(8 * BLOCK, generator=g)[:n].cuda()
    pkv.kv_append_fp8(x[0], x[1], slots, *cache)
    back = torch.zeros_like(x)
    pkv.kv_gather_fp8(*cache, slots, back[0], back[1])
    assert torch.equal(back, x)
    assert device_errors() == 0


@pytest.mark.parametrize("d,hkv", [(64, 1), (64, 3), (128, 8), (128, 5)])
@pytest.mark.parametrize("pairs", [1, 7, 600])
def test_copy_blocks(pairs, hkv, d):
    g = torch.Generator().manual_seed(pairs)
    nb = 2 * pairs + 3
    cache = [torch.randint(0, 256, s, generator=g, dtype=torch.uint8)
             for s in ((nb, hkv, BLOCK, d), (nb, hkv, BLOCK, d), (nb, hkv, 2, BLOCK))]
    order = torch.randperm(nb, generator=g)
    sd = torch.stack([order[torch.randint(0, pairs, (pairs,), generator=g)], order[pairs:2 * pairs]], 1)
    bad = torch.tensor([[-1, int(order[-1])], [0, nb], [nb, int(order[-1])], [0, -1]])
    on = [x.cuda() for x in cache]
    pkv.copy_blocks_fp8(on[0].view(FP8), on[1].view(FP8), on[2], torch.cat([sd, bad]).cuda())
    for x, got in zip(cache, on):
        x[sd[:, 1]] = x[sd[:, 0]]
        assert torch.equal(got.cpu(), x)
    assert device_errors() == pkv.DEVERR_COPY_OUT_OF_RANGE


def test_no_rows_and_no_pairs():
    cache = empty_cache(2, 2, 64)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    pkv.kv_append_fp8(none, none, slots, *cache)
    pkv.kv_gather_fp8(*cache, slots, none, none)
    pkv.copy_blocks_fp8(*cache, torch.empty(0, 2, dtype=torch.int64, device="cuda"))
    pkv.rope_append_fp8(none, none, none, slots, slots, table(4, 64).cuda(), *cache, none)
    assert device_errors() == 0


def test_refusals_of_the_tensors():
    cache = empty_cache(2, 2, 64)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(3, device="cuda")
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        pkv.kv_append_fp8(x, x, slots, cache[0].view(torch.uint8), cache[1], cache[2])
    with pytest.raises(ValueError, match="kv_scales must be"):
        pkv.kv_append_fp8(x, x, slots, cache[0], cache[1], cache[2][:1].contiguous())
    with pytest.raises(ValueError, match="k must be"):
        pkv.kv_append_fp8(x[:2], x, slots, *cache)
    with pytest.raises(ValueError, match="contiguous"):
        pkv.kv_append_fp8(x.repeat(1, 1, 2)[:, :, ::2], x, slots, *cache)
    with pytest.raises(TypeError):
        pkv.kv_gather_fp8(*cache, slots, x.float(), x)
    with pytest.raises(ValueError, match="src_dst"):
        pkv.copy_blocks_fp8(*cache, torch.zeros(2, 3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_append_fp8(x.cpu(), x, slots, *cache)
