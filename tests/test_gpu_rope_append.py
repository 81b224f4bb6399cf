"""rope_append on the GPU: q_out and the caches bit for bit against the formula with every 32-bit operation rounded
on its own; rows and slots that the call does not own keep their bits."""
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from plain64 import rotated_bits
from workloads import make_decode_case, make_generator, randn_bf16, rope_cos_sin

pytestmark = pytest.mark.gpu


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16)


def inputs(n, hq, hkv, d, axes=1, packed=False, seed=0, max_position=300):
    g = make_generator(seed)
    if packed:  # one projection's output, wider than the three together
        rows = randn_bf16((n, hq + 2 * hkv + 1, d), g)
        q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:hq + 2 * hkv]
    else:
        q, k, v = randn_bf16((n, hq, d), g), randn_bf16((n, hkv, d), g), randn_bf16((n, hkv, d), g)
    positions = torch.randint(0, max_position, (axes, n), generator=g)
    freq_axes = torch.randint(0, axes, (d // 2,), generator=g).tolist()
    return q, k, v, positions, freq_axes, rope_cos_sin(max_position, d, 1e4)


def to_cuda(*views):
    """CUDA copies that keep strides and shared storage."""
    moved = {}
    out = []
    for t in views:
        base = t if t._base is None else t._base
        if id(base) not in moved:
            moved[id(base)] = base.cuda()
        out.append(moved[id(base)].as_strided(t.shape, t.stride(), t.storage_offset()))
    return out


def check(n, hq, hkv, d, axes=1, packed=False, in_place=False, seed=0, pad_every=0, blocks=None):
    q, k, v, positions, freq_axes, table = inputs(n, hq, hkv, d, axes, packed, seed)
    nb = blocks or -(-n // 16) + 5
    slots = torch.randperm(nb * 16, generator=make_generator(seed + 1))[:n]
    if pad_every:
        slots[::pad_every] = -1 - torch.arange(len(slots[::pad_every]))
        positions[:, ::pad_every] = -12345  # padding's positions are not looked at
    kc = torch.full((nb, hkv, 16, d), -3.5, dtype=torch.bfloat16)
    vc = torch.full_like(kc, 2.25)
    qg, kg, vg = to_cuda(q, k, v)
    kcg, vcg = kc.cuda(), vc.cuda()
    out = qg if in_place else torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    pos = positions.cuda() if axes > 1 else positions[0].cuda()
    got = pkv.rope_append(qg, kg, vg, pos, slots.cuda(), table.cuda(), kcg, vcg, out,
                          freq_axes=freq_axes if axes > 1 else None)
    assert got is out
    live = slots >= 0
    want_q = q.clone() if in_place else torch.full((n, hq, d), 7.0, dtype=torch.bfloat16)
    if live.any():
        want_q[live] = rotated_bits(q[live], positions[:, live], freq_axes, table)
        kc[slots[live] // 16, :, slots[live] % 16] = rotated_bits(k[live], positions[:, live], freq_axes, table)
        vc[slots[live] // 16, :, slots[live] % 16] = v[live]
    assert torch.equal(bits(out), bits(want_q))
    assert torch.equal(bits(kcg), bits(kc)) and torch.equal(bits(vcg), bits(vc))
    assert torch.equal(bits(vg), bits(v)) and torch.equal(bits(kg), bits(k))  # inputs as they were
    if not in_place:
        assert torch.equal(bits(qg), bits(q))
    assert device_errors() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 3), (8, 8), (32, 8), (40, 5), (64, 8)])
def test_layouts(hq, hkv, d):
    check(37, hq, hkv, d, seed=hq + d)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 700, 2049])
@pytest.mark.parametrize("packed", [False, True])
def test_lengths(n, packed):
    check(n, 16, 8, 128, packed=packed, seed=n)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 130])
def test_several_axes(axes, d, n):
    check(n, 8, 2, d, axes=axes, seed=axes)


@pytest.mark.parametrize("packed", [False, True])
def test_in_place(packed):
    check(100, 8, 4, 128, packed=packed, in_place=True, seed=5)


@pytest.mark.parametrize("pad_every", [1, 2, 7])
@pytest.mark.parametrize("axes", [1, 3])
def test_padding_is_left_alone(pad_every, axes):
    check(60, 8, 2, 64, axes=axes, pad_every=pad_every, seed=9)


def test_cache_rows_have_the_bits_of_the_fused_decode_step():
    c = make_decode_case("qwen3_0.6b", seed=3)
    a, b = c.to("cuda"), c.to("cuda")
    table = rope_cos_sin(c.block_tables.shape[1] * 16, c.q.shape[2], 1e6).cuda()
    out = torch.empty_like(a.q)
    pkv.decode_step(a.q, a.new_k, a.new_v, a.k_cache, a.v_cache, a.block_tables, a.context_lens, a.scale, out, table)
    q = torch.empty_like(b.q)
    pkv.rope_append(b.q, b.new_k, b.new_v, b.context_lens.long() - 1, b.slot_mapping, table, b.k_cache, b.v_cache, q)
    assert torch.equal(bits(a.k_cache), bits(b.k_cache)) and torch.equal(bits(a.v_cache), bits(b.v_cache))
    again = torch.empty_like(out)
    pkv.paged_decode_attention(q, b.k_cache, b.v_cache, b.block_tables, b.context_lens, b.scale, again)
    assert torch.allclose(out.float(), again.float(), rtol=2.0**-7, atol=1e-3)  # a step of bf16, and the sums' order
    assert device_errors() == 0


def test_positions_outside_the_table_are_flagged_and_clamped():
    q, k, v, _, freq_axes, table = inputs(4, 2, 1, 64, max_position=10)
    positions = torch.tensor([[-1, 9, 10, 1 << 40]])
    kc = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert device_errors() == 0
    pkv.rope_append(q.cuda(), k.cuda(), v.cuda(), positions[0].cuda(), torch.arange(4).cuda(), table.cuda(), kc,
                    kc.clone(), out)
    assert device_errors() == pkv.DEVERR_POSITION_OUT_OF_TABLE
    assert torch.equal(bits(out), bits(rotated_bits(q, [[0, 9, 9, 9]], freq_axes, table)))


def test_slots_past_the_pool_are_flagged_and_skipped():
    q, k, v, positions, freq_axes, table = inputs(3, 2, 1, 64)
    kc = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc, out = kc.clone(), torch.empty(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert device_errors() == 0
    pkv.rope_append(q.cuda(), k.cuda(), v.cuda(), positions[0].cuda(), torch.tensor([5, 32, 1 << 50]).cuda(),
                    table.cuda(), kc, vc, out)
    assert device_errors() == pkv.DEVERR_SLOT_OUT_OF_RANGE
    assert torch.equal(bits(out), bits(rotated_bits(q, positions, freq_axes, table)))
    want = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    want[0, :, 5] = v[0]
    assert torch.equal(bits(vc), bits(want))


def test_cache_offsets_past_32_bits():
    nb, hkv, d = 140_000, 8, 128  # 2.3e9 elements a cache
    q, k, v, positions, freq_axes, table = inputs(2, 8, hkv, d)
    kc = torch.empty(nb, hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    out = torch.empty(2, 8, d, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([nb * 16 - 1, 3])
    pkv.rope_append(q.cuda(), k.cuda(), v.cuda(), positions[0].cuda(), slots.cuda(), table.cuda(), kc, vc, out)
    want = rotated_bits(k, positions, freq_axes, table)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(bits(kc[s // 16, :, s % 16]), bits(want[i]))
        assert torch.equal(bits(vc[s // 16, :, s % 16]), bits(v[i]))
    assert device_errors() == 0


def test_another_stream_and_a_graph():
    n, hq, hkv, d = 50, 16, 8, 128
    q, k, v, positions, freq_axes, table = inputs(n, hq, hkv, d, axes=3)
    args = [t.cuda() for t in (q, k, v, positions, torch.arange(n), table)]
    kc = torch.zeros(4, hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    vc, out = kc.clone(), torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    want = rotated_bits(q, positions, freq_axes, table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pkv.rope_append(*args, kc, vc, out, freq_axes=bytes(freq_axes), stream=s)
    s.synchronize()
    assert torch.equal(bits(out), bits(want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pkv.rope_append(*args, kc, vc, out, freq_axes=freq_axes)
    for _ in range(2):
        out.zero_()
        g.replay()
        assert torch.equal(bits(out), bits(want))
    assert device_errors() == 0


def test_refusals():
    q, k, v, positions, _, table = (t.cuda() if isinstance(t, torch.Tensor) else t for t in inputs(4, 2, 1, 64))
    kc = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    slots, out, pos = torch.arange(4).cuda(), torch.empty_like(q), positions[0]
    call = pkv.rope_append
    with pytest.raises(ValueError, match="freq_axes"):
        call(q, k, v, torch.stack([pos, pos]), slots, table, kc, kc.clone(), out)
    with pytest.raises(ValueError, match="head_dim / 2"):
        call(q, k, v, torch.stack([pos, pos]), slots, table, kc, kc.clone(), out, freq_axes=[0, 1])
    with pytest.raises(pkv.PagedKVError, match="freq_axes"):
        call(q, k, v, torch.stack([pos, pos]), slots, table, kc, kc.clone(), out, freq_axes=[2] * 32)
    with pytest.raises(pkv.PagedKVError, match="num_axes"):
        call(q, k, v, torch.stack([pos] * 5), slots, table, kc, kc.clone(), out, freq_axes=[0] * 32)
    with pytest.raises(ValueError, match="positions"):
        call(q, k, v, pos.int(), slots, table, kc, kc.clone(), out)
    with pytest.raises(ValueError, match="contiguous"):
        call(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, pos, slots, table, kc, kc.clone(), out)
    with pytest.raises(ValueError, match="k must be"):
        call(q, q, v, pos, slots, table, kc, kc.clone(), out)
    with pytest.raises(TypeError, match="q_out"):
        call(q, k, v, pos, slots, table, kc, kc.clone(), out.float())
    with pytest.raises(pkv.PagedKVError, match="aligned"):
        odd = torch.empty(4 * 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 2, 64)
        call(odd, k, v, pos, slots, table, kc, kc.clone(), out)
    with pytest.raises(pkv.PagedKVError, match="stride"):
        wide = torch.empty(4, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, :128].unflatten(1, (2, 64))
        call(wide, k, v, pos, slots, table, kc, kc.clone(), out)
    with pytest.raises(ValueError, match="cos_sin"):
        call(q, k, v, pos, slots, table[:, :32].contiguous(), kc, kc.clone(), out)
    assert device_errors() == 0
