"""The operators together, as a server runs a layer: prompts rotated and appended in chunks and attended with a window,
forks of one prompt decoded behind it, each against the definition in 64 bits on the rows that were really cached."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from plain64 import assert_within, attend, f64, rotated_bits, sees
from workloads import make_generator, randn_bf16, rope_cos_sin

pytestmark = pytest.mark.gpu

HQ, HKV, D, SCALE = 8, 2, 128, 128 ** -0.5


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Layer:
    """One layer's cache, the block manager over it, and what was projected for every cached token."""

    def __init__(self, blocks, seed):
        self.bm = pkv.BlockManager(blocks, np.random.RandomState(seed).permutation(blocks))
        self.k = torch.zeros(blocks, HKV, 16, D, dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.table = rope_cos_sin(2048, D, 1e4)
        self.table_gpu = self.table.cuda()
        self.g = make_generator(seed)

    def project(self, positions, slots):
        """Projects, rotates and appends a batch of tokens; returns the rotated queries."""
        n = len(slots)
        qkv = randn_bf16((n, HQ + 2 * HKV, D), self.g)
        gpu = qkv.cuda()
        q = torch.empty(n, HQ, D, dtype=torch.bfloat16, device="cuda")
        pkv.rope_append(gpu[:, :HQ], gpu[:, HQ:HQ + HKV], gpu[:, HQ + HKV:], torch.as_tensor(positions).cuda(),
                        torch.as_tensor(slots).cuda(), self.table_gpu, self.k, self.v, q)
        assert torch.equal(q.cpu(), rotated_bits(qkv[:, :HQ], [positions], [0] * (D // 2), self.table))
        return q

    def exact(self, q, tables, positions, window, sinks, extra):
        k, v, qf = f64(self.k), f64(self.v), f64(q)
        rows = [attend(qf[i], k, v, tables[i], sees(p, window, sinks), SCALE, extra) for i, p in enumerate(positions)]
        return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


@pytest.mark.parametrize("window,sinks", [(40, 4), (17, 0)])
def test_prompt_chunks_then_decode_with_a_window(window, sinks):
    layer = Layer(64, 1)
    prompts = (150, 61)
    slots = [layer.bm.add_sequence(b, n) for b, n in enumerate(prompts)]
    tables, _ = layer.bm.block_tables([0, 1], 16)
    gpu_table = torch.from_numpy(tables).cuda()
    done = [0, 0]
    for chunk in ((64, 61), (86, 0)):  # the second prompt is in whole after the first chunk
        rows = [(b, p) for b in (0, 1) for p in range(done[b], done[b] + chunk[b])]
        q = layer.project(np.array([p for _, p in rows]), np.array([slots[b][p] for b, p in rows]))
        done = [d + c for d, c in zip(done, chunk)]
        out = torch.empty_like(q)
        pkv.paged_window_prefill_attention(q, layer.k, layer.v, gpu_table, i32(done), i32([0, chunk[0], sum(chunk)]),
                                           max(chunk), SCALE, out, window, sinks)
        ref, allowed = layer.exact(q, [tables[b] for b, _ in rows], [p for _, p in rows], window, sinks, 2.0**-8)
        assert_within(out, ref, allowed, f"chunk {chunk}")
    for _ in range(20):  # single tokens, over a block's border
        new, _ = layer.bm.append_slots([0, 1])
        tables, lens = layer.bm.block_tables([0, 1], 16)
        q = layer.project(lens.astype(np.int64) - 1, new)
        out = torch.empty_like(q)
        pkv.paged_window_decode_attention(q, layer.k, layer.v, torch.from_numpy(tables).cuda(), i32(lens.tolist()), SCALE,
                                          out, window, sinks)
        ref, allowed = layer.exact(q, tables, lens - 1, window, sinks, 0.0)
        assert_within(out, ref, allowed, "step")
    assert device_errors() == 0


def test_forks_of_one_prompt_decode_behind_it():
    layer = Layer(96, 2)
    n = 203  # the last block is shared and partly filled: the first step copies it for every fork but one
    slots = layer.bm.add_sequence(0, n)
    layer.project(np.arange(n), slots)
    ids = list(range(6))
    for child in ids[1:]:
        layer.bm.fork(0, child)
    for _ in range(18):
        new, copies = layer.bm.append_slots(ids)
        if len(copies):
            pkv.copy_blocks(layer.k, layer.v, torch.from_numpy(copies).cuda())
        tables, lens = layer.bm.block_tables(ids, 16)
        q = layer.project(lens.astype(np.int64) - 1, new)
        args = (q, layer.k, layer.v, torch.from_numpy(tables).cuda(), i32(lens.tolist()))
        out, plain = torch.empty_like(q), torch.empty_like(q)
        pkv.paged_prefix_decode_attention(*args, i32([0, len(ids)]), i32([n]), SCALE, out)
        ref, allowed = layer.exact(q, tables, lens - 1, None, 0, 2.0**-8)
        assert_within(out, ref, allowed, "step behind the prompt")
        pkv.paged_decode_attention(*args, SCALE, plain)
        assert_within(plain, ref, allowed, "the same without sharing")
    assert device_errors() == 0
