"""The 8-bit cache's calls together, as a server uses them: prompts appended and attended to, sequences forked with their last
block copied before it is written, tokens decoded, drafted tokens checked, rows read back into a bf16 cache."""
import numpy as np
import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from fp8_plain import FP8, attend_fp8, quantise
from gpu_util import device_errors
from plain64 import BLOCK, assert_within, f64, rotated_bits

pytestmark = pytest.mark.gpu

HQ, HKV, D, POOL, SCALE = 8, 2, 128, 96, 0.09


class Model:
    """What every sequence's cache must hold, on the CPU: its rows' values in order."""

    def __init__(self):
        self.k, self.v = {}, {}

    def append(self, seq, k, v):
        for store, x in ((self.k, k), (self.v, v)):
            codes, e = quantise(x)
            rows = codes * 2.0 ** (e[..., None] - 127.0)
            store[seq] = np.concatenate([store[seq], rows]) if seq in store else rows

    def fork(self, parent, child):
        self.k[child], self.v[child] = self.k[parent].copy(), self.v[parent].copy()


class View:
    """A sequence of the model as attend_fp8 reads it: one block after the other."""

    def __init__(self, k, v):
        n = len(k)
        pad = -n % BLOCK
        shape = lambda x: np.concatenate([x, np.zeros((pad, *x.shape[1:]))]).reshape(-1, BLOCK, HKV, D).transpose(0, 2, 1, 3)  # noqa: E731
        self.kf, self.vf = shape(k), shape(v)
        self.table = np.arange(len(self.kf))[None]
        # The bound's exponents: those of rows of these values, at least.
        e = np.ceil(np.log2(np.maximum(np.abs(self.vf).max(-1), 2.0**-100) / 448)) + 127
        self.scales = torch.from_numpy(np.stack([e, e], 2).clip(0, 254)).to(torch.uint8)


def test_a_server_s_steps():
    g = torch.Generator().manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    manager, model = pkv.BlockManager(POOL), Model()
    kc = torch.full((POOL, HKV, BLOCK, D), 0x7F, dtype=torch.uint8).view(FP8).cuda()
    vc, sc = kc.clone(), torch.full((POOL, HKV, 2, BLOCK), 255, dtype=torch.uint8, device="cuda")
    inverse = 1e4 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))
    angle = torch.arange(4096, dtype=torch.float64)[:, None] * inverse
    cs = torch.cat([angle.cos(), angle.sin()], 1).float()

    def step(seqs, counts, slots):
        """Rotate and append each sequence's next tokens, attend, and check against the model."""
        n = sum(counts)
        q, k, v = randn(n, HQ, D), randn(n, HKV, D), randn(n, HKV, D)
        pos = np.concatenate([np.arange(c) + (len(model.k[s]) if s in model.k else 0) for s, c in zip(seqs, counts)])
        q_out = torch.empty_like(q).cuda()
        pkv.rope_append_fp8(q.cuda(), k.cuda(), v.cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(), cs.cuda(),
                            kc, vc, sc, q_out)
        turned, rk = rotated_bits(q, pos[None], [0] * (D // 2), cs), rotated_bits(k, pos[None], [0] * (D // 2), cs)
        assert torch.equal(q_out.cpu(), turned)
        at = np.concatenate([[0], np.cumsum(counts)])
        for i, s in enumerate(seqs):
            model.append(s, rk[at[i]:at[i + 1]], v[at[i]:at[i + 1]])
        width = max(-(-len(model.k[s]) // BLOCK) for s in seqs) + 1
        tables, lens = manager.block_tables(seqs, width)
        assert [len(model.k[s]) for s in seqs] == lens.tolist()
        out = torch.empty_like(q_out)
        args = (q_out, kc, vc, sc, torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda())
        decode = all(c == 1 for c in counts)
        if decode:
            pkv.paged_fp8_decode_attention(*args, SCALE, out)
        else:
            pkv.paged_fp8_prefill_attention(*args, torch.from_numpy(at.astype(np.int32)).cuda(), max(counts), SCALE, out)
        for i, s in enumerate(seqs):
            view = View(model.k[s], model.v[s])
            for r in range(counts[i]):
                ref, allowed = attend_fp8(view, 0, f64(turned)[at[i] + r], len(model.k[s]) - counts[i] + r + 1, SCALE,
                                          2.0**-11 if decode else 2.0**-8)
                assert_within(out[at[i] + r], ref, allowed, f"sequence {s}")

    prompts = {0: 100, 1: 33, 2: 1}
    step(list(prompts), list(prompts.values()), np.concatenate([manager.add_sequence(s, n) for s, n in prompts.items()]))
    for child in (10, 11, 12):  # samples of the first prompt, whose last block is partly filled
        manager.fork(0, child)
        model.fork(0, child)
    seqs = [0, 1, 2, 10, 11, 12]
    copied = 0
    for _ in range(5):
        slots, copies = manager.append_slots(seqs)
        copied += len(copies)
        if len(copies):
            pkv.copy_blocks_fp8(kc, vc, sc, torch.from_numpy(copies).cuda())
        step(seqs, [1] * len(seqs), slots)
    assert copied == 3
    for drafts in (2, 4):  # drafted tokens: their slots a token at a time, then one call for all
        slots = np.stack([manager.append_slots(seqs)[0] for _ in range(drafts)], 1).reshape(-1)
        step(seqs, [drafts] * len(seqs), slots)
    manager.free_sequence(11)
    # A sequence read back into a bf16 cache: the bf16 decode call there agrees with this one here.
    tables, lens = manager.block_tables([12], 8)
    n = int(lens[0])
    slots = torch.from_numpy(tables[0, np.arange(n) // BLOCK].astype(np.int64) * BLOCK + np.arange(n) % BLOCK).cuda()
    k, v = (torch.empty(n, HKV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.kv_gather_fp8(kc, vc, sc, slots, k, v)
    assert np.array_equal(f64(k), model.k[12]) and np.array_equal(f64(v), model.v[12])
    kb, vb = (torch.zeros(POOL, HKV, BLOCK, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.kv_append(k, v, slots, kb, vb)
    q = randn(1, HQ, D)
    ref, allowed = attend_fp8(View(model.k[12], model.v[12]), 0, f64(q)[0], n, SCALE, 2.0**-11)
    args = torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), SCALE
    for out in (pkv.paged_decode_attention(q.cuda(), kb, vb, *args, torch.empty_like(q).cuda()),
                pkv.paged_fp8_decode_attention(q.cuda(), kc, vc, sc, *args, torch.empty_like(q).cuda())):
        assert_within(out[0], ref, allowed, "read back")
    assert device_errors() == 0
