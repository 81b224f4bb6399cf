"""Attention and rotation from their formulas in 64 bits, a row at a time, for the parity tests (not a test module)."""
from __future__ import annotations

import numpy as np
import torch

BLOCK = 16


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def sees(position: int, window: int | None = None, sinks: int = 0) -> np.ndarray:
    """Cached tokens that a query at `position` sees."""
    j = np.arange(position + 1)
    return j if window is None else j[(j > position - window) | (j < sinks)]


def attend(q, k_cache, v_cache, table_row, keys, scale, extra: float):
    """Rows q [Hq, D] over the cached tokens `keys` of one sequence.

    Returns (out, allowed), both [Hq, D]: the exact result, and how far the kernel's may be from it:

    * 2^-8 |out|: the output's rounding to bf16 (half a step);
    * `extra` sum p |v|: a rounding of each weight (2^-8 where the weights enter the product as bf16, 0 where
      they stay in 32 bits or in two bf16 parts);
    * c sum p |v|, the 32-bit arithmetic: a score's error is at most (D + 4) 2^-23 of |scale| sum |q| |k| (a
      product and a sum each may be off by 2^-23, truncation included) and enters weight and normaliser, so
      twice; the exponential and its argument's rounding are off by 2^-22 (1 + |score|); the sums over n keys
      by n 2^-24 each, twice; a weight in two bf16 parts by 2^-16.
    """
    hq, d = q.shape
    hkv = k_cache.shape[1]
    group = hq // hkv
    out, allowed = np.zeros((hq, d)), np.zeros((hq, d))
    if len(keys) == 0:
        return out, allowed
    blocks = np.asarray(table_row)[keys // BLOCK]
    k, v = k_cache[blocks, :, keys % BLOCK], v_cache[blocks, :, keys % BLOCK]  # [n, Hkv, D]
    for h in range(hq):
        kh, vh = k[:, h // group], v[:, h // group]
        s = scale * (kh @ q[h])
        p = np.exp(s - s.max())
        p /= p.sum()
        out[h] = p @ vh
        largest = abs(scale) * (np.abs(kh) @ np.abs(q[h])).max()
        c = 2 * (d + 4) * 2.0**-23 * largest + 2 * 2.0**-22 * (1 + largest) + 2 * len(keys) * 2.0**-24 + 2.0**-16
        allowed[h] = 2.0**-8 * np.abs(out[h]) + (extra + c) * (p @ np.abs(vh))
    return out, allowed


def assert_within(got: torch.Tensor, out: np.ndarray, allowed: np.ndarray, what: str = "") -> None:
    g = f64(got)
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    over = np.abs(g - out) - allowed
    at = np.unravel_index(over.argmax(), over.shape)
    assert over.max() <= 0, f"{what}: at {at} got {g[at]}, exact {out[at]}, allowed {allowed[at]}"


def rotated_bits(x: torch.Tensor, positions, freq_axes, cos_sin: torch.Tensor) -> torch.Tensor:
    """x [N, H, D] bf16 rotated: every product, difference and sum rounded to 32 bits, then to bf16.

    positions: [axes][N]; freq_axes: the axis of each of the D / 2 frequencies.
    """
    d = x.shape[-1]
    half = d // 2
    a, b = x[..., :half].float().numpy(), x[..., half:].float().numpy()
    pos = np.asarray(positions)[np.asarray(freq_axes)].T  # [N, D / 2]
    table = cos_sin.numpy()
    c, n = table[pos, np.arange(half)][:, None], table[pos, half + np.arange(half)][:, None]
    assert a.dtype == np.float32 and c.dtype == np.float32
    y = np.concatenate([a * c - b * n, b * c + a * n], -1)
    return torch.from_numpy(y).to(torch.bfloat16)


class Pages:
    """Sequences' blocks drawn from one shuffled pool; blocks that nothing was drawn for hold NaN."""

    def __init__(self, lens, hkv: int, d: int, seed: int, spare: int = 3, width: int | None = None):
        self.g = torch.Generator().manual_seed(seed)
        counts = [-(-int(n) // BLOCK) for n in lens]
        self.pool = sum(counts) + spare
        order = torch.randperm(self.pool, generator=self.g).tolist()
        self.lens = [int(n) for n in lens]
        self.width = width or max([1, *counts])
        self.table = np.full((len(counts), self.width), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.k = torch.full((self.pool, hkv, BLOCK, d), float("nan"), dtype=torch.bfloat16)
        self.v = self.k.clone()
        for b, n in enumerate(self.lens):
            self.fill(b, range(n))

    def randn(self, *shape) -> torch.Tensor:
        return torch.randn(*shape, generator=self.g).to(torch.bfloat16)

    def fill(self, b: int, tokens) -> None:
        """Values for these tokens of sequence b."""
        t = np.fromiter(tokens, dtype=np.int64)
        blocks = self.table[b, t // BLOCK].astype(np.int64)
        _, hkv, _, d = self.k.shape
        self.k[blocks, :, t % BLOCK] = self.randn(len(t), hkv, d)
        self.v[blocks, :, t % BLOCK] = self.randn(len(t), hkv, d)

    def poison(self, b: int, tokens, value: float = float("nan")) -> None:
        t = np.fromiter(tokens, dtype=np.int64)
        blocks = self.table[b, t // BLOCK].astype(np.int64)
        self.k[blocks, :, t % BLOCK] = value
        self.v[blocks, :, t % BLOCK] = value

    def cuda(self):
        return (self.k.cuda(), self.v.cuda(), torch.from_numpy(self.table).cuda(),
                torch.tensor(self.lens, dtype=torch.int32).cuda())
