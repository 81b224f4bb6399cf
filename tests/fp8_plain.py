"""The 8-bit cache's format and attention over it from their definitions in 64 bits, for the tests (not a test module)."""
from __future__ import annotations

import numpy as np
import torch

from plain64 import BLOCK, Pages, attend, f64

FP8 = torch.float8_e4m3fn

# The values of the 256 codes: sign, four exponent bits of bias 7, three mantissa bits; 0x7f and 0xff are NaN.
_BITS = np.arange(256)
_EXP, _MAN = (_BITS >> 3) & 15, _BITS & 7
CODES = np.where(_EXP > 0, (8 + _MAN) * 2.0 ** (_EXP - 10.0), _MAN * 2.0 ** -9) * np.where(_BITS & 128, -1.0, 1.0)
CODES[[0x7F, 0xFF]] = np.nan


def quantise(x: torch.Tensor) -> tuple[np.ndarray, np.ndarray]:
    """Code values [..., D] (not scaled) and exponent bytes [...] of bf16 rows, by search: the first exponent that is large
    enough, and of the values that the type has the nearest, the even code of two."""
    x = f64(x)
    finite = np.where(np.isfinite(x), np.abs(x), 0.0)
    limits = 448.0 * 2.0 ** np.arange(-127.0, 128.0)
    e = np.searchsorted(limits, finite.max(-1))
    y = np.where(np.isfinite(x), x, 0.0) * 2.0 ** (127.0 - e)[..., None]
    grid = CODES[:0x7F]  # the magnitudes, rising
    hi = np.searchsorted(grid, np.abs(y)).clip(0, 0x7E)
    lo = (hi - 1).clip(0)
    below, above = np.abs(y) - grid[lo], grid[hi] - np.abs(y)
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isfinite(x), np.copysign(grid[code], y), np.nan), e.astype(np.int64)


def values(codes: torch.Tensor, exponents: torch.Tensor) -> np.ndarray:
    """What codes [..., D] and exponent bytes [...] stand for."""
    return CODES[codes.cpu().view(torch.uint8).numpy()] * (2.0 ** (exponents.cpu().numpy().astype(np.float64) - 127))[..., None]


def to_cache(k: torch.Tensor, v: torch.Tensor):
    """The 8-bit caches and exponents of bf16 caches [NB, Hkv, 16, D], on the CPU."""
    out, scales = [], []
    for x in (k, v):
        codes, e = quantise(x)
        out.append(torch.from_numpy(codes).float().to(FP8))
        scales.append(torch.from_numpy(e).to(torch.uint8))
    return *out, torch.stack(scales, 2).contiguous()


class Fp8Pages(Pages):
    """Sequences in an 8-bit cache; what no token was drawn for holds NaN codes and the largest exponent."""

    def __init__(self, lens, hkv: int, d: int, seed: int, spare: int = 3, width: int | None = None, spread: float = 1.0):
        self.spread = spread
        super().__init__(lens, hkv, d, seed, spare, width)
        self.quantise()

    def fill(self, b, tokens):
        super().fill(b, tokens)
        t = np.fromiter(tokens, dtype=np.int64)
        blocks = self.table[b, t // BLOCK].astype(np.int64)
        for x in (self.k, self.v):  # rows of different sizes
            size = torch.exp2(torch.randn(len(t), x.shape[1], 1, generator=self.g) * self.spread).to(torch.bfloat16)
            x[blocks, :, t % BLOCK] = x[blocks, :, t % BLOCK] * size

    def quantise(self):
        self.k8, self.v8, self.scales = to_cache(self.k, self.v)
        for i, x in enumerate((self.k, self.v)):
            self.scales[:, :, i][torch.isnan(x).all(-1)] = 255
        self.kf, self.vf = values(self.k8, self.scales[:, :, 0]), values(self.v8, self.scales[:, :, 1])

    def cuda(self):
        return (self.k8.cuda(), self.v8.cuda(), self.scales.cuda(), torch.from_numpy(self.table).cuda(),
                torch.tensor(self.lens, dtype=torch.int32).cuda())


def attend_fp8(pages: Fp8Pages, b: int, q: np.ndarray, n: int, scale: float, weight: float):
    """Rows q [Hq, D] over the first n tokens of sequence b: (out, allowed) as plain64.attend, with `weight` the rounding of a
    weight relative to itself.  Weights in 16 bits besides have an absolute rounding of 2^-32 of the largest weight times its
    row's scale (the largest is brought above 2^7, half the type's least step is 2^-25), times a code of up to 448."""
    keys = np.arange(n)
    out, allowed = attend(q, pages.kf, pages.vf, pages.table[b], keys, scale, weight)
    if n:
        blocks = pages.table[b][keys // BLOCK]
        size = 448.0 * 2.0 ** (pages.scales[blocks, :, 1, keys % BLOCK].numpy().astype(np.float64) - 127)  # [n, Hkv]
        group = q.shape[0] // size.shape[1]
        for h in range(q.shape[0]):
            s = scale * (pages.kf[blocks, h // group, keys % BLOCK] @ q[h])
            p = np.exp(s - s.max())
            allowed[h] += n * 2.0**-32 * (p / p.sum() * size[:, h // group]).max()
    return out, allowed
