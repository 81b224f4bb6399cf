"""Measured cases of the paged cache in 8 bits: quantising append, reading back, block copies, decode and chunk attention.

Five operators, each in a plain form of elementary torch operations in 32 bits (``own = False``) and as the
framework's own calls (``own = True``):

    append_fp8    quantise each new token's k and v rows as they are written into the paged cache; with ``rotary`` the
                  rotation of q and k at the tokens' positions goes before it, q to its own buffer
    gather_fp8    read cached rows back as bf16, by slot
    copy_fp8      copy whole blocks inside the pool (copy-on-write of forked sequences)
    decode_fp8    one query token a sequence over its cached tokens
    prefill_fp8   chunks of query tokens, causal, over the cached tokens and the chunk's own

The format: a row of one kv head (head_dim values) is held as e4m3 codes and one exponent byte e, and stands for
code * 2^(e - 127).  With a the row's largest magnitude, e - 127 is the least integer s >= -127 with a <= 448 * 2^s, and
the codes are x * 2^-s rounded to nearest even.  Caches are float8_e4m3fn [blocks, kv heads, 16, head_dim], their
exponents uint8 [blocks, kv heads, 2, 16], K's sixteen and then V's.

Sequences, lengths and block tables are drawn so that a case's amount of work is fixed by the case: the lengths of a
batch are spread evenly over their range and only their order, the block ids and the values go by the seed.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
DEVICE = "cuda"
FP8 = torch.float8_e4m3fn


# ----------------------------------------------------------------------------
# The cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # The attention input of one decode step of a small model: eight sequences, latency alone.
        dict(name="append_fp8 decode 8", op="append_fp8", tokens=8, pad=0, hq=16, hkv=8, d=128, rotary=True, packed=True,
             max_position=32768),
        # Whole prompts appended at once, a padded batch, k and v as separate tensors.
        dict(name="append_fp8 prompts 32773", op="append_fp8", tokens=32773, pad=27, hq=32, hkv=8, d=128, rotary=False,
             packed=False, max_position=32768),
        # One short sequence read back: latency alone.
        dict(name="gather_fp8 777", op="gather_fp8", tokens=777, pad=0, hkv=8, d=128),
        # A batch of prompts' rows read back, of small heads.
        dict(name="gather_fp8 65536", op="gather_fp8", tokens=65536, pad=5, hkv=8, d=64),
        # The copies of one decode step: a few forked sequences write into a shared block.
        dict(name="copy_fp8 4", op="copy_fp8", pairs=4, hkv=8, d=128),
        # Many samples of many prompts fork at once.
        dict(name="copy_fp8 2048", op="copy_fp8", pairs=2048, hkv=8, d=128),
        # A single chat sequence: latency alone.
        dict(name="decode_fp8 1", op="decode_fp8", seqs=1, len_lo=4097, len_hi=4097, hq=16, hkv=8, d=128),
        # A serving batch of one layer.
        dict(name="decode_fp8 128", op="decode_fp8", seqs=128, len_lo=512, len_hi=4096, hq=32, hkv=8, d=128),
        # A batch of very different lengths, eight q heads to a kv head, small heads.
        dict(name="decode_fp8 61 long", op="decode_fp8", seqs=61, len_lo=16, len_hi=65536, hq=64, hkv=8, d=64),
        # One chunk of a single long sequence: too few tiles to fill the GPU.
        dict(name="prefill_fp8 1x512", op="prefill_fp8", seqs=1, chunk_lo=512, chunk_hi=512, past_lo=8192, past_hi=8192,
             hq=16, hkv=8, d=128),
        # Drafted tokens of a serving batch checked at once: a few rows a sequence over a long cache.
        dict(name="prefill_fp8 64 drafts", op="prefill_fp8", seqs=64, chunk_lo=1, chunk_hi=5, past_lo=512, past_hi=8192,
             hq=32, hkv=8, d=128),
        # Whole long prompts, no tokens cached.
        dict(name="prefill_fp8 2x8192", op="prefill_fp8", seqs=2, chunk_lo=8192, chunk_hi=8192, past_lo=0, past_hi=0,
             hq=32, hkv=8, d=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hkv = rng.choice([1, 2, 3, 4, 8])
    heads = dict(hq=hkv * rng.choice([1, 2, 4, 8]), hkv=hkv, d=rng.choice([64, 128]))
    op = rng.choice(["append_fp8", "gather_fp8", "copy_fp8", "decode_fp8", "decode_fp8", "prefill_fp8", "prefill_fp8"])
    if op == "append_fp8":
        return dict(op=op, tokens=_log_int(rng, 1, 32768), pad=rng.choice([0, 0, 1, 5]), **heads,
                    rotary=rng.random() < 0.5, packed=rng.random() < 0.5, max_position=32768)
    if op == "gather_fp8":
        return dict(op=op, tokens=_log_int(rng, 1, 65536), pad=rng.choice([0, 0, 1, 5]), hkv=hkv, d=heads["d"])
    if op == "copy_fp8":
        return dict(op=op, pairs=_log_int(rng, 1, 2048), hkv=hkv, d=heads["d"])
    if op == "decode_fp8":
        lens = sorted(_log_int(rng, 1, 8192) for _ in range(2))
        return dict(op=op, seqs=_log_int(rng, 1, 128), len_lo=lens[0], len_hi=lens[1], **heads)
    past = sorted(rng.randint(0, 4096) for _ in range(2))
    if rng.random() < 0.4:
        chunk = sorted(rng.randint(1, 8) for _ in range(2))
        return dict(op=op, seqs=_log_int(rng, 1, 64), chunk_lo=chunk[0], chunk_hi=chunk[1], past_lo=past[0],
                    past_hi=past[1], **heads)
    chunk = sorted(_log_int(rng, 1, 2048) for _ in range(2))
    return dict(op=op, seqs=rng.randint(1, 8), chunk_lo=chunk[0], chunk_hi=chunk[1], past_lo=past[0], past_hi=past[1],
                **heads)


# ----------------------------------------------------------------------------
# Sizes that a case fixes
# ----------------------------------------------------------------------------
def _even(lo, hi, n):
    """n lengths spread evenly over [lo, hi] (over their logarithm where it spans more than a factor of ten)."""
    if lo > 0 and hi > 10 * lo:
        return np.rint(np.exp(np.linspace(math.log(lo), math.log(hi), n))).astype(np.int64)
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64)


def work(case):
    hkv, d, op = case["hkv"], case["d"], case["op"]
    row = 2 * hkv * (d + 1)  # one token's codes and exponents
    if op == "append_fp8":
        n, hq = case["tokens"], case["hq"]
        bytes_, flops = n * (4 * hkv * d + row + 8), 2 * n * hkv * d
        if case["rotary"]:  # q read and written, the position and the rotation's angles
            bytes_, flops = bytes_ + n * (4 * hq * d + 8 + 4 * d), flops + 3 * n * (hq + hkv) * d
        return dict(bytes=bytes_, flops=flops)
    if op == "gather_fp8":
        return dict(bytes=case["tokens"] * (row + 4 * hkv * d + 8), flops=2 * case["tokens"] * hkv * d)
    if op == "copy_fp8":
        return dict(bytes=case["pairs"] * (2 * BLOCK * row + 16), flops=0)
    hq = case["hq"]
    if op == "decode_fp8":
        seen = int(_even(case["len_lo"], case["len_hi"], case["seqs"]).sum())
        return dict(bytes=seen * row + case["seqs"] * (4 * hq * d + 4) + seen // BLOCK * 4, flops=4 * seen * hq * d)
    past, chunk = (_even(case[x + "_lo"], case[x + "_hi"], case["seqs"]) for x in ("past", "chunk"))
    seen = int((chunk * past + chunk * (chunk + 1) // 2).sum())
    tokens = int((past + chunk).sum())
    return dict(bytes=tokens * row + int(chunk.sum()) * 4 * hq * d + tokens // BLOCK * 4, flops=4 * seen * hq * d)


# ----------------------------------------------------------------------------
# The format, in elementary operations
# ----------------------------------------------------------------------------
def _quantised(x):
    """Codes [..., D] and exponent bytes [...] of rows x [..., D] in 32 bits."""
    top = x.abs().amax(-1)
    mantissa, exponent = torch.frexp(top)  # top = mantissa 2^exponent, mantissa in [1/2, 1)
    s = torch.where(mantissa <= 0.875, exponent - 9, exponent - 8).clamp(min=-127)
    s = torch.where(top > 0, s, torch.full_like(s, -127))
    return torch.ldexp(x, -s[..., None]).to(FP8), (s + 127).to(torch.uint8)


def _scale(exponents):
    """2^(e - 127) in 32 bits."""
    return torch.ldexp(torch.ones_like(exponents, dtype=torch.float32), exponents.int() - 127)


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32).to(torch.bfloat16)


def _rows(gen, *shape):
    """Rows whose sizes differ, as those of a model's keys and values do from token to token and head to head."""
    size = torch.exp2(torch.randn(*shape[:-1], 1, generator=gen, device=DEVICE))
    return (torch.randn(*shape, generator=gen, device=DEVICE) * size).to(torch.bfloat16)


def _caches(gen, blocks, hkv, d):
    k, ke = _quantised(_rows(gen, blocks, hkv, BLOCK, d).float())
    v, ve = _quantised(_rows(gen, blocks, hkv, BLOCK, d).float())
    return dict(k_cache=k, v_cache=v, kv_scales=torch.stack([ke, ve], 2).contiguous())


def _tables(gen, lens, pool, width):
    """Block tables [seqs, width] of distinct blocks in random order, -1 behind each sequence's last block."""
    counts = torch.as_tensor(-(-lens // BLOCK), device=DEVICE)
    starts = torch.cumsum(counts, 0) - counts
    order = torch.randperm(pool, generator=gen, device=DEVICE)
    col = torch.arange(width, device=DEVICE)
    inside = col[None, :] < counts[:, None]
    flat = torch.where(inside, starts[:, None] + col[None, :], torch.zeros((), dtype=torch.long, device=DEVICE))
    return torch.where(inside, order[flat], torch.full((), -1, dtype=torch.long, device=DEVICE)).to(torch.int32)


def _slots(gen, tokens, total, blocks):
    """Slots of `tokens` consecutive tokens in blocks of random order; padding (-1) behind them."""
    at = torch.arange(total, device=DEVICE)
    slots = torch.randperm(blocks, generator=gen, device=DEVICE)[at // BLOCK] * BLOCK + at % BLOCK
    slots[tokens:] = -1
    return slots


def _int32(values):
    return torch.as_tensor(np.asarray(values), device=DEVICE).to(torch.int32)


def _append_state(case, gen, rng):
    n, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    total = n + case["pad"]
    if case["packed"]:  # views of the fused projection's output
        rows = _rows(gen, total, hq + 2 * hkv, d)
        q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    else:
        q, k, v = _rows(gen, total, hq, d), _rows(gen, total, hkv, d), _rows(gen, total, hkv, d)
    blocks = -(-total // BLOCK) + 8
    state = dict(k=k, v=v, slots=_slots(gen, n, total, blocks), **_caches(gen, blocks, hkv, d))
    if case["rotary"]:
        # Chunks of up to 512 consecutive tokens, each from a random position on.
        at = torch.arange(total, device=DEVICE)
        start = torch.randint(0, case["max_position"] - 512, (total // 512 + 1,), generator=gen, device=DEVICE)
        inverse = 5e5 ** (-torch.arange(d // 2, device=DEVICE, dtype=torch.float64) / (d // 2))
        angle = torch.arange(case["max_position"], device=DEVICE, dtype=torch.float64)[:, None] * inverse
        state.update(q=q, positions=start[at // 512] + at % 512, cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(),
                     q_out=torch.zeros(total, hq, d, dtype=torch.bfloat16, device=DEVICE))
    return state


def _gather_state(case, gen, rng):
    total = case["tokens"] + case["pad"]
    blocks = -(-total // BLOCK) + 8
    out = torch.zeros(2, total, case["hkv"], case["d"], dtype=torch.bfloat16, device=DEVICE)
    return dict(slots=_slots(gen, case["tokens"], total, blocks), k=out[0], v=out[1],
                **_caches(gen, blocks, case["hkv"], case["d"]))


def _copy_state(case, gen, rng):
    n = case["pairs"]
    # Samples of one prompt share a source; every copy has a block of its own.
    order = torch.randperm(2 * n + 8, generator=gen, device=DEVICE)
    source = order[torch.randint(0, max(1, n // 2), (n,), generator=gen, device=DEVICE)]
    return dict(src_dst=torch.stack([source, order[n:2 * n]], 1).contiguous(), **_caches(gen, 2 * n + 8, case["hkv"], case["d"]))


def _attention_state(case, gen, lens, rows):
    pool = int((-(-lens // BLOCK)).sum()) + 4
    q = _normal(gen, rows, case["hq"], case["d"])
    return dict(q=q, table=_tables(gen, lens, pool, -(-int(lens.max()) // BLOCK)), lens=_int32(lens), out=torch.empty_like(q),
                most_keys=int(lens.max()), scale=case["d"] ** -0.5, **_caches(gen, pool, case["hkv"], case["d"]))


def _decode_state(case, gen, rng):
    return _attention_state(case, gen, rng.permutation(_even(case["len_lo"], case["len_hi"], case["seqs"])), case["seqs"])


def _prefill_state(case, gen, rng):
    order = rng.permutation(case["seqs"])
    past = _even(case["past_lo"], case["past_hi"], case["seqs"])[order]
    chunk = _even(case["chunk_lo"], case["chunk_hi"], case["seqs"])[order]
    return dict(_attention_state(case, gen, past + chunk, int(chunk.sum())), most_rows=int(chunk.max()),
                query_start=_int32(np.concatenate([[0], np.cumsum(chunk)])))


_STATES = dict(append_fp8=_append_state, gather_fp8=_gather_state, copy_fp8=_copy_state, decode_fp8=_decode_state,
               prefill_fp8=_prefill_state)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    return dict(_STATES[case["op"]](case, gen, np.random.RandomState(seed % (1 << 32))), case=case)


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state["case"]["op"], state["case"], state)


def _run_own(op, case, s):
    import paged_kv_cache_275_gb300 as pkv

    cache = s["k_cache"], s["v_cache"], s["kv_scales"]
    if op == "append_fp8":
        if case["rotary"]:
            return pkv.rope_append_fp8(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos_sin"], *cache,
                                       s["q_out"]), *cache
        pkv.kv_append_fp8(s["k"], s["v"], s["slots"], *cache)
        return cache
    if op == "gather_fp8":
        pkv.kv_gather_fp8(*cache, s["slots"], s["k"], s["v"])
        return s["k"], s["v"]
    if op == "copy_fp8":
        pkv.copy_blocks_fp8(*cache, s["src_dst"])
        return cache
    if op == "decode_fp8":
        return pkv.paged_fp8_decode_attention(s["q"], *cache, s["table"], s["lens"], s["scale"], s["out"])
    return pkv.paged_fp8_prefill_attention(s["q"], *cache, s["table"], s["lens"], s["query_start"], s["most_rows"],
                                           s["scale"], s["out"])


def _run_plain(op, case, s):
    return dict(append_fp8=_plain_append, gather_fp8=_plain_gather, copy_fp8=_plain_copy, decode_fp8=_plain_decode,
                prefill_fp8=_plain_prefill)[op](case, s)


def _plain_append(case, s):
    n, d = case["tokens"], case["d"]
    k, outputs = s["k"][:n].float(), ()
    if case["rotary"]:
        table = s["cos_sin"][s["positions"][:n]]
        cos, sin = table[:, None, :d // 2], table[:, None, d // 2:]

        def turned(x):
            a, b = x[:n, :, :d // 2].float(), x[:n, :, d // 2:].float()
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)

        s["q_out"][:n] = turned(s["q"])
        k, outputs = turned(s["k"]).float(), (s["q_out"],)
    block, offset = s["slots"][:n] // BLOCK, s["slots"][:n] % BLOCK
    for i, (x, cache) in enumerate(((k, s["k_cache"]), (s["v"][:n].float(), s["v_cache"]))):
        codes, exponents = _quantised(x)
        cache.view(torch.uint8)[block, :, offset] = codes.view(torch.uint8)
        s["kv_scales"][block, :, i, offset] = exponents
    return *outputs, s["k_cache"], s["v_cache"], s["kv_scales"]


def _dequantised(s, i, block, offset):
    """Rows of K (i = 0) or V (i = 1) in 32 bits: those of all kv heads, of the given blocks and rows."""
    codes = s["v_cache" if i else "k_cache"].view(torch.uint8)[block, :, offset].view(FP8).float()
    return codes * _scale(s["kv_scales"][block, :, i, offset])[..., None]


def _plain_gather(case, s):
    n = case["tokens"]
    block, offset = s["slots"][:n] // BLOCK, s["slots"][:n] % BLOCK
    s["k"][:n] = _dequantised(s, 0, block, offset).to(torch.bfloat16)
    s["v"][:n] = _dequantised(s, 1, block, offset).to(torch.bfloat16)
    return s["k"], s["v"]


def _plain_copy(case, s):
    source, target = s["src_dst"][:, 0], s["src_dst"][:, 1]
    for cache in (s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8), s["kv_scales"]):
        cache[target] = cache[source]
    return s["k_cache"], s["v_cache"], s["kv_scales"]


def _gathered(s, i, pos):
    """Cache rows [seqs, n, kv heads, d] of the positions [seqs, n], in 32 bits."""
    block = s["table"].gather(1, pos // BLOCK).clamp(min=0).long()
    return _dequantised(s, i, block, pos % BLOCK)


def _weights(scores, seen):
    """Softmax over the last axis of the scores that are seen."""
    scores = torch.where(seen, scores, torch.full((), -math.inf, device=scores.device))
    e = torch.exp(scores - scores.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_decode(case, s):
    n, hq, d = s["q"].shape
    hkv = case["hkv"]
    lens = s["lens"].long()[:, None]
    pos = torch.arange(s["most_keys"], device=lens.device)[None, :].expand(n, -1)
    q = s["q"].float().view(n, hkv, hq // hkv, d)
    p = _weights(torch.einsum("bhgd,bnhd->bhgn", q, _gathered(s, 0, pos)) * s["scale"], (pos < lens)[:, None, None, :])
    s["out"].copy_(torch.einsum("bhgn,bnhd->bhgd", p, _gathered(s, 1, pos)).reshape(n, hq, d))
    return s["out"]


def _plain_prefill(case, s):
    tokens, hq, d = s["q"].shape
    hkv, n, device = case["hkv"], case["seqs"], s["q"].device
    start, lens = s["query_start"].long(), s["lens"].long()
    chunk = start[1:] - start[:-1]
    row = torch.arange(s["most_rows"], device=device)[None, :]
    q = s["q"][(start[:-1, None] + row).clamp(max=tokens - 1)].float()  # [seqs, rows, hq, d]
    q = q.view(n, s["most_rows"], hkv, hq // hkv, d)
    pos = torch.arange(s["most_keys"], device=device)[None, :].expand(n, -1)
    at = (lens - chunk)[:, None] + row  # the rows' positions
    seen = pos[:, None, :] <= at[:, :, None]
    p = _weights(torch.einsum("brhgd,bnhd->bhgrn", q, _gathered(s, 0, pos)) * s["scale"], seen[:, None, None])
    o = torch.einsum("bhgrn,bnhd->brhgd", p, _gathered(s, 1, pos)).reshape(n, s["most_rows"], hq, d)
    token = torch.arange(tokens, device=device)
    seq = torch.searchsorted(start[1:].contiguous(), token, right=True)
    s["out"].copy_(o[seq, token - start[seq]])
    return s["out"]


# ----------------------------------------------------------------------------
# The definition in 64 bits: a row's exponent by comparison with powers of two, its codes as multiples of their
# spacing, a token's rotation as a complex product, attention a sequence and kv head at a time
# ----------------------------------------------------------------------------
def _exact_rows(x):
    """Codes' values and exponent bytes of rows x [..., D] in 64 bits."""
    limits = 448.0 * torch.exp2(torch.arange(-127, 128, device=x.device, dtype=torch.float64))
    e = torch.bucketize(x.abs().amax(-1), limits)  # the first limit that is not below the largest
    y = x / torch.exp2(e.double() - 127)[..., None]
    spacing = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / spacing) * spacing, e


def _exact_value(s, i, blocks, heads, offsets):
    e = s["kv_scales"][blocks, heads, i, offsets].double() - 127
    codes = s["v_cache" if i else "k_cache"].view(torch.uint8)[blocks, heads, offsets].view(FP8)
    return codes.double() * torch.exp2(e)[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append_fp8":
        return _exact_append(case, s)
    if case["op"] == "gather_fp8":
        at, heads = s["slots"][:case["tokens"], None], torch.arange(case["hkv"], device=DEVICE)[None]
        rows = [_exact_value(s, i, at // BLOCK, heads, at % BLOCK) for i in (0, 1)]
        return tuple(torch.cat([r, s["k"][case["tokens"]:].double()]) for r in rows)
    if case["op"] == "copy_fp8":
        of = torch.arange(s["kv_scales"].shape[0], device=DEVICE)
        of[s["src_dst"][:, 1]] = s["src_dst"][:, 0]
        return s["k_cache"].double()[of], s["v_cache"].double()[of], s["kv_scales"][of]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lens = s["lens"].tolist()
    starts = s["query_start"].tolist() if "query_start" in s else list(range(len(lens) + 1))
    group = case["hq"] // case["hkv"]
    for b, n in enumerate(lens):
        rows = slice(starts[b], starts[b + 1])
        p = torch.arange(n - (rows.stop - rows.start), n, device=DEVICE)
        keys = torch.arange(n, device=DEVICE)
        blocks = s["table"][b, keys // BLOCK].long()
        for h in range(case["hkv"]):
            k, v = (_exact_value(s, i, blocks, h, keys % BLOCK) for i in (0, 1))
            q = s["q"][rows, h * group:(h + 1) * group].double()
            scores = torch.matmul(q.transpose(0, 1), k.T) * s["scale"]  # [group, rows, keys]
            scores = scores.masked_fill((keys[None] > p[:, None])[None], -math.inf)
            out[rows, h * group:(h + 1) * group] = torch.matmul(torch.softmax(scores, -1), v).transpose(0, 1)
    return out


def _exact_append(case, s):
    n, d = case["tokens"], case["d"]
    k, outputs = s["k"][:n].double(), ()
    if case["rotary"]:
        at = s["cos_sin"][s["positions"][:n]].double()
        turn = torch.complex(at[:, :d // 2], at[:, d // 2:])[:, None]

        def turned(x):
            z = torch.complex(x[:n, :, :d // 2].double(), x[:n, :, d // 2:].double()) * turn
            return torch.cat([z.real, z.imag], 2)

        q_out = s["q_out"].double()
        q_out[:n] = turned(s["q"])
        k, outputs = turned(s["k"]).to(torch.bfloat16).double(), (q_out,)  # a rotated key is a bf16 value, then quantised
    block, offset = s["slots"][:n] // BLOCK, s["slots"][:n] % BLOCK
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    scales = s["kv_scales"].clone()
    for i, x in enumerate((k, s["v"][:n].double())):
        caches[i][block, :, offset], e = _exact_rows(x)
        scales[block, :, i, offset] = e.to(torch.uint8)
    return *outputs, *caches, scales
