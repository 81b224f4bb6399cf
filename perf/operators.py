"""Measured cases of the paged cache's rotary append, windowed attention and shared-prefix decode attention.

Four operators, each in a plain form of elementary torch operations in 32 bits (``own = False``) and as the
framework's own calls (``own = True``):

    rope_append      rotate q and k at their tokens' positions (one or several position axes), q to its own
                     buffer, k and v into the paged cache
    window_decode    one query token a sequence over the last ``window`` cached tokens and the first ``sinks``
    window_prefill   chunks of query tokens, causal, each row over the last ``window`` tokens and the first ``sinks``
    prefix_decode    one query token a sequence; groups of sequences share the blocks of a long prefix

Sequences, lengths and block tables are drawn so that a case's amount of work is fixed by the case: the lengths
of a batch are spread evenly over their range and only their order, the block ids and the values go by the seed.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
DEVICE = "cuda"


# ----------------------------------------------------------------------------
# The cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # The attention input of one decode step of a small model: eight sequences, latency alone.
        dict(name="rope_append decode 8", op="rope_append", tokens=8, pad=0, hq=16, hkv=8, d=128, axes=1,
             packed=True, max_position=32768),
        # Eight prompt chunks of 512 tokens of one layer, q, k and v as views of the fused projection.
        dict(name="rope_append chunks 4096", op="rope_append", tokens=4096, pad=0, hq=32, hkv=8, d=128, axes=1,
             packed=True, max_position=32768),
        # Prompts with images: time, height and width positions, a padded batch, separate q, k and v.
        dict(name="rope_append images 32773", op="rope_append", tokens=32773, pad=27, hq=32, hkv=8, d=128, axes=3,
             packed=False, max_position=32768),
        # A single chat sequence with a short window: latency alone.
        dict(name="window_decode 1", op="window_decode", seqs=1, len_lo=4097, len_hi=4097, hq=16, hkv=8, d=128,
             window=1024, sinks=4),
        # A serving batch of one layer; some sequences are shorter than the window.
        dict(name="window_decode 128", op="window_decode", seqs=128, len_lo=512, len_hi=16384, hq=32, hkv=8, d=128,
             window=2048, sinks=4),
        # Streams that ran far past their window, eight q heads to a kv head, small heads, an odd window.
        dict(name="window_decode 61 long", op="window_decode", seqs=61, len_lo=16, len_hi=65536, hq=64, hkv=8, d=64,
             window=4095, sinks=33),
        # One chunk of a single long sequence: too few tiles to fill the GPU.
        dict(name="window_prefill 1x512", op="window_prefill", seqs=1, chunk_lo=512, chunk_hi=512, past_lo=8192,
             past_hi=8192, hq=16, hkv=8, d=128, window=1024, sinks=4),
        # Ragged chunks of a serving batch after up to 3584 cached tokens.
        dict(name="window_prefill 8 ragged", op="window_prefill", seqs=8, chunk_lo=33, chunk_hi=1001, past_lo=0,
             past_hi=3584, hq=32, hkv=8, d=128, window=1024, sinks=4),
        # Whole long prompts, no tokens cached, a wide window and no sinks.
        dict(name="window_prefill 2x8192", op="window_prefill", seqs=2, chunk_lo=8192, chunk_hi=8192, past_lo=0,
             past_hi=0, hq=32, hkv=8, d=128, window=4096, sinks=0),
        # A few samples of one prompt: latency alone.
        dict(name="prefix_decode 4", op="prefix_decode", seqs=4, groups=1, prefix_lo=1024, prefix_hi=1024, tail_lo=1,
             tail_hi=64, hq=16, hkv=8, d=128),
        # A serving batch behind one long system prompt.
        dict(name="prefix_decode 128", op="prefix_decode", seqs=128, groups=1, prefix_lo=8192, prefix_hi=8192,
             tail_lo=16, tail_hi=1024, hq=32, hkv=8, d=128),
        # Several prompts of different lengths, each with its own samples, eight q heads to a kv head.
        dict(name="prefix_decode 150 in 5", op="prefix_decode", seqs=150, groups=5, prefix_lo=1000, prefix_hi=16384,
             tail_lo=1, tail_hi=777, hq=64, hkv=8, d=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hkv = rng.choice([1, 2, 3, 4, 8])
    heads = dict(hq=hkv * rng.choice([1, 2, 4, 8]), hkv=hkv, d=rng.choice([64, 128]))
    op = rng.choice(["rope_append", "window_decode", "window_prefill", "prefix_decode"])
    if op == "rope_append":
        return dict(op=op, tokens=_log_int(rng, 1, 32768), pad=rng.choice([0, 0, 1, 5]), **heads,
                    axes=rng.choice([1, 1, 2, 3]), packed=rng.random() < 0.5, max_position=32768)
    if op == "window_decode":
        lens = sorted(_log_int(rng, 1, 32768) for _ in range(2))
        return dict(op=op, seqs=_log_int(rng, 1, 128), len_lo=lens[0], len_hi=lens[1], **heads,
                    window=_log_int(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 16, 61]))
    if op == "window_prefill":
        chunk = sorted(_log_int(rng, 1, 2048) for _ in range(2))
        past = sorted(rng.randint(0, 4096) for _ in range(2))
        return dict(op=op, seqs=rng.randint(1, 8), chunk_lo=chunk[0], chunk_hi=chunk[1], past_lo=past[0],
                    past_hi=past[1], **heads, window=_log_int(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 16, 61]))
    seqs = _log_int(rng, 1, 128)
    prefix = sorted(_log_int(rng, 16, 16384) for _ in range(2))
    tail = sorted(_log_int(rng, 1, 1024) for _ in range(2))
    return dict(op=op, seqs=seqs, groups=rng.randint(1, min(seqs, 6)), prefix_lo=prefix[0], prefix_hi=prefix[1],
                tail_lo=tail[0], tail_hi=tail[1], **heads)


# ----------------------------------------------------------------------------
# Sizes that a case fixes
# ----------------------------------------------------------------------------
def _even(lo, hi, n):
    """n lengths spread evenly over [lo, hi] (over their logarithm where it spans more than a factor of ten)."""
    if lo > 0 and hi > 10 * lo:
        return np.rint(np.exp(np.linspace(math.log(lo), math.log(hi), n))).astype(np.int64)
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64)


def _groups(case):
    """Row bounds and prefix lengths of prefix_decode's groups."""
    bounds = np.rint(np.linspace(0, case["seqs"], case["groups"] + 1)).astype(np.int64)
    return bounds, _even(case["prefix_lo"], case["prefix_hi"], case["groups"])


def _seen(lo, hi, window, sinks):
    """Tokens seen by the query rows at positions lo .. hi - 1, summed over the rows."""
    p = np.arange(lo, hi)
    return int((np.minimum(p + 1, window) + np.minimum(sinks, np.maximum(0, p + 1 - window))).sum())


def work(case):
    hq, hkv, d, op = case["hq"], case["hkv"], case["d"], case["op"]
    kv_token = 4 * hkv * d  # bytes of one token's K and V
    qo_row = 4 * hq * d     # bytes of one token's q and its output
    if op == "rope_append":
        n, axes = case["tokens"], case["axes"]
        # q read and written, k and v read and written to the cache; positions, slots and the rotation's angles.
        return dict(bytes=n * (qo_row + 2 * kv_token + 8 * axes + 8 + 4 * d), flops=3 * n * (hq + hkv) * d)
    if op == "window_decode":
        seen = [_seen(n - 1, n, case["window"], case["sinks"])
                for n in _even(case["len_lo"], case["len_hi"], case["seqs"])]
        return dict(bytes=sum(seen) * kv_token + case["seqs"] * (qo_row + 4) + sum(seen) // BLOCK * 4,
                    flops=4 * sum(seen) * hq * d)
    if op == "window_prefill":
        past = _even(case["past_lo"], case["past_hi"], case["seqs"])
        chunk = _even(case["chunk_lo"], case["chunk_hi"], case["seqs"])
        rows = [_seen(p, p + c, case["window"], case["sinks"]) for p, c in zip(past, chunk)]
        # Tokens that any row of the chunk sees: from the first row's window on, and the sinks before it.
        first = np.maximum(0, past + 1 - case["window"])
        union = int((past + chunk - first + np.minimum(first, case["sinks"])).sum())
        return dict(bytes=union * kv_token + int(chunk.sum()) * qo_row, flops=4 * sum(rows) * hq * d)
    bounds, prefix = _groups(case)
    tail = _even(case["tail_lo"], case["tail_hi"], case["seqs"])
    rows = np.diff(bounds)
    total = int((rows * prefix).sum() + tail.sum())
    return dict(bytes=int(prefix.sum() + tail.sum()) * kv_token + case["seqs"] * (qo_row + 4), flops=4 * total * hq * d)


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32).to(torch.bfloat16)


def _caches(gen, blocks, hkv, d):
    return _normal(gen, blocks, hkv, BLOCK, d), _normal(gen, blocks, hkv, BLOCK, d)


def _tables(gen, lens, pool, width):
    """Block tables [seqs, width] of distinct blocks in random order, -1 behind each sequence's last block."""
    counts = torch.as_tensor(-(-lens // BLOCK), device=DEVICE)
    starts = torch.cumsum(counts, 0) - counts
    order = torch.randperm(pool, generator=gen, device=DEVICE)
    col = torch.arange(width, device=DEVICE)
    inside = col[None, :] < counts[:, None]
    flat = torch.where(inside, starts[:, None] + col[None, :], torch.zeros((), dtype=torch.long, device=DEVICE))
    return torch.where(inside, order[flat], torch.full((), -1, dtype=torch.long, device=DEVICE)).to(torch.int32)


def _int32(values):
    return torch.as_tensor(np.asarray(values), device=DEVICE).to(torch.int32)


def _freq_axes(case):
    """The position axis of each rotation frequency: in order, about a quarter of them time, the rest split."""
    half, axes = case["d"] // 2, case["axes"]
    if axes == 1:
        return None
    first = half // (axes + 1)
    rest = np.rint(np.linspace(first, half, axes)).astype(np.int64)
    return bytes(np.searchsorted(rest, np.arange(half), side="right").astype(np.uint8))


def _rope_state(case, gen, rng):
    n, hq, hkv, d, axes = case["tokens"], case["hq"], case["hkv"], case["d"], case["axes"]
    total = n + case["pad"]
    if case["packed"]:
        rows = _normal(gen, total, hq + 2 * hkv, d)
        q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    else:
        q, k, v = _normal(gen, total, hq, d), _normal(gen, total, hkv, d), _normal(gen, total, hkv, d)
    # Chunks of up to 512 consecutive tokens, each from a random position on; with several axes a chunk is
    # a picture of 32 columns: the time of its start, then its rows and columns.
    chunk = torch.arange(total, device=DEVICE) // 512
    within = torch.arange(total, device=DEVICE) % 512
    start = torch.randint(0, case["max_position"] - 512, (total // 512 + 1,), generator=gen, device=DEVICE)[chunk]
    by_axis = [start + within] if axes == 1 else [start, start + within // 32, start + within % 32][:axes]
    positions = torch.stack(by_axis) if axes > 1 else by_axis[0]
    blocks = -(-total // BLOCK) + 8
    slots = torch.randperm(blocks, generator=gen, device=DEVICE)[torch.arange(total, device=DEVICE) // BLOCK]
    slots = slots * BLOCK + torch.arange(total, device=DEVICE) % BLOCK
    slots[n:] = -1
    inverse = 5e5 ** (-torch.arange(d // 2, device=DEVICE, dtype=torch.float64) / (d // 2))
    angle = torch.arange(case["max_position"], device=DEVICE, dtype=torch.float64)[:, None] * inverse
    k_cache, v_cache = _caches(gen, blocks, hkv, d)
    return dict(q=q, k=k, v=v, positions=positions.contiguous(), slots=slots, k_cache=k_cache, v_cache=v_cache,
                cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(), freq_axes=_freq_axes(case),
                q_out=torch.zeros(total, hq, d, dtype=torch.bfloat16, device=DEVICE))


def _window_decode_state(case, gen, rng):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lens = rng.permutation(_even(case["len_lo"], case["len_hi"], case["seqs"]))
    width = -(-int(lens.max()) // BLOCK)
    # Blocks that the window has left behind are back in the pool: the pool holds what is seen, and their
    # table entries are -1.
    sinks_end = -(-np.minimum(case["sinks"], lens) // BLOCK)
    first = np.maximum(np.maximum(0, lens - case["window"]) // BLOCK, sinks_end)
    held = sinks_end + np.maximum(0, -(-lens // BLOCK) - first)
    packed = _tables(gen, held * BLOCK, int(held.sum()) + 4, int(held.max()))
    col = torch.arange(width, device=DEVICE)[None, :]
    low, high = (torch.as_tensor(x, device=DEVICE)[:, None] for x in (sinks_end, first))
    at = torch.where(col < low, col, col - high + low).clamp(0, packed.shape[1] - 1)
    keep = (col < low) | ((col >= high) & (col < torch.as_tensor(-(-lens // BLOCK), device=DEVICE)[:, None]))
    table = torch.where(keep, packed.gather(1, at), torch.full_like(at, -1, dtype=torch.int32))
    k_cache, v_cache = _caches(gen, int(held.sum()) + 4, hkv, d)
    q = _normal(gen, case["seqs"], hq, d)
    return dict(q=q, k_cache=k_cache, v_cache=v_cache, table=table.contiguous(), lens=_int32(lens),
                out=torch.empty_like(q), scale=d ** -0.5)


def _window_prefill_state(case, gen, rng):
    hq, hkv, d, n = case["hq"], case["hkv"], case["d"], case["seqs"]
    order = rng.permutation(n)
    past = _even(case["past_lo"], case["past_hi"], n)[order]
    chunk = _even(case["chunk_lo"], case["chunk_hi"], n)[order]
    lens = past + chunk
    pool = int((-(-lens // BLOCK)).sum()) + 4
    k_cache, v_cache = _caches(gen, pool, hkv, d)
    q = _normal(gen, int(chunk.sum()), hq, d)
    return dict(q=q, k_cache=k_cache, v_cache=v_cache, table=_tables(gen, lens, pool, -(-int(lens.max()) // BLOCK)),
                lens=_int32(lens), query_start=_int32(np.concatenate([[0], np.cumsum(chunk)])),
                most_rows=int(chunk.max()), most_keys=int(lens.max()), out=torch.empty_like(q), scale=d ** -0.5)


def _prefix_decode_state(case, gen, rng):
    hq, hkv, d, n = case["hq"], case["hkv"], case["d"], case["seqs"]
    bounds, prefix = _groups(case)
    group = np.repeat(np.arange(case["groups"]), np.diff(bounds))
    lens = prefix[group] + rng.permutation(_even(case["tail_lo"], case["tail_hi"], n))
    # A group's whole prefix blocks are the same in every one of its tables; a sequence's own blocks follow.
    shared = prefix // BLOCK
    mine = -(-lens // BLOCK) - shared[group]
    width = int((-(-lens // BLOCK)).max())
    pool = int(shared.sum() + mine.sum()) + 4
    order = torch.randperm(pool, generator=gen, device=DEVICE)
    col = torch.arange(width, device=DEVICE)[None, :]
    as_column = lambda x: torch.as_tensor(x, device=DEVICE)[:, None]  # noqa: E731
    shared_at = as_column((np.cumsum(shared) - shared)[group])
    mine_at = as_column(int(shared.sum()) + np.cumsum(mine) - mine)
    count = as_column(shared[group])
    flat = torch.where(col < count, shared_at + col, mine_at + col - count)
    held = col < as_column(-(-lens // BLOCK))
    table = torch.where(held, order[torch.where(held, flat, torch.zeros_like(flat))], torch.full_like(flat, -1))
    k_cache, v_cache = _caches(gen, pool, hkv, d)
    q = _normal(gen, n, hq, d)
    return dict(q=q, k_cache=k_cache, v_cache=v_cache, table=table.to(torch.int32).contiguous(), lens=_int32(lens),
                group_start=_int32(bounds), prefix_lens=_int32(prefix), most_keys=int(lens.max()),
                out=torch.empty_like(q), scale=d ** -0.5)


_STATES = dict(rope_append=_rope_state, window_decode=_window_decode_state, window_prefill=_window_prefill_state,
               prefix_decode=_prefix_decode_state)


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

    if op == "rope_append":
        pkv.rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos_sin"], s["k_cache"], s["v_cache"],
                        s["q_out"], freq_axes=s["freq_axes"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "window_decode":
        return pkv.paged_window_decode_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["scale"],
                                                 s["out"], case["window"], case["sinks"])
    if op == "window_prefill":
        return pkv.paged_window_prefill_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                                  s["query_start"], s["most_rows"], s["scale"], s["out"],
                                                  case["window"], case["sinks"])
    return pkv.paged_prefix_decode_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                             s["group_start"], s["prefix_lens"], s["scale"], s["out"])


def _run_plain(op, case, s):
    return dict(rope_append=_plain_rope_append, window_decode=_plain_window_decode,
                window_prefill=_plain_window_prefill, prefix_decode=_plain_prefix_decode)[op](case, s)


def _plain_rope_append(case, s):
    n, d = case["tokens"], case["d"]
    positions = s["positions"][..., :n]
    if case["axes"] == 1:
        table = s["cos_sin"][positions]
        cos, sin = table[:, None, :d // 2], table[:, None, d // 2:]
    else:
        axis = torch.tensor(list(s["freq_axes"]), device=positions.device)
        at, freq = positions[axis].T, torch.arange(d // 2, device=positions.device)
        cos, sin = s["cos_sin"][at, freq][:, None], s["cos_sin"][at, d // 2 + freq][:, None]

    def turned(x):
        a, b = x[:n, :, :d // 2].float(), x[:n, :, d // 2:].float()
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)

    slots = s["slots"][:n]
    s["q_out"][:n] = turned(s["q"])
    s["k_cache"][slots // BLOCK, :, slots % BLOCK] = turned(s["k"])
    s["v_cache"][slots // BLOCK, :, slots % BLOCK] = s["v"][:n]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _gathered(cache, table, pos):
    """Cache rows [seqs, n, kv heads, d] of the positions [seqs, n], in 32 bits."""
    block = table.gather(1, (pos // BLOCK).clamp(0, table.shape[1] - 1)).clamp(min=0).long()
    return cache[block, :, pos % BLOCK].float()


def _weights(scores, seen):
    """Softmax over the last axis of the scores that are seen; a row that sees nothing has no weights."""
    scores = torch.where(seen, scores, torch.full((), -math.inf, device=scores.device))
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total))


def _plain_decode(s, pos, seen):
    n, hq, d = s["q"].shape
    hkv = s["k_cache"].shape[1]
    q = s["q"].float().view(n, hkv, hq // hkv, d)
    k = _gathered(s["k_cache"], s["table"], pos)
    p = _weights(torch.einsum("bhgd,bnhd->bhgn", q, k) * s["scale"], seen[:, None, None, :])
    o = torch.einsum("bhgn,bnhd->bhgd", p, _gathered(s["v_cache"], s["table"], pos))
    s["out"].copy_(o.reshape(n, hq, d))
    return s["out"]


def _plain_window_decode(case, s):
    lens = s["lens"].long()[:, None]
    first = torch.arange(case["sinks"], device=lens.device)[None, :].expand(lens.shape[0], -1)
    last = lens - case["window"] + torch.arange(case["window"], device=lens.device)[None, :]
    pos = torch.cat([first, last], 1)
    seen = torch.cat([first < lens, last >= case["sinks"]], 1)
    return _plain_decode(s, pos.clamp(min=0), seen)


def _plain_prefix_decode(case, s):
    lens = s["lens"].long()[:, None]
    pos = torch.arange(s["most_keys"], device=lens.device)[None, :].expand(lens.shape[0], -1)
    return _plain_decode(s, pos, pos < lens)


def _plain_window_prefill(case, s):
    tokens, hq, d = s["q"].shape
    hkv, n = s["k_cache"].shape[1], s["lens"].shape[0]
    device = s["q"].device
    start, lens = s["query_start"].long(), s["lens"].long()
    chunk = start[1:] - start[:-1]
    row = torch.arange(s["most_rows"], device=device)[None, :]
    q = s["q"][(start[:-1, None] + row).clamp(max=tokens - 1)].float()  # [seqs, rows, hq, d]
    q = q.view(n, s["most_rows"], hkv, hq // hkv, d)
    pos = torch.arange(s["most_keys"], device=device)[None, :].expand(n, -1)
    at = (lens - chunk)[:, None] + row                                  # the rows' positions
    seen = (pos[:, None, :] <= at[:, :, None]) & ((pos[:, None, :] > at[:, :, None] - case["window"])
                                                  | (pos[:, None, :] < case["sinks"]))
    k = _gathered(s["k_cache"], s["table"], pos)
    p = _weights(torch.einsum("brhgd,bnhd->bhgrn", q, k) * s["scale"], seen[:, None, None])
    o = torch.einsum("bhgrn,bnhd->brhgd", p, _gathered(s["v_cache"], s["table"], pos))
    o = o.reshape(n, s["most_rows"], hq, d)
    token = torch.arange(tokens, device=device)
    seq = torch.searchsorted(start[1:].contiguous(), token, right=True)
    s["out"].copy_(o[seq, token - start[seq]])
    return s["out"]


# ----------------------------------------------------------------------------
# The definition in 64 bits, a sequence (or a token's rotation as a complex product) at a time
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope_append":
        return _exact_rope_append(case, s)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lens = s["lens"].tolist()
    starts = s["query_start"].tolist() if "query_start" in s else list(range(len(lens) + 1))
    window, sinks = case.get("window", 1 << 40), case.get("sinks", 0)
    group = case["hq"] // case["hkv"]
    for b, n in enumerate(lens):
        rows = slice(starts[b], starts[b + 1])
        p = torch.arange(n - (rows.stop - rows.start), n, device=DEVICE)
        keys = torch.arange(n, device=DEVICE)
        keys = keys[(keys < sinks) | (keys > n - (rows.stop - rows.start) - window)]  # what any row sees
        blocks = s["table"][b, keys // BLOCK].long()
        hidden = (keys[None] > p[:, None]) | ((keys[None] <= p[:, None] - window) & (keys[None] >= sinks))
        for h in range(case["hkv"]):
            k, v = (s[c][blocks, h, keys % BLOCK].double() for c in ("k_cache", "v_cache"))
            q = s["q"][rows, h * group:(h + 1) * group].double()
            scores = torch.matmul(q.transpose(0, 1), k.T) * s["scale"]  # [group, rows, keys]
            scores = scores.masked_fill(hidden[None], -math.inf)
            out[rows, h * group:(h + 1) * group] = torch.matmul(torch.softmax(scores, -1), v).transpose(0, 1)
    return out


def _exact_rope_append(case, s):
    n, d = case["tokens"], case["d"]
    axis = torch.tensor(list(s["freq_axes"] or bytes(d // 2)), device=DEVICE)
    positions = s["positions"].reshape(case["axes"], -1)[:, :n]
    freq = torch.arange(d // 2, device=DEVICE)
    at = positions[axis].transpose(0, 1)
    turn = torch.complex(s["cos_sin"][at, freq].double(), s["cos_sin"][at, freq + d // 2].double())

    def turned(x):
        z = torch.complex(x[:n, :, :d // 2].double(), x[:n, :, d // 2:].double()) * turn[:, None, :]
        return torch.cat([z.real, z.imag], 2)

    q_out, k_cache, v_cache = (s[x].double() for x in ("q_out", "k_cache", "v_cache"))
    q_out[:n] = turned(s["q"])
    block, offset = s["slots"][:n] // BLOCK, s["slots"][:n] % BLOCK
    k_cache[block, :, offset] = turned(s["k"])
    v_cache[block, :, offset] = s["v"][:n].double()
    return q_out, k_cache, v_cache
