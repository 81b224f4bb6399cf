"""Refusals of the rotary append, the windowed and the shared-prefix attention, on the CPU: host-checkable errors
return before any CUDA call (pointers are fake, nothing is dereferenced)."""
import ctypes

import pytest

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_275_gb300 import build
    build.build(quiet=True)
    from paged_kv_cache_275_gb300 import _capi
    return _capi.load()


def msg(lib) -> str:
    return lib.pkv_last_error_message().decode()


def rope(lib, **kw):
    a = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, pos=FAKE, axes=1, axs=0, fa=None, cs=FAKE, mp=100,
             slots=FAKE, n=4, hq=32, hkv=8, d=128, qo=FAKE, qos=4096, kc=FAKE, vc=FAKE, nb=10, bs=16, stream=None)
    assert set(kw) <= set(a)
    return lib.pkv_rope_append(*{**a, **kw}.values())


@pytest.mark.parametrize("kw,status,says", [
    (dict(n=-1), 1, "num_tokens"), (dict(n=(1 << 32) + 1), 2, "num_tokens"),
    (dict(hq=0), 1, "head counts"), (dict(hkv=0), 1, "head counts"), (dict(d=96), 2, "head_dim"),
    (dict(bs=32), 2, "block_size"), (dict(nb=0), 1, "num_blocks"), (dict(mp=0), 1, "max_position"),
    (dict(axes=0), 1, "num_axes"), (dict(axes=5), 1, "num_axes"), (dict(axes=2), 1, "freq_axes is null"),
    (dict(axes=2, axs=-8, fa=bytes(64)), 1, "axis_stride"), (dict(axes=2, fa=bytes([0] * 63 + [2])), 1, "freq_axes[63] = 2"),
    (dict(qs=4097), 1, "q_stride"), (dict(ks=-8), 1, "k_stride"), (dict(vs=1020), 1, "v_stride"),
    (dict(qos=4088), 1, "q_out_stride"), (dict(q=None), 1, "null"), (dict(qo=None), 1, "null"), (dict(cs=None), 1, "null"),
    (dict(k=FAKE + 8), 1, "aligned"), (dict(pos=FAKE + 4), 1, "aligned"), (dict(slots=FAKE + 4), 1, "aligned"),
])
def test_rope_append_refuses(lib, kw, status, says):
    assert rope(lib, **kw) == status and says in msg(lib)


def test_rope_append_zero_tokens_is_a_noop(lib):
    assert rope(lib, n=0, q=None, kc=None) == 0 and msg(lib) == ""


def window_decode(lib, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, W=8, cl=FAKE, B=4, hq=32, hkv=8, d=128, nb=100, bs=16, scale=0.088,
             window=64, sinks=4, out=FAKE, ws=FAKE, wsb=16, parts=64, stream=None)
    assert set(kw) <= set(a)
    return lib.pkv_paged_window_decode_attention(*{**a, **kw}.values())


@pytest.mark.parametrize("kw,status,says", [
    (dict(window=0), 1, "window"), (dict(window=-1), 1, "window"), (dict(sinks=-1), 1, "num_sink_tokens"),
    (dict(hq=30), 1, "multiple"), (dict(hq=24, hkv=2), 2, "group"), (dict(d=256), 2, "head_dim"), (dict(bs=8), 2, "block_size"),
    (dict(B=-1), 1, "num_seqs"), (dict(W=0), 1, "max_blocks"), (dict(nb=0), 1, "num_blocks"),
    (dict(scale=float("nan")), 1, "scale"), (dict(parts=-1), 1, "num_partitions"), (dict(out=None), 1, "null"),
    (dict(nb=1 << 24), 2, "2^31"),
    (dict(q=FAKE + 2), 1, "aligned"), (dict(), 1, "workspace too small"), (dict(B=5000), 1, "workspace too small"),
])
def test_window_decode_refuses(lib, kw, status, says):
    assert window_decode(lib, **kw) == status and says in msg(lib)


def test_window_decode_zero_sequences_is_a_noop(lib):
    assert window_decode(lib, B=0, q=None) == 0


def test_window_decode_workspace_size(lib):
    n = ctypes.c_size_t(0)
    size = lib.pkv_window_decode_workspace_size
    assert size(128, 32, 8, 128, 256, 100, 4, 1000, ctypes.byref(n)) == 0
    # The block prefix, the pairs' records and two states per piece, as for a whole-sequence call.
    header = ((128 + 1) * 4 + 255) // 256 * 256 + (128 * 8 * 8 + 255) // 256 * 256
    assert n.value == header + 1000 * 2 * (4 * 128 + 8) * 4
    assert size(128, 32, 8, 128, 256, 0, 4, 1000, ctypes.byref(n)) == 1
    assert size(128, 32, 8, 128, 256, 100, -1, 1000, ctypes.byref(n)) == 1
    assert size(128, 32, 8, 128, 256, 100, 4, 1000, None) == 1


def window_prefill(lib, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, W=8, cl=FAKE, qs=FAKE, T=2048, mql=512, B=4, hq=32, hkv=8, d=128, nb=100,
             bs=16, scale=0.088, window=64, sinks=4, out=FAKE, S=1, ws=None, wsb=0, stream=None)
    assert set(kw) <= set(a)
    return lib.pkv_paged_window_prefill_attention(*{**a, **kw}.values())


@pytest.mark.parametrize("kw,status,says", [
    (dict(window=0), 1, "window"), (dict(sinks=-1), 1, "num_sink_tokens"), (dict(scale=0.0), 1, "scale"),
    (dict(scale=-1.0), 1, "scale"), (dict(scale=float("inf")), 1, "scale"), (dict(scale=float("nan")), 1, "scale"),
    (dict(B=65536), 2, "65535"), (dict(mql=65535 * 64 + 1), 2, "max_query_len"), (dict(mql=-1), 1, "max_query_len"),
    (dict(S=0), 1, "num_splits"), (dict(S=33), 1, "num_splits"), (dict(S=2), 1, "workspace too small"),
    (dict(S=2, ws=FAKE, wsb=16), 1, "workspace too small"), (dict(S=2, ws=FAKE + 8, wsb=1 << 40), 1, "aligned"),
    (dict(q=None), 1, "null"), (dict(d=32), 2, "head_dim"), (dict(hq=48, hkv=3), 2, "group"), (dict(T=-1), 1, "num_query_tokens"),
])
def test_window_prefill_refuses(lib, kw, status, says):
    assert window_prefill(lib, **kw) == status and says in msg(lib)


def test_window_prefill_without_rows_is_a_noop(lib):
    assert window_prefill(lib, mql=0, q=None) == 0 and window_prefill(lib, B=0, q=None) == 0


def test_window_prefill_default_splits_checks_arguments_before_the_device(lib):
    n = ctypes.c_int32(0)
    splits = lib.pkv_window_prefill_default_splits
    assert splits(1, 512, 32, 8, 64, 4, None) == 1
    assert splits(1, 512, 32, 8, 0, 4, ctypes.byref(n)) == 1 and "window" in msg(lib)
    assert splits(-1, 512, 32, 8, 64, 4, ctypes.byref(n)) == 1


@pytest.mark.parametrize("window,sinks,want", [(1, 0, 1), (192, 0, 1), (193, 0, 2), (192, 1, 2), (1024, 0, 5), (1 << 30, 0, 32)])
def test_window_prefill_default_splits(lib, window, sinks, want):
    """Two steps of 128 keys each for the window, the sinks and the 64 tokens of a tile pair."""
    n = ctypes.c_int32(0)
    assert lib.pkv_window_prefill_default_splits(1, 512, 32, 8, window, sinks, ctypes.byref(n)) == 0 and n.value == want
    assert lib.pkv_window_prefill_default_splits(321, 512, 32, 8, window, sinks, ctypes.byref(n)) == 0 and n.value == 1


def test_window_prefill_workspace_size(lib):
    n = ctypes.c_size_t(0)
    size = lib.pkv_window_prefill_workspace_size
    assert size(128, 1, ctypes.byref(n)) == 0 and n.value == 0
    for d in (64, 128):
        for splits in (2, 32):
            assert size(d, splits, ctypes.byref(n)) == 0 and n.value == 160 * 256 * (d + 2) * 4 + 80 * 16 + 16
    assert size(96, 2, ctypes.byref(n)) == 2 and size(128, 0, ctypes.byref(n)) == 1 and size(128, 33, ctypes.byref(n)) == 1
    assert size(128, 2, None) == 1


def prefix_decode(lib, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, W=8, cl=FAKE, gs=FAKE, pl=FAKE, groups=2, B=4, hq=32, hkv=8, d=128,
             nb=100, bs=16, scale=0.088, out=FAKE, ws=FAKE, wsb=16, stream=None)
    assert set(kw) <= set(a)
    return lib.pkv_paged_prefix_decode_attention(*{**a, **kw}.values())


@pytest.mark.parametrize("kw,status,says", [
    (dict(B=-1), 1, "num_seqs"), (dict(B=4097), 2, "PKV_MAX_SEQS"), (dict(groups=-1), 1, "num_groups"),
    (dict(groups=4097), 1, "num_groups"), (dict(gs=None), 1, "null"), (dict(pl=None), 1, "null"), (dict(q=None), 1, "null"),
    (dict(gs=FAKE + 2), 1, "aligned"), (dict(out=FAKE + 8), 1, "aligned"), (dict(scale=0.0), 1, "scale"),
    (dict(scale=-0.1), 1, "scale"), (dict(scale=float("nan")), 1, "scale"), (dict(nb=0), 2, "num_blocks"),
    (dict(nb=1 << 24), 2, "2^31"), (dict(bs=32), 2, "block_size"), (dict(d=80), 2, "head_dim"), (dict(hq=20), 1, "multiple"),
    (dict(W=0), 1, "max_blocks"),
])
def test_prefix_decode_refuses(lib, kw, status, says):
    assert prefix_decode(lib, **kw) == status and says in msg(lib)


def test_prefix_decode_zero_sequences_is_a_noop(lib):
    assert prefix_decode(lib, B=0, q=None, gs=None) == 0


def test_binding_refuses_cpu_tensors():
    import torch
    import paged_kv_cache_275_gb300 as pkv
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    kc = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    table, lens, start = (torch.zeros(*s, dtype=torch.int32) for s in ((1, 1), (1,), (2,)))
    one = torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.rope_append(q, q[:, :1], q[:, :1], one, one, torch.zeros(4, 64), kc, kc, q.clone())
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_window_decode_attention(q, kc, kc, table, lens, 0.1, q.clone(), 16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_window_prefill_attention(q, kc, kc, table, lens, start, 1, 0.1, q.clone(), 16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_prefix_decode_attention(q, kc, kc, table, lens, start, lens, 0.1, q.clone())
    with pytest.raises(TypeError):
        pkv.paged_window_decode_attention(None, kc, kc, table, lens, 0.1, q, 16)


def test_freq_axes_of_sections():
    import paged_kv_cache_275_gb300 as pkv
    assert pkv.rope_freq_axes([2, 1, 3]) == bytes([0, 0, 1, 2, 2, 2])
