"""The 8-bit cache on the CPU: refusals of its calls (host-checkable errors return before any CUDA call; pointers are fake,
nothing is dereferenced), and the plain form of its format that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

from fp8_plain import CODES, FP8, quantise, values

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_275_gb300 import build
    build.build(quiet=True)
    from paged_kv_cache_275_gb300 import _capi
    return _capi.load()


def msg(lib) -> str:
    return lib.pkv_last_error_message().decode()


def call(function, defaults, kw):
    assert set(kw) <= set(defaults)
    return function(*{**defaults, **kw}.values())


def append(lib, **kw):
    return call(lib.pkv_kv_append_fp8, dict(k=FAKE, ks=1024, v=FAKE, vs=1024, slots=FAKE, n=4, hkv=8, d=128, kc=FAKE, vc=FAKE,
                                            sc=FAKE, nb=10, bs=16, stream=None), kw)


@pytest.mark.parametrize("kw,status,says", [
    (dict(n=-1), 1, "num_tokens"), (dict(n=(1 << 32) + 1), 2, "num_tokens"), (dict(hkv=0), 1, "num_kv_heads"),
    (dict(d=96), 2, "head_dim"), (dict(bs=32), 2, "block_size"), (dict(nb=0), 1, "num_blocks"), (dict(ks=1020), 1, "k_stride"),
    (dict(vs=-8), 1, "v_stride"), (dict(k=None), 1, "null"), (dict(sc=None), 1, "null"), (dict(v=FAKE + 8), 1, "aligned"),
    (dict(sc=FAKE + 8), 1, "aligned"), (dict(slots=FAKE + 4), 1, "aligned"),
])
def test_append_refuses(lib, kw, status, says):
    assert append(lib, **kw) == status and says in msg(lib)


def rope(lib, **kw):
    return call(lib.pkv_rope_append_fp8,
                dict(q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, pos=FAKE, axes=1, axs=0, fa=None, cs=FAKE, mp=100,
                     slots=FAKE, n=4, hq=32, hkv=8, d=128, qo=FAKE, qos=4096, kc=FAKE, vc=FAKE, sc=FAKE, nb=10, bs=16,
                     stream=None), kw)


@pytest.mark.parametrize("kw,status,says", [
    (dict(n=-1), 1, "num_tokens"), (dict(hq=0), 1, "num_q_heads"), (dict(hkv=0), 1, "num_kv_heads"), (dict(mp=0), 1, "max_position"),
    (dict(axes=0), 1, "num_axes"), (dict(axes=5), 1, "num_axes"), (dict(axes=2), 1, "freq_axes is null"),
    (dict(axes=2, axs=-8, fa=bytes(64)), 1, "axis_stride"), (dict(axes=2, fa=bytes([0] * 63 + [2])), 1, "freq_axes[63] = 2"),
    (dict(qs=4097), 1, "q_stride"), (dict(qos=4088), 1, "q_out_stride"), (dict(q=None), 1, "null"), (dict(cs=None), 1, "null"),
    (dict(sc=None), 1, "null"), (dict(pos=FAKE + 4), 1, "aligned"), (dict(kc=FAKE + 8), 1, "aligned"), (dict(d=80), 2, "head_dim"),
])
def test_rope_append_refuses(lib, kw, status, says):
    assert rope(lib, **kw) == status and says in msg(lib)


def gather(lib, **kw):
    return call(lib.pkv_kv_gather_fp8, dict(kc=FAKE, vc=FAKE, sc=FAKE, nb=10, bs=16, slots=FAKE, n=4, hkv=8, d=128, k=FAKE,
                                            ks=1024, v=FAKE, vs=1024, stream=None), kw)


@pytest.mark.parametrize("kw,status,says", [
    (dict(n=-1), 1, "num_tokens"), (dict(ks=1016), 1, "k_stride"), (dict(vs=1028), 1, "v_stride"), (dict(v=None), 1, "null"),
    (dict(k=FAKE + 2), 1, "aligned"), (dict(bs=8), 2, "block_size"), (dict(nb=-1), 1, "num_blocks"),
])
def test_gather_refuses(lib, kw, status, says):
    assert gather(lib, **kw) == status and says in msg(lib)


def copy(lib, **kw):
    return call(lib.pkv_copy_blocks_fp8, dict(kc=FAKE, vc=FAKE, sc=FAKE, sd=FAKE, n=3, hkv=8, d=128, nb=10, stream=None), kw)


@pytest.mark.parametrize("kw,status,says", [
    (dict(n=-1), 1, "num_pairs"), (dict(n=(1 << 30) + 1), 2, "num_pairs"), (dict(sd=None), 1, "null"), (dict(sc=FAKE + 4), 1, "aligned"),
    (dict(d=32), 2, "head_dim"), (dict(hkv=-1), 1, "num_kv_heads"),
])
def test_copy_refuses(lib, kw, status, says):
    assert copy(lib, **kw) == status and says in msg(lib)


def decode(lib, **kw):
    return call(lib.pkv_paged_fp8_decode_attention,
                dict(q=FAKE, kc=FAKE, vc=FAKE, sc=FAKE, bt=FAKE, W=8, cl=FAKE, B=4, hq=32, hkv=8, d=128, nb=100, bs=16,
                     scale=0.088, out=FAKE, ws=FAKE, wsb=1 << 40, stream=None), kw)


@pytest.mark.parametrize("kw,status,says", [
    (dict(hq=30), 1, "multiple"), (dict(hq=24), 2, "group"), (dict(d=256), 2, "head_dim"), (dict(bs=8), 2, "block_size"),
    (dict(B=-1), 1, "num_seqs"), (dict(B=65536), 2, "65535"), (dict(W=0), 1, "max_blocks"), (dict(nb=0), 2, "2^31"),
    (dict(nb=1 << 24), 2, "2^31"), (dict(scale=float("nan")), 1, "scale"), (dict(out=None), 1, "null"), (dict(sc=None), 1, "null"),
    (dict(q=FAKE + 2), 1, "aligned"), (dict(sc=FAKE + 2), 1, "aligned"), (dict(cl=FAKE + 2), 1, "aligned"),
    (dict(ws=FAKE + 8), 1, "aligned"),
])
def test_decode_refuses(lib, kw, status, says):
    assert decode(lib, **kw) == status and says in msg(lib)


def prefill(lib, **kw):
    return call(lib.pkv_paged_fp8_prefill_attention,
                dict(q=FAKE, kc=FAKE, vc=FAKE, sc=FAKE, bt=FAKE, W=8, cl=FAKE, qs=FAKE, T=2048, mql=512, B=4, hq=32, hkv=8,
                     d=128, nb=100, bs=16, scale=0.088, out=FAKE, ws=FAKE, wsb=1 << 40, stream=None), kw)


@pytest.mark.parametrize("kw,status,says", [
    (dict(scale=0.0), 1, "scale"), (dict(scale=-1.0), 1, "scale"), (dict(scale=float("inf")), 1, "scale"),
    (dict(scale=float("nan")), 1, "scale"), (dict(B=65536), 2, "65535"), (dict(mql=65535 * 64 + 1), 2, "max_query_len"),
    (dict(mql=-1), 1, "max_query_len"), (dict(T=-1), 1, "num_query_tokens"), (dict(q=None), 1, "null"), (dict(qs=None), 1, "null"),
    (dict(sc=None), 1, "null"), (dict(d=32), 2, "head_dim"), (dict(hq=48, hkv=3), 2, "group"), (dict(out=FAKE + 8), 1, "aligned"),
    (dict(nb=1 << 24), 2, "2^31"),
])
def test_prefill_refuses(lib, kw, status, says):
    assert prefill(lib, **kw) == status and says in msg(lib)


def test_calls_without_work_are_noops(lib):
    assert append(lib, n=0, k=None) == 0 and rope(lib, n=0, q=None) == 0 and gather(lib, n=0, k=None) == 0
    assert copy(lib, n=0, kc=None) == 0 and decode(lib, B=0, q=None) == 0
    assert prefill(lib, B=0, q=None) == 0 and prefill(lib, T=0, q=None) == 0 and prefill(lib, mql=0, q=None) == 0
    assert msg(lib) == ""


def test_workspace_queries_check_their_arguments(lib):
    n = ctypes.c_size_t(0)
    assert lib.pkv_fp8_decode_workspace_size(4, 32, 8, 128, 8, None) == 1
    assert lib.pkv_fp8_decode_workspace_size(4, 32, 8, 96, 8, ctypes.byref(n)) == 2
    assert lib.pkv_fp8_prefill_workspace_size(4, 1, 4, 32, 8, 128, 8, None) == 1
    assert lib.pkv_fp8_prefill_workspace_size(-1, 1, 4, 32, 8, 128, 8, ctypes.byref(n)) == 1
    assert lib.pkv_fp8_prefill_workspace_size(4, 1, 4, 30, 8, 128, 8, ctypes.byref(n)) == 1


def test_code_values_are_the_type_s():
    have = torch.arange(256, dtype=torch.uint8).view(FP8).double().numpy()
    assert np.array_equal(have, CODES, equal_nan=True)


def test_quantise_keeps_four_bits_and_the_largest_fits():
    x = torch.randn(400, 64, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16) * 2.0 ** torch.arange(-100, 100, 0.5)[:, None]
    x = x.to(torch.bfloat16)
    codes, e = quantise(x)
    got, want = codes * 2.0 ** (e[:, None] - 127.0), x.double().numpy()
    top = np.abs(want).max(-1)
    assert (top <= 448 * 2.0 ** (e - 127.0)).all() and (top > 448 * 2.0 ** (e - 128.0)).all()
    # Half a step is 2^-4 of the value, or of the least normal value.
    assert (np.abs(got - want) <= 2.0**-4 * np.maximum(np.abs(want), 2.0**-6 * 2.0 ** (e[:, None] - 127.0))).all()
    # Every value is one that bf16 has.
    assert np.array_equal(torch.from_numpy(got).to(torch.bfloat16).double().numpy(), got)


def test_quantise_at_the_borders():
    bf = lambda *x: torch.tensor([x], dtype=torch.float64).to(torch.bfloat16)  # noqa: E731
    assert quantise(bf(0.0, 0.0))[1][0] == 0
    assert quantise(bf(448.0, 1.0))[1][0] == 127 and quantise(bf(450.0, 1.0))[1][0] == 128
    codes, e = quantise(bf(float("inf"), 3.0, float("nan"), -float("inf")))
    assert e[0] == 127 - 7 and np.isnan(codes[0, [0, 2, 3]]).all() and codes[0, 1] == 384.0
    # Ties to even: halfway between 16 and 18, and between 18 and 20.
    assert quantise(bf(448.0, 17.0, 19.0))[0][0, 1:].tolist() == [16.0, 20.0]
    # The least subnormal code, and half of it.
    assert quantise(bf(448.0, 2.0**-9, 2.0**-10, 1.5 * 2.0**-9))[0][0, 1:].tolist() == [2.0**-9, 0.0, 2.0**-8]
    assert values(torch.tensor([[1.0]]).to(FP8), torch.tensor([130], dtype=torch.uint8))[0, 0] == 8.0


@pytest.mark.parametrize("function", [decode, prefill])
def test_tables_of_more_than_2_26_blocks_are_refused(lib, function):
    kw = dict(B=1, hq=1, hkv=1)
    assert function(lib, W=(1 << 26) + 1, **kw) == 2 and "max_blocks_per_seq" in msg(lib)
    n = ctypes.c_size_t(0)
    assert lib.pkv_fp8_decode_workspace_size(1, 1, 1, 128, (1 << 26) + 1, ctypes.byref(n)) == 2
    assert lib.pkv_fp8_prefill_workspace_size(4, 4, 1, 1, 1, 128, (1 << 26) + 1, ctypes.byref(n)) == 2
