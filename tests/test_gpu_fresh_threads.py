"""Calls that are a host thread's first use of CUDA: nothing has bound the device's context to the thread yet."""
import threading

import pytest
import torch

import paged_kv_cache_275_gb300 as pkv
from gpu_util import device_errors
from plain64 import Pages

pytestmark = pytest.mark.gpu


def calls(hq, d):
    """name -> call(out): every attention call and the appends, with tensors that exist before the thread does."""
    lens, hkv = (300, 40, 700), 2
    p = Pages(lens, hkv, d, hq, width=60)
    kc, vc, table, cl = p.cuda()
    wide = torch.full((3, 4000), -1, dtype=torch.int32, device="cuda")
    wide[:, :60] = table
    q, k, v = p.randn(3, hq, d).cuda(), p.randn(3, hkv, d).cuda(), p.randn(3, hkv, d).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    rows, start, prefix = torch.arange(4, **i32), torch.tensor([0, 1], **i32), torch.tensor([160], **i32)
    none, pos = torch.full((3,), -1, dtype=torch.int64, device="cuda"), torch.arange(3, device="cuda")
    cos_sin = torch.ones(1000, d, device="cuda")
    scratch = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    attend = (q, kc, vc, table, cl)
    return {
        "decode": lambda out: pkv.paged_decode_attention(*attend, 0.1, out),
        "decode with a workspace": lambda out: pkv.paged_decode_attention(*attend, 0.1, out, workspace=scratch),
        "decode step": lambda out: pkv.decode_step(q, k, v, kc, vc, table, cl, 0.1, out, cos_sin),
        "prefill": lambda out: pkv.paged_prefill_attention(*attend, rows, 1, 0.1, out),
        "prefill in splits": lambda out: pkv.paged_prefill_attention(*attend, rows, 1, 0.1, out, num_splits=3),
        "append": lambda out: pkv.kv_append(k, v, none, kc, vc),
        "rotary append": lambda out: pkv.rope_append(q, k, v, pos, pos, cos_sin, kc, vc, out),
        "window decode": lambda out: pkv.paged_window_decode_attention(*attend, 0.1, out, 64, 4),
        "window decode in pieces": lambda out: pkv.paged_window_decode_attention(*attend, 0.1, out, 64, 4, num_partitions=30),
        "window prefill": lambda out: pkv.paged_window_prefill_attention(*attend, rows, 1, 0.1, out, 64, 4, num_splits=1),
        "window prefill in splits": lambda out: pkv.paged_window_prefill_attention(*attend, rows, 1, 0.1, out, 64, 4,
                                                                                  num_splits=3),
        "prefix decode": lambda out: pkv.paged_prefix_decode_attention(*attend, start, prefix, 0.1, out),
        "prefix decode, wide": lambda out: pkv.paged_prefix_decode_attention(q, kc, vc, wide, cl, start, prefix, 0.1, out),
    }, lambda: torch.zeros_like(q)


NAMES = ["decode", "decode with a workspace", "decode step", "prefill", "prefill in splits", "append", "rotary append",
         "window decode", "window decode in pieces", "window prefill", "window prefill in splits", "prefix decode",
         "prefix decode, wide"]


@pytest.mark.parametrize("hq,d", [(16, 128), (4, 64)])
@pytest.mark.parametrize("name", NAMES)
def test_a_threads_first_cuda_call(name, hq, d):
    made, zeros = calls(hq, d)
    assert sorted(made) == sorted(NAMES)
    want, got, raised = zeros(), zeros(), []
    made[name](want)  # (what a process looks up once is looked up here)
    torch.cuda.synchronize()

    def body():
        try:
            made[name](got)
        except Exception as e:
            raised.append(e)

    thread = threading.Thread(target=body)
    thread.start()
    thread.join()
    if raised:
        raise raised[0]
    torch.cuda.synchronize()
    assert torch.equal(want, got)
    assert device_errors() == 0
