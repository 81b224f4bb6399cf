"""Host side of the windowed prefill: calls without rows, the split count and the workspace that a call needs (on the
CPU: what is looked at here returns before any CUDA call; pointers are fake, nothing is dereferenced)."""
import ctypes

import pytest

from test_window_prefix_rope_host import lib, msg, window_prefill  # noqa: F401  (lib: a fixture)


@pytest.mark.parametrize("splits", [1, 2])
def test_no_query_rows_is_a_noop(lib, splits):  # noqa: F811
    """Empty chunks under a bound that a caller keeps for a fixed schedule: q and out have no rows, so no address."""
    assert window_prefill(lib, T=0, q=None, out=None, S=splits) == 0 and msg(lib) == ""
    assert window_prefill(lib, T=0, S=splits) == 0
    assert window_prefill(lib, T=0, q=None, window=0) == 1 and "window" in msg(lib)  # (still checked)


@pytest.mark.parametrize("seqs,splits", [(2048, 32), (32768, 2), (65535, 32)])
def test_many_sequences_are_not_refused_for_splits_that_they_do_not_take(lib, seqs, splits):  # noqa: F811
    """Calls of more than 320 sequences are not split, so a count is no reason to refuse them."""
    assert window_prefill(lib, B=seqs, S=splits, T=0) == 0 and msg(lib) == ""
    assert window_prefill(lib, B=seqs, S=33, T=0) == 1 and "num_splits" in msg(lib)


def test_splits_of_a_call_check_arguments_before_the_device(lib):  # noqa: F811
    n = ctypes.c_int32(-1)
    splits = lib.pkv_window_prefill_splits
    assert splits(512, 512, 1, 32, 8, 4, None) == 1 and "used" in msg(lib)
    for bad in ((-1, 512, 1, 32, 8, 4), (512, -1, 1, 32, 8, 4), (512, 512, -1, 32, 8, 4), (512, 512, 1, 30, 8, 4),
                (512, 512, 1, 32, 8, 0), (512, 512, 1, 32, 8, 33)):
        assert splits(*bad, ctypes.byref(n)) == 1, bad
    for one in ((512, 512, 1, 32, 8, 1), (0, 512, 1, 32, 8, 4), (512, 0, 1, 32, 8, 4), (512, 512, 0, 32, 8, 4),
                (512, 512, 321, 32, 8, 4)):
        n.value = -1
        assert splits(*one, ctypes.byref(n)) == 0 and n.value == 1, one
