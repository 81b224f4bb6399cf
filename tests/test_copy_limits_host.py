"""The most pairs that a block copy takes: two CTAs a pair have to fit a grid of 2^31 - 1.  (Host-checkable: nothing is
dereferenced.)"""
import pytest

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_275_gb300 import _capi, build
    build.build(quiet=True)
    return _capi.load()


def test_pairs(lib):
    assert lib.pkv_copy_blocks(FAKE, FAKE, FAKE, 1 << 30, 8, 128, 10, None) == 2
    assert "num_pairs" in lib.pkv_last_error_message().decode()
    assert lib.pkv_copy_blocks_fp8(FAKE, FAKE, FAKE, FAKE, 1 << 30, 8, 128, 10, None) == 2
    assert "num_pairs" in lib.pkv_last_error_message().decode()
