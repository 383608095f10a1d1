"""Sizes that select_blocks' 32-bit list positions cannot take are refused
(nothing reaches a device)."""
import ctypes

import pytest

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pkv.lib()


def test_longest_lists(lib):
    # far apart, so that nothing overlaps; never dereferenced
    at = [ctypes.c_void_p((i + 1) << 44) for i in range(8)]

    def call(take, S=1, last=1):
        return lib.pkv_select_blocks(at[0], at[1], at[2], at[3], pkv.CacheDesc(8, 16, 1, 128, 0),
                                     at[4], 64, at[5], S, 4, 1024, take, 1, last, at[6], 1 << 40,
                                     None)

    for take in ((1 << 30) + 1, (1 << 31) - 1024, (1 << 31) - 1):
        assert call(take) == pkv.PKV_ERR_UNSUPPORTED
        assert call(take, last=take - 1) == pkv.PKV_ERR_UNSUPPORTED
        assert call(take, last=take) == pkv.PKV_ERR_INVALID_ARG
    assert call(1 << 30, S=0) == pkv.PKV_OK
