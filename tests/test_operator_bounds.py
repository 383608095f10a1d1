"""Refusals of sizes and pools that the tree and accept calls cannot take
(nothing reaches a device)."""
import ctypes

import pytest

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
OTHER = ctypes.c_void_p(0x20000)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pkv.lib()


def test_tree_work_beyond_its_numbers(lib):
    """(num_seqs + num_queries g / 128) num_kv_heads (max_context / 128 + 3) of
    2^29 or more is refused."""
    desc = pkv.CacheDesc(8, 16, 8, 128, 0)

    def call(S, N, context):
        return lib.pkv_paged_attention_tree(
            OTHER, FAKE, FAKE, FAKE, desc, None, None, FAKE, 1 << 24, FAKE, FAKE, S, N, 64, None,
            64, context, 0.1, FAKE, 1 << 40, None)

    assert call(65535, 1, 1 << 24) == pkv.PKV_ERR_UNSUPPORTED
    assert call(1, (1 << 30) - 1, 1 << 20) == pkv.PKV_ERR_UNSUPPORTED
    assert call(65535, 1, 128 * 1024) == pkv.PKV_ERR_UNSUPPORTED
    assert call(0, 1 << 30, 1 << 24) == pkv.PKV_OK


@pytest.mark.parametrize("layers", [1, 2, 40, 128, 200])
def test_accept_same_pool_twice(lib, layers):
    def call(k, v):
        arr = ctypes.c_void_p * layers
        return lib.pkv_kv_cache_accept(arr(*k), arr(*v), layers, pkv.CacheDesc(8, 16, 2, 128, 0),
                                       FAKE, 8, FAKE, FAKE, 4, FAKE, 4, FAKE, None, None)

    k = [0x100000 + 0x1000 * i for i in range(layers)]
    v = [0x900000 + 0x1000 * i for i in range(layers)]
    assert call(k, k) == pkv.PKV_ERR_INVALID_ARG
    assert call(k, v[:-1] + [k[0]]) == pkv.PKV_ERR_INVALID_ARG
    if layers > 1:
        assert call([k[1]] + k[1:], v) == pkv.PKV_ERR_INVALID_ARG
