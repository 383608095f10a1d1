"""Buffers that overlap where one is written while another is read (nothing
reaches a device)."""
import ctypes

import pytest

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build

OK, INV = pkv.PKV_OK, pkv.PKV_ERR_INVALID_ARG
DESC = pkv.CacheDesc(8, 16, 2, 128, 0)
POOL = 8 * 16 * 2 * 128 * 2  # bytes


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pkv.lib()


def at(x):
    return ctypes.c_void_p(x)


def accept(lib, new, k=(0x100000, 0x200000), v=(0x300000, 0x400000), S=4, M=3):
    """Addresses, 4-byte elements: lengths 0x10000, starts 0x20000, lists
    0x30000, their numbers 0x40000, tables 0x50000 (8 blocks a sequence)."""
    arr = ctypes.c_void_p * len(k)
    return lib.pkv_kv_cache_accept(arr(*k), arr(*v), len(k), DESC, at(0x50000), 8, at(0x10000),
                                   at(0x20000), S, at(0x30000), M, at(0x40000), at(new), None)


# every CTA of the launch reads the lists, their numbers, the starts, the
# lengths and the tables; one of them writes the new lengths
@pytest.mark.parametrize("new", [0x10000, 0x10000 - 12, 0x10000 + 12,     # lengths
                                 0x20000, 0x20000 + 16, 0x20000 - 12,     # starts
                                 0x30000, 0x30000 + 44, 0x30000 - 12,     # lists
                                 0x40000, 0x40000 + 12, 0x40000 - 12,     # numbers
                                 0x50000, 0x50000 + 124])                 # tables
def test_new_lengths_over_what_is_read(lib, new):
    assert accept(lib, new) == INV


@pytest.mark.parametrize("layers", [2, 130])
def test_pools_that_overlap(lib, layers):
    """A row of one pool would move while the other pool's move reads it."""
    step = 2 * POOL
    k = [0x10000000 + step * i for i in range(layers)]
    v = [0x40000000 + step * i for i in range(layers)]
    for shift in (16, POOL // 2, POOL - 16, -16, 16 - POOL):
        assert accept(lib, 0x60000, k, [k[-1] + shift] + v[1:]) == INV
        assert accept(lib, 0x60000, k, v[:-1] + [v[0] + shift]) == INV


@pytest.mark.parametrize("op", ["window", "tree"])
def test_result_over_the_queries(lib, op):
    """q and out: 4 rows of 8 heads of 128 (8192 bytes)."""
    def call(out):
        if op == "window":
            return lib.pkv_paged_attention_window(
                at(out), at(0x100000), at(0x200000), at(0x300000), DESC, None, None, at(0x10000),
                64, at(0x20000), 4, 8, 1024, 0.1, 100, 4, 0, None, 0, None, None)
        return lib.pkv_paged_attention_tree(
            at(out), at(0x100000), at(0x200000), at(0x300000), DESC, None, None, at(0x10000), 64,
            at(0x20000), at(0x30000), 2, 4, 3, None, 8, 1024, 0.1, at(0x400000), 1 << 40, None)

    for out in (0x100000, 0x100010, 0x100000 + 8192 - 16, 0x100000 - 16, 0x100000 - 8192 + 16):
        assert call(out) == INV
