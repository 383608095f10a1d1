"""Contexts whose positions would not fit the kernels' 32-bit numbers (nothing
reaches a device)."""
import ctypes

import pytest

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build

DESC = pkv.CacheDesc(8, 16, 1, 128, 0)


@pytest.mark.parametrize("blocks", [(1 << 26) + 1, (1 << 27) - 1])
@pytest.mark.parametrize("op", ["window", "tree"])
def test_tables_of_more_than_2_30_tokens(op, blocks):
    """Positions of a step or page may lie behind the context; up to 2^30
    tokens they stay below 2^31."""
    build.build()
    lib, at = pkv.lib(), ctypes.c_void_p
    for context in (0, 1 << 20, 16 * blocks):
        if op == "window":
            rc = lib.pkv_paged_attention_window(
                at(0x10000000), at(0x100000), at(0x200000), at(0x300000), DESC, None, None,
                at(0x10000), blocks, at(0x20000), 1, 8, context, 0.1, 100, 4, 0, None, 0, None,
                None)
        else:
            rc = lib.pkv_paged_attention_tree(
                at(0x10000000), at(0x100000), at(0x200000), at(0x300000), DESC, None, None,
                at(0x10000), blocks, at(0x20000), at(0x30000), 1, 4, 3, None, 8, context, 0.1,
                at(0x400000), 1 << 40, None)
        assert rc == pkv.PKV_ERR_UNSUPPORTED
