"""paged_attention_tree where the bound of the contexts is 0: a batch of empty
sequences with a padded q."""
import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build


def test_workspace_of_empty_contexts():
    """The size that the query names is the size that the call asks for: it
    does not depend on the contexts."""
    pkv_build.build()
    for args in ((1, 3, 8, 2, 128), (40, 64, 24, 4, 256)):
        some = pkv.tree_workspace_bytes(*args, 1000, 8)
        assert some > 0 and pkv.tree_workspace_bytes(*args, 0, 8) == some


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_nothing_cached(fp8, given):
    """Nothing is written and nothing reported; a context or drafts that the
    bound does not allow are reported."""
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    dt = torch.uint8 if fp8 else torch.bfloat16
    k = torch.zeros(4, 2, 16, 128, dtype=dt, device="cuda")
    one = torch.ones(2, device="cuda") if fp8 else None
    q = torch.ones(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    tables = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    ws = None
    if given:
        ws = torch.empty(pkv.tree_workspace_bytes(2, 3, 8, 2, 128, 0, 4), dtype=torch.uint8,
                         device="cuda")
    for lens, start, code in (([0, 0], [0, 0, 0], 0), ([0, 0], [1, 1, 1], 0),
                              ([0, 5], [0, 0, 0], pkv.DEVERR_CONTEXT),
                              ([0, 0], [0, 0, 1], pkv.DEVERR_DRAFT)):
        pkv.paged_attention_tree(
            q, k, k.clone(), tables, torch.tensor(lens, dtype=torch.int32, device="cuda"),
            torch.tensor(start, dtype=torch.int32, device="cuda"), 0.1, 0, 4, k_scale=one,
            v_scale=one, out=out, workspace=ws)
        torch.cuda.synchronize()
        assert int(flag.item()) == code
        flag.zero_()
        assert bool((out == 7).all())
    pkv.set_device_check(None)
