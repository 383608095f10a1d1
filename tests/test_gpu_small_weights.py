"""Softmax weights far below the largest one: a key that dominates (an
attention sink) and a long tail of equal small weights whose sum still counts."""
import math

import pytest
import torch

import paged_kv_cache_220_gb300 as pkv
from paged_kv_cache_220_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu

T = 65536
LOGIT = 17.75  # the tail's weights are e^-17.75 = 2^-25.6 of the largest


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.set_device_check(flag)
    yield flag
    pkv.set_device_check(None)


def sink_cache(d, fp8):
    """One sequence's blocks: token 0 has logit LOGIT and V = 0, the others
    logit 0 and V = 1. Codes and values are exact."""
    nb = T // 32
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k = torch.zeros(nb, 1, 32, d, device="cuda")
    v = torch.ones(nb, 1, 32, d, device="cuda")
    k[0, 0, 0, 0] = 16
    v[0, 0, 0] = 0
    k, v = k.to(dt), v.to(dt)
    if fp8:
        k, v = k.view(torch.uint8), v.view(torch.uint8)
    one = torch.ones(1, device="cuda") if fp8 else None
    return k, v, torch.arange(nb, dtype=torch.int32, device="cuda"), one


def verify(out, visible, what):
    """Weights w = e^-LOGIT of `visible` tokens beside the sink's 1: out = n w /
    (1 + n w). Off by the output's rounding to bf16 (2^-8), the fp32 sums and
    exponentials and, on E4M3 pools, a weight's rounding to f16: its exponents
    end at 2^-24 and the largest weight lies at 2^7 or more, so a weight is off
    by at most 2^-25 of 2^7 (below 2^-14 of it; above, by 2^-11 of itself)."""
    n = visible - 1
    w = math.exp(-LOGIT)
    want = n * w / (1 + n * w)
    tol = want * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12) + n * 2.0 ** -32
    err = float((out.double() - want).abs().max())
    assert err <= tol, "%s: off by %.3e, allowed %.3e of %.3e" % (what, err, tol, want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("extra", [0, 40])
def test_tree_counts_a_tail_of_small_weights(d, fp8, extra, _lib):
    """A sequence to a CTA (all share one sequence's blocks), and a few more
    of them, which cuts the sequences between CTAs."""
    k, v, blocks, one = sink_cache(d, fp8)
    S = torch.cuda.get_device_properties(0).multi_processor_count + extra
    q = torch.zeros(S, 2, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1
    out = pkv.paged_attention_tree(
        q, k, v, blocks.repeat(S, 1), torch.full((S,), T, dtype=torch.int32, device="cuda"),
        torch.arange(S + 1, dtype=torch.int32, device="cuda"), LOGIT / 16, T, 1, k_scale=one,
        v_scale=one)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    verify(out, T, "tree")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,block", [(128, 32), (256, 32)])
@pytest.mark.parametrize("partition", [0, 32768])
def test_window_counts_a_tail_of_small_weights(d, block, fp8, partition, _lib):
    """The sink through `sinks`, the tail through the window, one CTA to a
    sequence (partition 0) or two partitions."""
    k, v, blocks, one = sink_cache(d, fp8)
    S = 400
    window = T - 5000
    q = torch.zeros(S, 2, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1
    out = pkv.paged_attention_window(
        q, k, v, blocks.repeat(S, 1), torch.full((S,), T, dtype=torch.int32, device="cuda"),
        LOGIT / 16, T, window, 1, partition, k_scale=one, v_scale=one)
    torch.cuda.synchronize()
    assert int(_lib.item()) == 0
    verify(out, window + 1, "window")
