"""The bounded waits of the packed forward, the tree attention and the score, made to run out.

The test-only knob shortens every wait to 1 ms and makes the kernels' TMA producers issue no loads.
Each CTA then records the timeout, lets its products in flight finish, releases its tensor memory
and leaves by its normal exit; the next call without the knob gives the same bits as one before it.
Nothing here traps, faults or hangs the GPU.
"""
import pytest
import torch

import depth_aware_attention_b200 as moda
from ragged_util import randn

pytestmark = pytest.mark.gpu

FAULT_NO_LOADS = 1
WAIT_LIMIT_NS = 1_000_000  # 1 ms


def ints(*v):
    return torch.tensor(v, device="cuda", dtype=torch.int32)


def packed(g, lens, Hq, Hkv, d, L):
    N = sum(lens)
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    kd, vd = (randn(g, Hkv, N, L, d) if L else None for _ in range(2))
    args = [randn(g, Hq, N, d), randn(g, Hkv, N, d), randn(g, Hkv, N, d), ints(*ends), kd, vd]
    return lambda: moda.forward_packed(*args)


def tree(g, lens, N, Hq, Hkv, d, L):
    B, S = len(lens), max(lens)
    x = [randn(g, B, Hq, N, d), randn(g, B, Hkv, S, d), randn(g, B, Hkv, S, d),
         randn(g, B, Hkv, N, d), randn(g, B, Hkv, N, d),
         torch.arange(-1, N - 1, device="cuda", dtype=torch.int32).repeat(B, 1), ints(*lens)]
    kd, vd = (randn(g, B, Hkv, N, L, d) if L else None for _ in range(2))
    return lambda: moda.tree_decode(*x, kd, vd)


def score(g, lens, N, Hq, Hkv, d):
    B, S = len(lens), max(lens)
    x = [randn(g, B, Hq, N, d), randn(g, B, Hkv, S, d), torch.full((B, Hq, N), 9.0, device="cuda"),
         ints(*lens), torch.rand(B, Hkv, S, generator=g, device="cuda")]
    return lambda: (moda.cache_score(*x),)


CALLS = {
    "packed-forward": lambda g: packed(g, [2000, 1300], 8, 2, 128, 5),
    "packed-forward-d64": lambda g: packed(g, [2500, 900], 8, 4, 64, 0),
    "packed-single-tiles": lambda g: packed(g, [300, 77], 8, 2, 128, 5),
    "packed-many-items": lambda g: packed(g, [40] * 200, 8, 2, 64, 3),
    "packed-pairs-g3": lambda g: packed(g, [2600, 2300, 2200], 6, 2, 128, 4),
    "tree-4-rows": lambda g: tree(g, [3000, 500, 0], 1, 16, 4, 128, 9),
    "tree-16-rows": lambda g: tree(g, [3000, 500], 4, 16, 4, 128, 9),
    "tree-tile": lambda g: tree(g, [3000, 500], 13, 8, 4, 64, 9),
    "tree-pair": lambda g: tree(g, [3000, 500], 61, 16, 4, 128, 9),
    "tree-many-items": lambda g: tree(g, [333, 1, 129] * 20, 1, 32, 8, 128, 2),
    "score-one-token": lambda g: score(g, [9000, 500], 1, 16, 4, 128),
    "score-four-tiles": lambda g: score(g, [900, 500], 128, 16, 4, 64),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_waits_run_out_and_the_context_recovers(name):
    call = CALLS[name](torch.Generator(device="cuda").manual_seed(7))
    want = call()
    moda.check_device_errors()
    try:
        assert moda.moda_test_set_device_fault(FAULT_NO_LOADS, WAIT_LIMIT_NS) == moda.MODA_OK
        call()
        st, flags = moda.moda_check_device_errors()
    finally:
        assert moda.moda_test_set_device_fault(0, 0) == moda.MODA_OK
    assert st == moda.MODA_ERR_TIMEOUT and flags & 1
    again = call()
    moda.check_device_errors()
    for a, b in zip(want, again):
        assert torch.equal(a, b)
