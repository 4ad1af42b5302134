"""Packed batches whose bounds break the rules (they are known on the device alone): the sequences
with the bad entries are treated as empty and reported, and the others are computed as ever, in the
forward and in the backward.  Rows of no sequence stay as they were (in dq, dkd and dvd those before
the first and behind the last good sequence)."""
import math

import pytest
import torch

import depth_aware_attention_b200 as moda
from ragged_util import BF, LSE_BOUND, assert_close, joint_attention, randn

pytestmark = pytest.mark.gpu

# bounds in units, the last one of N = 12 units; what is left of them
BOUNDS = {
    "last-too-low": ([0, 4, 9, 2], [(0, 4), (4, 9)]),
    "last-too-high": ([0, 4, 9, 50], [(0, 4), (4, 9)]),
    "first-negative": ([-3, 4, 9, 12], [(4, 9), (9, 12)]),
    "first-too-high": ([9, 2, 6, 12], [(2, 6), (6, 12)]),
    "gap-in-the-middle": ([1, 4, 20, 7, 11], [(1, 4), (7, 11)]),
    "nothing-left": ([9, 7, -1, -5], []),
}


def step(unit, bounds, G, d, L, causal, seed):
    Hkv, N = 2, 12 * unit
    Hq = G * Hkv
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = dict(q=randn(g, Hq, N, d), k=randn(g, Hkv, N, d), v=randn(g, Hkv, N, d),
             kd=randn(g, Hkv, N, L, d) if L else None, vd=randn(g, Hkv, N, L, d) if L else None,
             dout=randn(g, Hq, N, d))
    cu = torch.tensor([b * unit for b in bounds], device="cuda", dtype=torch.int32)
    args = [x["q"], x["k"], x["v"], cu, x["kd"], x["vd"]]
    out = torch.full((Hq, N, d), 7.0, device="cuda", dtype=BF)
    lse = torch.full((Hq, N), 7.0, device="cuda")
    moda.forward_packed(*args, causal=causal, out=out, lse=lse)
    st = moda.moda_check_device_errors()
    names = ("q", "k", "v") + (("kd", "vd") if L else ())
    grads = {"d" + n: torch.full_like(x[n], 7.0) for n in names}
    ws = torch.full((moda.moda_backward_workspace_size(1, Hq, Hkv, N, L, d),), 255, device="cuda",
                    dtype=torch.uint8)  # NaN bits: nothing in it may be used
    moda.backward_packed(*args, out, lse, x["dout"], causal=causal, grads=grads, workspace=ws)
    return x, out, lse, grads, (st, moda.moda_check_device_errors())


@pytest.mark.parametrize("G,d,L,causal", [(4, 128, 2, True), (3, 64, 3, True), (2, 128, 20, True),
                                          (1, 64, 0, False), (32, 64, 2, True),
                                          (8, 128, 17, False)])
@pytest.mark.parametrize("unit", [1, 10, 150])
@pytest.mark.parametrize("name", sorted(BOUNDS))
def test_good_sequences_among_bad_bounds(name, unit, G, d, L, causal):
    bounds, good = BOUNDS[name]
    x, out, lse, grads, states = step(unit, bounds, G, d, L, causal, 900 + unit)
    assert states == ((moda.MODA_ERR_INTERNAL, 2),) * 2
    left = torch.ones(12 * unit, device="cuda", dtype=torch.bool)
    for a, e in good:
        a, e = a * unit, e * unit
        left[a:e] = False
        see = torch.ones(e - a, e - a, device="cuda", dtype=torch.bool)
        see = see.tril() if causal else see
        for h in range(2):
            rows = slice(h * G, h * G + G)
            w = {n: x[n][h, a:e].double() if x[n] is not None else None
                 for n in ("k", "v", "kd", "vd")}
            r = joint_attention(x["q"][rows, a:e].double(), w["k"], w["v"], see, w["kd"], w["vd"],
                                1 / math.sqrt(d), x["dout"][rows, a:e].double())
            what = f"{name} [{a},{e})"
            assert_close(out[rows, a:e], r["out"], r["out_bound"], what + " out")
            assert_close(lse[rows, a:e], r["lse"], LSE_BOUND, what + " lse")
            assert_close(grads["dq"][rows, a:e], r["dq"], r["dq_bound"], what + " dq")
            for n in list(grads)[1:]:
                assert_close(grads[n][h, a:e], r[n], r[n + "_bound"], f"{what} {n}")
    between = left.clone()
    if good:  # (what the backward leaves alone where some bounds are bad)
        between[good[0][0] * unit:good[-1][1] * unit] = False
    for n, t in dict(grads, out=out, lse=lse).items():
        rows = between if n in ("dq", "dkd", "dvd") else left
        assert (t[:, rows] == 7.0).all(), f"{name}: {n} was written outside the good sequences"
