"""GPU attention over packed batches (moda_forward_packed, moda_backward_packed) against the
definition in 64 bits, sequence by sequence, with bounds derived from the kernels' roundings.

Cases: every group-size class, both head sizes, both depth paths, lengths 0, 1 and around the
tile and block borders, rows before the first and behind the last sequence (filled with NaN:
they must reach no result, and the outputs there must stay as they were), causal and full.
"""
import math

import pytest
import torch

import depth_aware_attention_b200 as moda
from ragged_util import BF, LSE_BOUND, assert_close, joint_attention, randn

pytestmark = pytest.mark.gpu

# name, lengths, rows before, rows behind, Hq, Hkv, d, L, causal
CASES = [
    ("mixed-g4-d128", [37, 0, 1, 300, 129, 64], 0, 0, 8, 2, 128, 5, True),
    ("borders-g4-d128", [127, 128, 129, 31, 32, 33, 63, 65], 3, 11, 4, 1, 128, 9, True),
    ("g1-d64", [200, 5, 128, 61], 2, 7, 2, 2, 64, 3, True),
    ("g2-d128-L0", [1, 255, 256, 257], 0, 5, 4, 2, 128, 0, True),
    ("g3-d128-fold", [43, 85, 1, 130, 260], 1, 1, 6, 2, 128, 4, True),
    ("g3-d64-fold", [42, 43, 300, 0, 7], 0, 9, 3, 1, 64, 2, True),
    ("g8-d64", [17, 16, 15, 190], 5, 0, 16, 2, 64, 17, True),
    ("g16-d128", [9, 200, 130], 0, 3, 16, 1, 128, 8, True),
    ("g32-d64", [5, 70, 140], 1, 2, 32, 1, 64, 6, True),
    ("g64-d128", [3, 66, 131], 0, 1, 64, 1, 128, 3, True),
    ("long-L", [20, 70], 0, 4, 4, 1, 128, 130, True),
    ("one-token-each", [1] * 70, 0, 0, 8, 2, 128, 1, True),
    ("many", [(7 * i) % 23 for i in range(90)], 4, 4, 4, 1, 64, 2, True),
    ("full-d128", [100, 0, 300, 28], 2, 6, 8, 2, 128, 5, False),
    ("full-d64", [129, 1, 260], 0, 3, 4, 2, 64, 0, False),
    ("full-g3", [50, 130], 3, 0, 6, 2, 128, 2, False),
    ("one-sequence", [1000], 0, 0, 8, 2, 128, 6, True),
    # enough tokens for the forward's own kernel (the ones above run on the tree attention's)
    ("big-g4-d128", [1300, 0, 1, 700, 129, 64, 127, 500], 3, 5, 8, 2, 128, 5, True),
    ("big-g4-d128-L0", [900, 31, 33, 1700, 255], 1, 2, 8, 2, 128, 0, True),
    ("big-g1-d64", [1100, 129, 128, 127, 1300, 260], 0, 7, 8, 8, 64, 3, True),
    ("big-g2-d64", [700, 1, 900, 65, 63], 2, 0, 8, 4, 64, 9, True),
    ("big-g16-d128", [500, 8, 9, 700], 0, 3, 16, 1, 128, 18, True),
    ("big-g32-d64", [300, 5, 400], 1, 1, 32, 1, 64, 33, True),
    ("big-g3-d128", [1200, 83, 85, 84, 1900, 0, 43], 2, 9, 6, 2, 128, 4, True),
    ("big-g3-d64-L0", [1700, 84, 1500], 0, 5, 6, 2, 64, 0, True),
    ("big-g64-d64", [100, 3, 200], 1, 1, 64, 1, 64, 5, True),
    ("big-full-g4", [700, 129, 1500, 1], 4, 3, 8, 2, 128, 5, False),
    ("big-full-g3", [1500, 90, 1700], 0, 3, 6, 2, 64, 3, False),
    # enough key blocks for a CTA each in the backward (the ones above share a block's walk)
    ("big-g1-d64-16-heads", [900, 1100, 1000, 127, 1, 1300, 950, 1029, 700, 800], 0, 3, 16, 16, 64,
     2, True),
    ("big-g1-d128-16-heads", [1000, 1200, 800, 129, 0, 1100, 950, 1029, 700, 900], 1, 0, 16, 16,
     128, 3, True),
    ("big-many", [(13 * i) % 61 for i in range(100)], 2, 2, 16, 4, 128, 4, True),
]
IDS = [c[0] for c in CASES]


def make(case, seed, dout=False, fill=float("nan")):
    _, lens, before, behind, Hq, Hkv, d, L, _ = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    N = before + sum(lens) + behind
    x = dict(q=randn(g, Hq, N, d), k=randn(g, Hkv, N, d), v=randn(g, Hkv, N, d),
             kd=randn(g, Hkv, N, L, d) if L else None, vd=randn(g, Hkv, N, L, d) if L else None)
    if dout:
        x["dout"] = randn(g, Hq, N, d)
    ends = [before]
    for n in lens:
        ends.append(ends[-1] + n)
    for t in x.values():
        if t is not None:
            t[:, :before] = fill
            t[:, ends[-1]:] = fill
    x["cu"] = torch.tensor(ends, device="cuda", dtype=torch.int32)
    return x, ends


def reference(x, a, e, Hq, Hkv, d, causal, dout=False):
    """One sequence in 64 bits, per KV head."""
    G = Hq // Hkv
    see = torch.ones(e - a, e - a, device="cuda", dtype=torch.bool)
    if causal:
        see = see.tril()
    for g in range(Hkv):
        w = {n: (None if t is None else t[g, a:e].double())
             for n, t in x.items() if n in ("k", "v", "kd", "vd")}
        rows = slice(g * G, g * G + G)
        yield g, rows, joint_attention(x["q"][rows, a:e].double(), w["k"], w["v"], see, w["kd"],
                                       w["vd"], 1.0 / math.sqrt(d),
                                       x["dout"][rows, a:e].double() if dout else None)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_packed(case):
    name, _, _, _, Hq, Hkv, d, L, causal = case
    x, ends = make(case, 1000 + IDS.index(name))
    N = x["q"].shape[1]
    out = torch.full((Hq, N, d), 7.0, device="cuda", dtype=BF)
    lse = torch.full((Hq, N), 7.0, device="cuda")
    moda.forward_packed(x["q"], x["k"], x["v"], x["cu"], x["kd"], x["vd"], causal=causal, out=out,
                        lse=lse)
    moda.check_device_errors()
    for a, e in zip(ends[:-1], ends[1:]):
        for _, rows, r in reference(x, a, e, Hq, Hkv, d, causal):
            assert_close(out[rows, a:e], r["out"], r["out_bound"], f"{name} out [{a},{e})")
            assert_close(lse[rows, a:e], r["lse"], LSE_BOUND, f"{name} lse [{a},{e})")
    for t in (out[:, :ends[0]], out[:, ends[-1]:], lse[:, :ends[0]], lse[:, ends[-1]:]):
        assert (t == 7.0).all(), f"{name}: a row outside all sequences was written"


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward_packed(case):
    name, _, _, _, Hq, Hkv, d, L, causal = case
    x, ends = make(case, 2000 + IDS.index(name), dout=True)
    args = [x[n] for n in ("q", "k", "v", "cu", "kd", "vd")]
    N = x["q"].shape[1]
    out = torch.full((Hq, N, d), float("nan"), device="cuda", dtype=BF)
    lse = torch.full((Hq, N), float("nan"), device="cuda")
    moda.forward_packed(*args, causal=causal, out=out, lse=lse)
    names = ("q", "k", "v") + (("kd", "vd") if L else ())
    grads = {"d" + n: torch.full_like(x[n], 7.0) for n in names}
    ws = torch.full((moda.moda_backward_workspace_size(1, Hq, Hkv, N, L, d),), 255,
                    device="cuda", dtype=torch.uint8)  # NaN bits: nothing in it may be used
    moda.backward_packed(*args, out, lse, x["dout"], causal=causal, grads=grads, workspace=ws)
    moda.check_device_errors()
    for a, e in zip(ends[:-1], ends[1:]):
        for g, rows, r in reference(x, a, e, Hq, Hkv, d, causal, dout=True):
            what = f"{name} [{a},{e})"
            assert_close(grads["dq"][rows, a:e], r["dq"], r["dq_bound"], what + " dq")
            for n in names[1:]:
                n = "d" + n
                assert_close(grads[n][g, a:e], r[n], r[n + "_bound"], f"{what} {n}")
    for n, t in grads.items():
        assert (t[:, :ends[0]] == 7.0).all() and (t[:, ends[-1]:] == 7.0).all(), (
            f"{name}: {n} was written outside all sequences")


@pytest.mark.parametrize("causal", [True, False])
def test_each_sequence_equals_its_own_forward(causal):
    # the forward's kernel over the same blocks: every bit agrees with moda_forward's
    case = ("bits", [3000, 64, 1, 1290], 0, 5, 8, 2, 128, 6, causal)
    x, ends = make(case, 31)
    out, lse = moda.forward_packed(x["q"], x["k"], x["v"], x["cu"], x["kd"], x["vd"],
                                   causal=causal)
    for a, e in zip(ends[:-1], ends[1:]):
        one = [x[n][None, :, a:e].contiguous() for n in ("q", "k", "v", "kd", "vd")]
        o, ls = moda.forward(*one, causal=causal)
        assert torch.equal(out[:, a:e], o[0]) and torch.equal(lse[:, a:e], ls[0])
    moda.check_device_errors()


@pytest.mark.parametrize("G", [3, 4])
@pytest.mark.parametrize("times", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_a_neighbours_infinities_stay_with_it(d, times, G):
    # one sequence full of NaN and infinities between two others, in every input
    case = ("neighbours", [45 * times, 50 * times, 75], 0, 0, 2 * G, 2, d, 3, True)
    x, ends = make(case, 77, dout=True)
    args = [x[n] for n in ("q", "k", "v", "cu", "kd", "vd")]
    out, lse = moda.forward_packed(*args)
    good = moda.backward_packed(*args, out, lse, x["dout"])
    for i, n in enumerate(("q", "k", "v", "kd", "vd", "dout")):
        x[n][:, ends[1]:ends[2]] = (float("nan"), float("inf"))[i % 2]
    out2, lse2 = moda.forward_packed(*args)
    bad = moda.backward_packed(*args, out2, lse2, x["dout"])
    moda.check_device_errors()
    for part in (slice(ends[0], ends[1]), slice(ends[2], ends[3])):
        assert torch.equal(out[:, part], out2[:, part]) and torch.equal(lse[:, part], lse2[:, part])
        for n in ("dkd", "dvd"):
            assert torch.equal(good[n][:, part], bad[n][:, part]), n
        for n in ("dq", "dk", "dv"):  # their last bits may differ between runs
            assert torch.isfinite(bad[n][:, part]).all(), n
            diff = (good[n][:, part].float() - bad[n][:, part].float()).abs()
            assert diff.max() <= 2.0 ** -7 * good[n][:, part].float().abs().max() * 2, n


def test_bad_bounds_are_reported_and_stay_in_range():
    case = ("bad", [40, 30, 50], 0, 0, 4, 1, 128, 2, True)
    x, ends = make(case, 5)
    ok, _ = moda.forward_packed(x["q"], x["k"], x["v"], x["cu"], x["kd"], x["vd"])
    moda.check_device_errors()
    for cu in ([0, 40, 30, 120], [0, 40, 200, 120], [-3, 40, 70, 120]):
        bad = torch.tensor(cu, device="cuda", dtype=torch.int32)
        moda.forward_packed(x["q"], x["k"], x["v"], bad, x["kd"], x["vd"])
        st, flags = moda.moda_check_device_errors()
        assert st == moda.MODA_ERR_INTERNAL and flags == 2, cu
    again, _ = moda.forward_packed(x["q"], x["k"], x["v"], x["cu"], x["kd"], x["vd"])
    moda.check_device_errors()
    assert torch.equal(ok, again)


def test_captured_graph_follows_new_lengths():
    # one graph, replayed after the bounds and the inputs changed, on a stream of its own
    first = ("graph", [100, 20, 44], 0, 0, 8, 2, 128, 4, True)
    second = ("graph", [3, 150, 11], 0, 0, 8, 2, 128, 4, True)
    x, _ = make(first, 11)
    y, _ = make(second, 12)
    want = [moda.forward_packed(z["q"], z["k"], z["v"], z["cu"], z["kd"], z["vd"])
            for z in (x, y)]
    buf = {n: t.clone() for n, t in x.items()}
    out, lse = torch.empty_like(x["q"]), torch.empty(8, 164, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moda.forward_packed(buf["q"], buf["k"], buf["v"], buf["cu"], buf["kd"], buf["vd"],
                            out=out, lse=lse)
    for z, (o, ls) in zip((x, y), want):
        for n in buf:
            buf[n].copy_(z[n])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(lse, ls)
    moda.check_device_errors()


def test_gradient_against_differences():
    # d/de of sum(out * dout) along random directions, by central differences of the
    # definition in 64 bits at the same bf16 inputs
    case = ("differences", [33, 70], 0, 0, 4, 2, 64, 3, True)
    name, _, _, _, Hq, Hkv, d, L, causal = case
    x, ends = make(case, 99, dout=True)
    args = [x[n] for n in ("q", "k", "v", "cu", "kd", "vd")]
    out, lse = moda.forward_packed(*args)
    grads = moda.backward_packed(*args, out, lse, x["dout"])
    moda.check_device_errors()

    def value(y):
        total = 0.0
        for a, e in zip(ends[:-1], ends[1:]):
            for _, rows, r in reference(y, a, e, Hq, Hkv, d, causal):
                total += (r["out"] * x["dout"][rows, a:e].double()).sum().item()
        return total

    g = torch.Generator(device="cuda").manual_seed(3)
    for n in ("q", "k", "v", "kd", "vd"):
        u = torch.randn(x[n].shape, generator=g, device="cuda", dtype=torch.float64)
        y = {m: (t if m == "cu" else t.double()) for m, t in x.items()}
        h = 1e-5
        y[n] = x[n].double() + h * u
        up = value(y)
        y[n] = x[n].double() - h * u
        slope = (up - value(y)) / (2 * h)
        got = (grads["d" + n].double() * u).sum().item()
        # the directional sum's error: each element off by a few U of its size, independently
        sigma = 4 * (2.0 ** -8) * (grads["d" + n].double() * u).pow(2).sum().sqrt().item()
        assert abs(got - slope) <= 6 * sigma + 1e-3, (n, got, slope)


@pytest.mark.parametrize("d,L,G,causal", [(64, 0, 1, True), (128, 0, 1, True), (128, 3, 3, True),
                                          (64, 5, 4, True), (128, 1, 16, False), (64, 0, 8, False)])
def test_short_sequences_lose_no_precision(d, L, G, causal):
    # many sequences of a few tokens: dq's relative error is made of two roundings of the same
    # size, of dS to bf16 and of dq itself (its row term D comes from the keys), so it is at
    # most sqrt(2) of the second alone; a tenth more for the fp32 sums and the sample
    case = ("short", [5, 2, 7, 3, 1, 6] * 40, 0, 0, 2 * G, 2, d, L, causal)
    x, ends = make(case, 321, dout=True)
    args = [x[n] for n in ("q", "k", "v", "cu", "kd", "vd")]
    out, lse = moda.forward_packed(*args, causal=causal)
    g = moda.backward_packed(*args, out, lse, x["dout"], causal=causal)
    moda.check_device_errors()
    off = rounding = 0.0
    for a, e in zip(ends[:-1], ends[1:]):
        for _, rows, r in reference(x, a, e, 2 * G, 2, d, causal, dout=True):
            off += (g["dq"][rows, a:e].double() - r["dq"]).square().sum().item()
            rounding += (r["dq"].to(BF).double() - r["dq"]).square().sum().item()
    assert math.sqrt(off) <= 1.1 * math.sqrt(2 * rounding), math.sqrt(off / rounding)
