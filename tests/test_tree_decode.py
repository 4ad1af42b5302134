"""GPU attention of drafted token trees over ragged caches (moda_tree_decode) against the
definition in 64 bits, with bounds derived from the kernel's roundings.

Cases: every group-size class, both head sizes, one tile and tile pairs per KV head, cache
lengths 0, 1, around the 128-key block border and long (items cut over many CTAs), lines,
stars and random trees, unused slots, L = 0 to 130.  What must not be read is NaN: the cache
behind each length, every input of an unused slot.
"""
import math
import random

import pytest
import torch

import depth_aware_attention_b200 as moda
from ragged_util import BF, LSE_BOUND, assert_close, joint_attention, randn

pytestmark = pytest.mark.gpu

# name, lengths, S, N, Hq, Hkv, d, L, tree
CASES = [
    ("one-token", [300, 1, 0, 128, 129, 127], 300, 1, 8, 2, 128, 5, "line"),
    ("one-token-L0", [40, 500, 1], 512, 1, 4, 4, 64, 0, "line"),
    ("one-token-long", [20000, 3], 20000, 1, 16, 4, 128, 24, "line"),
    ("line-8", [129, 0, 700], 700, 8, 8, 2, 128, 3, "line"),
    ("star-32-full-tile", [257, 64], 260, 32, 8, 2, 128, 7, "star"),
    ("random-24", [1000, 130, 5], 1024, 24, 16, 4, 128, 24, "random"),
    ("random-13-g3-d64", [77, 400], 400, 13, 6, 2, 64, 4, "random"),
    ("g1-128-tokens", [200, 131], 256, 128, 2, 2, 128, 2, "random"),
    ("g1-d64-5-tokens", [333], 340, 5, 1, 1, 64, 1, "random"),
    ("pair-33", [130, 0, 513], 520, 33, 8, 2, 128, 5, "random"),
    ("pair-61-deep", [3000], 3000, 61, 32, 8, 128, 32, "random"),
    ("pairs-128-g8-d64", [100, 290], 300, 128, 8, 1, 64, 3, "random"),
    ("pairs-odd-g3", [65, 140], 160, 100, 3, 1, 128, 2, "random"),
    ("g16-9", [512, 1], 512, 9, 16, 1, 64, 0, "random"),
    ("g64-3", [260], 260, 3, 64, 1, 128, 6, "random"),
    ("g64-one", [140, 0], 140, 1, 64, 1, 64, 3, "line"),
    ("long-L", [50, 0], 64, 6, 4, 1, 128, 130, "random"),
    ("many-sequences", [(37 * i) % 300 for i in range(70)], 300, 2, 4, 1, 64, 2, "line"),
    # few rows at d = 128: the transposed form, with 4 and with up to 16 rows
    ("rows-1", [700, 0, 128], 700, 1, 2, 2, 128, 3, "line"),
    ("rows-2-deep", [129, 4000], 4000, 2, 3, 3, 128, 200, "random"),
    ("rows-4-tree", [1000, 1, 255], 1024, 4, 2, 2, 128, 5, "random"),
    ("rows-6-odd", [333, 77], 400, 2, 6, 2, 128, 70, "star"),
    ("rows-16-tree", [513, 0, 2000], 2000, 8, 4, 2, 128, 9, "random"),
    ("rows-16-drafts", [1500, 40], 1500, 16, 3, 3, 128, 0, "random"),
    ("rows-15", [260, 127], 300, 5, 6, 2, 128, 17, "random"),
    ("rows-16-group", [3000], 3000, 1, 32, 2, 128, 40, "line"),
    ("rows-many-items", [(53 * i) % 700 for i in range(90)], 700, 1, 8, 4, 128, 24, "line"),
    ("long-64k", [65536, 40000], 65536, 16, 16, 4, 128, 0, "random"),
]
IDS = [c[0] for c in CASES]


def parents_of(kind, B, N, seed):
    r = random.Random(seed)
    rows = []
    for _ in range(B):
        if kind == "line":
            rows.append(list(range(-1, N - 1)))
        elif kind == "star":
            rows.append([-1] + [0] * (N - 1))
        else:
            p = []
            for i in range(N):
                live = [j for j in range(i) if p[j] != -2]
                p.append(-2 if r.random() < 0.2 and i else
                         (r.choice(live[-6:] + [-1]) if live else -1))
            rows.append(p)
    return rows


def visible(parents):
    N = len(parents)
    see = torch.zeros(N, N, dtype=torch.bool)
    for i, p in enumerate(parents):
        if p != -2:
            if p >= 0:
                see[i] = see[p]
            see[i, i] = True
    return see


def make(case, seed):
    _, lens, S, N, Hq, Hkv, d, L, kind = case
    B = len(lens)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = dict(q=randn(g, B, Hq, N, d), k=randn(g, B, Hkv, S, d), v=randn(g, B, Hkv, S, d),
             kt=randn(g, B, Hkv, N, d), vt=randn(g, B, Hkv, N, d))
    if L:
        x.update(kd=randn(g, B, Hkv, N, L, d), vd=randn(g, B, Hkv, N, L, d))
    rows = parents_of(kind, B, N, seed)
    for b in range(B):
        x["k"][b, :, lens[b]:] = float("nan")
        x["v"][b, :, lens[b]:] = float("nan")
        for i in range(N):
            if rows[b][i] == -2:
                for n in ("q", "kt", "vt", "kd", "vd"):
                    if n in x:
                        x[n][b, :, i] = float("inf")
    x["parents"] = torch.tensor(rows, device="cuda", dtype=torch.int32)
    x["lengths"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    return x, rows


def call(x, **kw):
    return moda.tree_decode(x["q"], x["k"], x["v"], x["kt"], x["vt"], x["parents"], x["lengths"],
                            x.get("kd"), x.get("vd"), **kw)


def check(x, rows, case, out, lse):
    name, lens, S, N, Hq, Hkv, d, L, _ = case
    G = Hq // Hkv
    for b, n in enumerate(lens):
        live = [i for i in range(N) if rows[b][i] != -2]
        dead = [i for i in range(N) if rows[b][i] == -2]
        see = visible(rows[b])[live][:, live].cuda()
        see = torch.cat([torch.ones(len(live), n, device="cuda", dtype=torch.bool), see], 1)
        assert (out[b][:, dead] == 0).all() and (lse[b][:, dead] == -math.inf).all(), name
        for g in range(Hkv):
            k = torch.cat([x["k"][b, g, :n], x["kt"][b, g, live]]).double()
            v = torch.cat([x["v"][b, g, :n], x["vt"][b, g, live]]).double()
            kd = x["kd"][b, g, live].double() if L else None
            vd = x["vd"][b, g, live].double() if L else None
            h = slice(g * G, g * G + G)
            r = joint_attention(x["q"][b, h][:, live].double(), k, v, see, kd, vd,
                                1 / math.sqrt(d))
            assert_close(out[b, h][:, live], r["out"], r["out_bound"], f"{name} out b={b} g={g}")
            assert_close(lse[b, h][:, live], r["lse"], LSE_BOUND, f"{name} lse b={b} g={g}")


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_tree_decode(case):
    x, rows = make(case, 4000 + IDS.index(case[0]))
    ws = torch.full((moda.moda_tree_decode_workspace_size(
        len(case[1]), case[4], case[5], case[2], case[3], case[7], case[6]),), 255,
        device="cuda", dtype=torch.uint8)  # NaN bits: nothing in it may be used
    out, lse = call(x, workspace=ws)
    moda.check_device_errors()
    check(x, rows, case, out, lse)
    again = call(x)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]), "not the same bits twice"


def test_one_token_agrees_with_decode_and_the_forwards_last_row():
    # the newest token's key and value are the cache's last entry for moda.decode, and the
    # drafted token's own here
    B, Hq, Hkv, S, d, L = 2, 8, 2, 321, 128, 6
    g = torch.Generator(device="cuda").manual_seed(8)
    k, v = randn(g, B, Hkv, S, d), randn(g, B, Hkv, S, d)
    q, kd, vd = randn(g, B, Hq, d), randn(g, B, Hkv, L, d), randn(g, B, Hkv, L, d)
    want, want_lse = moda.decode(q, k, v, kd, vd)
    lengths = torch.full((B,), S - 1, device="cuda", dtype=torch.int32)
    root = torch.full((B, 1), -1, device="cuda", dtype=torch.int32)
    out, lse = moda.tree_decode(q[:, :, None], k, v, k[:, :, -1:].contiguous(),
                                v[:, :, -1:].contiguous(), root, lengths, kd[:, :, None],
                                vd[:, :, None])
    moda.check_device_errors()
    assert (out[:, :, 0].float() - want.float()).abs().max() <= 1e-2
    assert (lse[:, :, 0] - want_lse).abs().max() <= 1e-3


def test_bad_parents_and_lengths_are_reported():
    case = ("bad", [100, 60], 128, 6, 4, 1, 128, 2, "line")
    x, rows = make(case, 3)
    good = call(x)
    moda.check_device_errors()
    for name, value in (("parents", [[-1, 0, 5, 2, 3, 4], rows[1]]),  # after its child
                        ("parents", [[-1, 0, -2, 2, 3, 4], rows[1]]),  # child of an unused slot
                        ("parents", [[-1, 0, 1, -7, 3, 4], rows[1]]),
                        ("lengths", [100, 129]), ("lengths", [-1, 60])):
        bad = dict(x)
        bad[name] = torch.tensor(value, device="cuda", dtype=torch.int32)
        if name == "lengths":  # a clamped length reads the cache to its end
            bad["k"], bad["v"] = torch.nan_to_num(x["k"]), torch.nan_to_num(x["v"])
        out, _ = call(bad)
        st, flags = moda.moda_check_device_errors()
        assert st == moda.MODA_ERR_INTERNAL and flags == 2, (name, value)
        if name == "parents":
            assert torch.equal(out[1], good[0][1])  # the other sequence is not touched
    again = call(x)
    moda.check_device_errors()
    assert torch.equal(again[0], good[0])


def test_captured_graph_follows_lengths_and_parents():
    first = ("graph", [700, 30, 0], 1000, 20, 8, 2, 128, 4, "random")
    second = ("graph", [10, 1000, 555], 1000, 20, 8, 2, 128, 4, "random")
    (x, xr), (y, yr) = make(first, 21), make(second, 22)
    buf = {n: t.clone() for n, t in x.items()}
    call(buf)  # (lazy loading before the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call(buf)
    for z, rows, case in ((x, xr, first), (y, yr, second), (x, xr, first)):
        for n in buf:
            buf[n].copy_(z[n])
        graph.replay()
        torch.cuda.synchronize()
        check(z, rows, case, out, lse)
    moda.check_device_errors()


def test_two_streams_with_a_workspace_each():
    cases = [("a", [3000, 100], 3000, 7, 8, 2, 128, 4, "random"),
             ("b", [50, 2222], 2300, 40, 8, 2, 128, 4, "random")]
    made = [make(c, 60 + i) for i, c in enumerate(cases)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, (x, _) in enumerate(made):
            with torch.cuda.stream(streams[i]):
                got[i] = call(x)
    torch.cuda.synchronize()
    moda.check_device_errors()
    for (x, rows), case, (out, lse) in zip(made, cases, got):
        check(x, rows, case, out, lse)
