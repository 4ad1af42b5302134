"""The ragged-batch operators together, as a server uses them: prompts of different lengths
are prefilled as one packed batch, fill the caches, drafted trees are checked against them,
the accepted tokens are appended, the keys are scored and the caches cut down, and decoding
goes on over the shorter caches.  Every attention and score is compared with the definition
in 64 bits on the very bits the operators were given.
"""
import math

import pytest
import torch

import depth_aware_attention_b200 as moda
from ragged_util import BF, LSE_BOUND, assert_close, joint_attention, randn
from test_tree_decode import visible

pytestmark = pytest.mark.gpu

HQ, HKV, D, L = 8, 2, 128, 5
G = HQ // HKV
SCALE = 1.0 / math.sqrt(D)


def check_tree(x, parents, lens, out, lse, what):
    for b, n in enumerate(lens):
        see = torch.cat([torch.ones(len(parents), n, dtype=torch.bool), visible(parents)], 1)
        for g in range(HKV):
            h = slice(g * G, g * G + G)
            r = joint_attention(
                x["q"][b, h].double(), torch.cat([x["k"][b, g, :n], x["kt"][b, g]]).double(),
                torch.cat([x["v"][b, g, :n], x["vt"][b, g]]).double(), see.cuda(),
                x["kd"][b, g].double(), x["vd"][b, g].double(), SCALE)
            assert_close(out[b, h], r["out"], r["out_bound"], f"{what} out {b}")
            assert_close(lse[b, h], r["lse"], LSE_BOUND, f"{what} lse {b}")


def test_prefill_draft_score_evict_decode():
    lens, S, keep, window = [190, 41, 333], 400, 100, 16
    B = len(lens)
    gen = torch.Generator(device="cuda").manual_seed(2024)

    # ---- prefill of the packed prompts
    N = sum(lens)
    ends = [0, 190, 231, 564]
    cu = torch.tensor(ends, device="cuda", dtype=torch.int32)
    p = dict(q=randn(gen, HQ, N, D), k=randn(gen, HKV, N, D), v=randn(gen, HKV, N, D),
             kd=randn(gen, HKV, N, L, D), vd=randn(gen, HKV, N, L, D))
    out, lse = moda.forward_packed(p["q"], p["k"], p["v"], cu, p["kd"], p["vd"])
    moda.check_device_errors()
    for b, (a, e) in enumerate(zip(ends[:-1], ends[1:])):
        see = torch.ones(e - a, e - a, device="cuda", dtype=torch.bool).tril()
        for g in range(HKV):
            h = slice(g * G, g * G + G)
            r = joint_attention(*(p[n][s].double() for n, s in (
                ("q", (h, slice(a, e))), ("k", (g, slice(a, e))), ("v", (g, slice(a, e))))), see,
                p["kd"][g, a:e].double(), p["vd"][g, a:e].double(), SCALE)
            assert_close(out[h, a:e], r["out"], r["out_bound"], f"prefill {b}")

    # ---- the caches (memory behind each length is whatever it was), scores of the window
    k = torch.full((B, HKV, S, D), float("nan"), device="cuda", dtype=BF)
    v = torch.full_like(k, float("nan"))
    for b, (a, e) in enumerate(zip(ends[:-1], ends[1:])):
        k[b, :, :e - a], v[b, :, :e - a] = p["k"][:, a:e], p["v"][:, a:e]
    lengths = torch.tensor(lens, device="cuda", dtype=torch.int32)
    qw = torch.stack([p["q"][:, e - window:e] for e in ends[1:]])
    lw = torch.stack([lse[:, e - window:e] for e in ends[1:]])
    score = moda.cache_score(qw, k, lw, lengths, torch.zeros(B, HKV, S, device="cuda"))

    # ---- a drafted tree; the path 0 -> 2 -> 3 is accepted
    parents = [-1, 0, 0, 2, 1]
    T = len(parents)
    x = dict(q=randn(gen, B, HQ, T, D), k=k, v=v, kt=randn(gen, B, HKV, T, D),
             vt=randn(gen, B, HKV, T, D), kd=randn(gen, B, HKV, T, L, D),
             vd=randn(gen, B, HKV, T, L, D))
    par = torch.tensor([parents] * B, device="cuda", dtype=torch.int32)
    o1, l1 = moda.tree_decode(x["q"], k, v, x["kt"], x["vt"], par, lengths, x["kd"], x["vd"])
    moda.check_device_errors()
    check_tree(x, parents, lens, o1, l1, "draft")
    path = [0, 2, 3]
    for b, n in enumerate(lens):
        k[b, :, n:n + 3], v[b, :, n:n + 3] = x["kt"][b, :, path], x["vt"][b, :, path]
    lengths = lengths + 3
    lens = [n + 3 for n in lens]

    # ---- the accepted tokens' weights (in place), against 64 bits over everything so far
    moda.cache_score(x["q"][:, :, path].contiguous(), k, l1[:, :, path].contiguous(), lengths,
                     score, out=score)
    moda.check_device_errors()
    for b, n in enumerate(lens):
        want = torch.zeros(HKV, n, device="cuda", dtype=torch.float64)
        queries = [(qw[b, :, i], lw[b, :, i], n - 3 - window + i) for i in range(window)]
        queries += [(x["q"][b, :, t], l1[b, :, t], n - 3 + i) for i, t in enumerate(path)]
        for q, ls, pos in queries:
            z = torch.einsum("hgd,hsd->hgs", q.double().view(HKV, G, D),
                             k[b, :, :pos + 1].double()) * SCALE
            want[:, :pos + 1] += torch.exp(z - ls.double().view(HKV, G, 1)).sum(1)
        # the bound of the score's own tests, over two calls
        assert ((score[b, :, :n].double() - want).abs() <= 2e-4 * want + 1e-9).all()

    # ---- eviction, and on with single tokens over the shorter caches
    r = moda.cache_evict(k, v, score, lengths, keep, sinks=4, recent=32)
    kept = [min(n, keep) for n in lens]
    assert r["lengths_out"].tolist() == kept
    for b, n in enumerate(kept):
        at = r["index"][b, :, :n].long()
        assert (at[:, 1:] > at[:, :-1]).all() and (at[:, -1] == lens[b] - 1).all()
        for g in range(HKV):
            assert torch.equal(r["k_out"][b, g, :n], k[b, g, at[g]])
            dropped = torch.ones(lens[b], device="cuda", dtype=torch.bool)
            dropped[at[g]] = False
            if dropped.any():
                free = at[g][(at[g] >= 4) & (at[g] < lens[b] - 32)]
                row = score[b, g, :lens[b]]
                assert row[dropped].max() <= row[free].min()
    y = dict(q=randn(gen, B, HQ, 1, D), k=r["k_out"], v=r["v_out"], kt=randn(gen, B, HKV, 1, D),
             vt=randn(gen, B, HKV, 1, D), kd=randn(gen, B, HKV, 1, L, D),
             vd=randn(gen, B, HKV, 1, L, D))
    root = torch.full((B, 1), -1, device="cuda", dtype=torch.int32)
    o2, l2 = moda.tree_decode(y["q"], y["k"], y["v"], y["kt"], y["vt"], root, r["lengths_out"],
                              y["kd"], y["vd"])
    moda.check_device_errors()
    check_tree(y, [-1], kept, o2, l2, "decode")
