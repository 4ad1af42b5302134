"""GPU cache scores and eviction (moda_cache_score, moda_cache_evict) against the definitions:
the scores in 64 bits, the eviction exactly (its outputs are copies and positions).

What must not be read is NaN: keys and scores behind each length, queries of rows that carry
no weight.  Outputs are filled beforehand and must stay as they were behind their last row.
"""
import math

import numpy as np
import pytest
import torch

import depth_aware_attention_b200 as moda
from ragged_util import BF, randn

pytestmark = pytest.mark.gpu

# ------------------------------------------------------------------------------- scores
# name, lengths, S, N, Hq, Hkv, d
SCORES = [
    ("one-token", [300, 1, 0, 128, 129], 300, 1, 8, 2, 128),
    ("one-token-g1-d64", [777, 40], 800, 1, 3, 3, 64),
    ("one-token-long", [50000, 12345], 50000, 1, 16, 4, 128),
    ("window-33", [500, 33, 12, 0], 512, 33, 8, 2, 128),
    ("window-g3", [260, 130], 300, 45, 6, 2, 64),
    ("two-tiles", [1000], 1024, 64, 8, 2, 128),
    ("three-tiles-d64", [400, 200], 400, 96, 4, 1, 64),
    ("two-launches", [300, 90], 320, 128, 4, 1, 128),
    ("three-launches-g8", [513], 520, 128, 8, 1, 128),
    ("g64", [140, 3], 150, 5, 64, 1, 64),
    ("g5-odd", [70], 71, 7, 5, 1, 128),
    ("many-sequences", [(31 * i) % 290 for i in range(80)], 290, 2, 4, 1, 64),
]


def score_inputs(case, seed):
    _, lens, S, N, Hq, Hkv, d = case
    B, G = len(lens), Hq // Hkv
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = dict(q=randn(g, B, Hq, N, d), k=randn(g, B, Hkv, S, d),
             score=torch.rand(B, Hkv, S, generator=g, device="cuda"))
    lse = torch.zeros(B, Hq, N, device="cuda")
    for b, n in enumerate(lens):
        x["k"][b, :, n:] = float("nan")
        x["score"][b, :, n:] = float("nan")
        for i in range(N):
            if n - N + i < 0:
                x["q"][b, :, i] = float("inf")
                continue
            z = torch.einsum("hgd,hsd->hgs", x["q"][b, :, i].double().view(Hkv, G, d),
                             x["k"][b, :, :n - N + i + 1].double()) / math.sqrt(d)
            lse[b, :, i] = torch.logsumexp(z, -1).view(Hq).float() + 0.25
    # a row that saw nothing (an unused slot of a drafted tree)
    if N > 2:
        lse[:, 0, 1] = -math.inf
        x["q"][:, 0, 1] = float("nan")
    x["lse"] = lse
    x["lengths"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    return x


def score_reference(x, case):
    _, lens, S, N, Hq, Hkv, d = case
    G = Hq // Hkv
    total = x["score"].double().clone()
    added = torch.zeros_like(total)
    for b, n in enumerate(lens):
        for h in range(Hq):
            for i in range(N):
                e = n - N + i + 1
                if e <= 0 or x["lse"][b, h, i] == -math.inf:
                    continue
                z = x["k"][b, h // G, :e].double() @ x["q"][b, h, i].double() / math.sqrt(d)
                added[b, h // G, :e] += torch.exp(z - x["lse"][b, h, i].double())
    return total + added, added


@pytest.mark.parametrize("case", SCORES, ids=[c[0] for c in SCORES])
def test_cache_score(case):
    x = score_inputs(case, 70 + len(case[0]))
    args = [x[n] for n in ("q", "k", "lse", "lengths", "score")]
    before = x["score"].clone()
    out = moda.cache_score(*args)
    moda.check_device_errors()
    assert torch.equal(x["score"].nan_to_num(-1), before.nan_to_num(-1)), "the input changed"
    ref, added = score_reference(x, case)
    # the exponent x = logit - lse is an fp32 sum of 128 exact products (worst case 128 * 2^-24
    # of sum |q k| scale, under 6e-5), of the scaled lse and its own rounding (under 1e-5), so
    # each weight is within 1e-4 of itself; then fp32 sums: 2^-24 a term, at most 1100 terms
    for b, n in enumerate(case[1]):
        err = (out[b, :, :n].double() - ref[b, :, :n]).abs()
        bound = 1e-4 * added[b, :, :n] + 1100 * 2.0 ** -24 * ref[b, :, :n] + 1e-12
        assert (err <= bound).all(), (case[0], b, (err - bound).max().item())
        assert out[b, :, n:].isnan().all()  # copied as they were
    again = x["score"].clone()
    moda.cache_score(*args[:4], again, out=again)  # in place
    assert torch.equal(again.nan_to_num(-1), out.nan_to_num(-1))
    moda.check_device_errors()


def test_the_weights_of_one_query_sum_to_what_attention_gave_them():
    # one token, no depth entries, lse from tree_decode over the cache and the token itself:
    # the scores of the cached keys and the token's own weight add up to 1 per head
    B, Hkv, G, S, d = 2, 2, 4, 600, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v, q = randn(g, B, Hkv, S, d), randn(g, B, Hkv, S, d), randn(g, B, Hkv * G, 1, d)
    lengths = torch.tensor([600, 77], device="cuda", dtype=torch.int32)
    kt, vt = k[:, :, :1].clone(), v[:, :, :1].clone()
    for b, n in enumerate((600, 77)):  # the newest token's entry is the cache's last
        kt[b, :, 0], vt[b, :, 0] = k[b, :, n - 1], v[b, :, n - 1]
    root = torch.full((B, 1), -1, device="cuda", dtype=torch.int32)
    _, lse = moda.tree_decode(q, k, v, kt, vt, root, lengths - 1)
    total = moda.cache_score(q, k, lse, lengths, torch.zeros(B, Hkv, S, device="cuda"))
    moda.check_device_errors()
    assert (total.sum(-1) - G).abs().max() <= G * 1e-3


# ------------------------------------------------------------------------------- eviction
def evict_reference(score, n, keep, sinks, recent):
    """Kept positions of one row, by the definition."""
    if n <= keep:
        return np.arange(n)
    s = score[:n].astype(np.float64).copy()
    rank = np.where(np.isnan(s), -np.inf, s)
    below = np.isnan(s)  # a NaN is less than -inf
    must = np.zeros(n, bool)
    must[:sinks] = True
    must[n - recent:] = True
    order = np.lexsort((np.arange(n), -rank, below & ~must, ~must))
    return np.sort(order[:keep])


# name, lengths, S, keep, sinks, recent, Hkv, d, kind of scores
EVICTS = [
    ("small", [300, 100, 0, 1, 64, 65], 300, 64, 4, 16, 2, 128, "weights"),
    ("keep-one", [50, 3], 64, 1, 0, 0, 1, 64, "weights"),
    ("all-equal", [200, 150], 200, 77, 3, 10, 2, 64, "equal"),
    ("special", [500, 333], 512, 100, 0, 5, 2, 128, "special"),
    ("all-protected", [400], 400, 60, 20, 40, 1, 128, "weights"),
    ("keep-over-S", [90, 128], 128, 200, 2, 3, 2, 64, "weights"),
    ("one-cta-limit", [4096, 4000], 4096, 1000, 4, 100, 1, 64, "ties"),
    ("cluster-first", [4097, 17, 1030], 4097, 1024, 4, 100, 2, 64, "ties"),
    ("cluster", [20000, 9999], 20000, 3001, 4, 256, 2, 128, "weights"),
    ("cluster-equal", [30000], 30000, 7001, 0, 0, 1, 64, "equal"),
    ("cluster-special", [33333, 33332], 33333, 12345, 1, 1, 1, 64, "special"),
    ("cluster-all-protected", [10000], 10000, 600, 100, 500, 2, 64, "weights"),
    ("cluster-one-left", [8193], 8193, 8192, 0, 8191, 1, 64, "weights"),
    ("one-cta-odd", [8191, 8192], 8192, 4095, 5, 77, 1, 64, "special"),
    ("cluster-8193", [8193, 8000], 8193, 100, 5, 77, 1, 64, "ties"),
    ("long", [131072, 100], 131072, 30000, 4, 1000, 1, 64, "ties"),
    ("not-held", [200001, 150, 60000], 200001, 30000, 4, 1000, 1, 64, "special"),
]


def evict_scores(kind, g, B, Hkv, S):
    u = torch.rand(B, Hkv, S, generator=g, device="cuda")
    if kind == "weights":
        return u.pow(8)
    if kind == "equal":
        return torch.full_like(u, 0.25)
    if kind == "ties":
        return (u * 16).floor() / 16
    special = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-40, -1e-40,
                            2e-40, 1.0, -1.0, 3.4e38, -3.4e38, -float("nan")], device="cuda")
    return special[(u * special.numel()).long()]


@pytest.mark.parametrize("case", EVICTS, ids=[c[0] for c in EVICTS])
def test_cache_evict(case):
    name, lens, S, keep, sinks, recent, Hkv, d, kind = case
    B = len(lens)
    g = torch.Generator(device="cuda").manual_seed(len(name))
    k, v = randn(g, B, Hkv, S, d), randn(g, B, Hkv, S, d)
    score = evict_scores(kind, g, B, Hkv, S)
    for b, n in enumerate(lens):
        score[b, :, n:] = float("inf")  # behind the length: would win everywhere
    lengths = torch.tensor(lens, device="cuda", dtype=torch.int32)
    outs = dict(k_out=torch.full((B, Hkv, keep, d), 7.0, device="cuda", dtype=BF),
                v_out=torch.full((B, Hkv, keep, d), 7.0, device="cuda", dtype=BF),
                score_out=torch.full((B, Hkv, keep), 7.0, device="cuda"),
                index=torch.full((B, Hkv, keep), 7, device="cuda", dtype=torch.int32),
                lengths_out=torch.full((B,), 7, device="cuda", dtype=torch.int32))
    r = moda.cache_evict(k, v, score, lengths, keep, sinks, recent, **outs)
    moda.check_device_errors()
    assert r["lengths_out"].tolist() == [min(n, keep) for n in lens]
    host = score.cpu().numpy()
    for b, n in enumerate(lens):
        kept = min(n, keep)
        for h in range(Hkv):
            at = evict_reference(host[b, h], n, keep, sinks, recent)
            assert np.array_equal(r["index"][b, h, :kept].cpu().numpy(), at), (name, b, h)
            rows = torch.from_numpy(at).cuda()
            assert torch.equal(r["k_out"][b, h, :kept], k[b, h, rows])
            assert torch.equal(r["v_out"][b, h, :kept], v[b, h, rows])
            assert torch.equal(r["score_out"][b, h, :kept].view(torch.int32),
                               score[b, h, rows].view(torch.int32))
        for n_, fill in (("k_out", 7.0), ("v_out", 7.0), ("score_out", 7.0), ("index", 7)):
            assert (r[n_][b, :, kept:] == fill).all(), (name, n_)


def test_bad_lengths_are_reported():
    g = torch.Generator(device="cuda").manual_seed(1)
    k, score = randn(g, 2, 1, 100, 64), torch.rand(2, 1, 100, device="cuda")
    q, lse = randn(g, 2, 4, 1, 64), torch.zeros(2, 4, 1, device="cuda")
    for lens in ([101, 5], [5, -1]):
        lengths = torch.tensor(lens, device="cuda", dtype=torch.int32)
        moda.cache_evict(k, k.clone(), score, lengths, 10)
        assert moda.moda_check_device_errors() == (moda.MODA_ERR_INTERNAL, 2)
        moda.cache_score(q, k, lse, lengths, score)
        assert moda.moda_check_device_errors() == (moda.MODA_ERR_INTERNAL, 2)
    moda.check_device_errors()


def test_captured_graph_scores_then_evicts():
    B, Hq, Hkv, S, d, keep = 2, 8, 2, 5000, 128, 700
    g = torch.Generator(device="cuda").manual_seed(9)
    k, v, q = randn(g, B, Hkv, S, d), randn(g, B, Hkv, S, d), randn(g, B, Hq, 3, d)
    lse = torch.full((B, Hq, 3), 9.0, device="cuda")
    score = torch.rand(B, Hkv, S, generator=g, device="cuda") * 1e-3
    lengths = torch.tensor([5000, 2500], device="cuda", dtype=torch.int32)

    def both():
        s = moda.cache_score(q, k, lse, lengths, score)
        return s, moda.cache_evict(k, v, s, lengths, keep, 4, 64)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s, r = both()
    for lens in ([5000, 2500], [300, 5000], [1, 0]):
        lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        ws, wr = both()
        torch.cuda.synchronize()
        for b, n in enumerate(lens):
            m = min(n, keep)
            assert torch.equal(s[b, :, :n], ws[b, :, :n])
            for name in ("k_out", "v_out", "score_out", "index"):
                assert torch.equal(r[name][b, :, :m], wr[name][b, :, :m])
        assert torch.equal(r["lengths_out"], wr["lengths_out"])
    moda.check_device_errors()
