"""The running softmax where scores grow along the keys, by jumps that move every row's reference.

The kernels keep a reference per row and let it move only when a score exceeds it by 2^8; then the
accumulator and the sum, which hold something by then, are rescaled.  Inputs of unit normals hardly
ever do that.  Here one key in four blocks of 128 exceeds all before it by 2^9 to 2^11, for each of
the two warpgroups that may share the blocks between them; the keys before it are as many at the
level of the last such one, so that what was summed before a jump keeps a weight of a seventh or
more: a factor left out, or applied to the sum or the accumulator alone, shows.
Depth entries come before, between or after the keys, in steps of their own.

`test_a_rescale_left_out_shows` runs a blockwise softmax with each such mistake on the CPU and
holds it against the same bounds.
"""
import math

import pytest
import torch

import depth_aware_attention_b200 as moda
import ragged_util
from ragged_util import BF, LSE_BOUND, assert_close, joint_attention, randn

JUMP = 9.5  # log2 units between levels
LOG2E = math.log2(math.e)


def levels(S):
    """Level of each key, in log2 units: the blocks of 128 keys in groups of four, a level each, and
    in the third and the fourth block of a group one key on the next level."""
    block = torch.arange(S) // 128
    lv = (block // 4).double() * JUMP
    for b in range(S // 128 + 1):
        at = 128 * b + 13 * b % 41
        if b % 4 >= 2 and at < S:
            lv[at] += JUMP
    return lv


def keys(gen, lv, d, *lead):
    """Keys [*lead, S, d] whose score with a query along the ones vector is lv (log2 units)."""
    dev = gen.device
    k = 0.25 * torch.randn(*lead, len(lv), d, generator=gen, device=dev)
    return (k + (lv.to(dev) / (LOG2E * math.sqrt(d)))[:, None]).to(BF)


def queries(gen, d, *lead):
    """Queries [*lead, d] near the ones vector, their lengths 0.95 to 1.15 of it."""
    dev = gen.device
    size = 0.95 + 0.2 * torch.rand(*lead, 1, generator=gen, device=dev)
    return (size * (1 + 0.05 * torch.randn(*lead, d, generator=gen, device=dev))).to(BF)


def logit_error(q, k, scale):
    """Bound of a logit's error: its fp32 sum of products is within 2^-20 of the sum of their
    absolute values, and the product with scale and the subtraction of the reference within 2^-23
    of its size.  (q and k of one KV head, any leading axes.)"""
    a, b = q.double().abs().reshape(-1, q.shape[-1]), k.double().abs().reshape(-1, k.shape[-1])
    return (2.0 ** -20 + 2.0 ** -23) * scale * (a.amax(0) * b.amax(0)).sum().item()


def use_error(monkeypatch, eps):
    """The bounds' fp32 share for logits with error eps: a weight's relative error is that of its
    logit and of lse, which is another eps at most."""
    monkeypatch.setattr(ragged_util, "FP32", 1e-4 + 2 * eps)
    return LSE_BOUND + eps


# ----------------------------------------------------------------------------- on the CPU
def blockwise(q, k, v, scale, mistake):
    """Softmax over 128-key blocks with a reference that moves past 2^8 only, with a mistake."""
    z = q @ k.T * scale * LOG2E
    m = torch.full(z.shape[:1], -math.inf, dtype=torch.float64)
    o, l, moved = torch.zeros(len(z), v.shape[1], dtype=torch.float64), torch.zeros(len(z)), 0
    for s in range(0, len(k), 128):
        x = z[:, s:s + 128]
        top = torch.maximum(m, x.amax(-1))
        new = torch.where(top > m + 8, top, m)
        f = torch.exp2(m - new)
        moved += int(((new > m) & (l > 0)).sum())
        p = torch.exp2(x - new[:, None])
        o = o * (1 if mistake in ("o", "both") else f[:, None]) + p @ v[s:s + 128]
        l = l * (1 if mistake in ("l", "both") else f) + p.sum(-1)
        if mistake == "dropped":
            o, l = torch.where((f < 1)[:, None], p @ v[s:s + 128], o), torch.where(f < 1, p.sum(-1), l)
        m = new
    return o / l[:, None], (m + torch.log2(l)) / LOG2E, moved


@pytest.mark.parametrize("mistake", ["none", "o", "l", "both", "dropped"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_rescale_left_out_shows(d, mistake, monkeypatch):
    g = torch.Generator().manual_seed(d)
    S, H = 1500, 6
    q, k = queries(g, d, H, 1), keys(g, levels(S), d)
    v = torch.randn(S, d, generator=g).to(BF)
    scale = 1 / math.sqrt(d)
    lse_bound = use_error(monkeypatch, logit_error(q, k, scale))
    see = torch.ones(1, S, dtype=torch.bool)
    r = joint_attention(q.double(), k.double(), v.double(), see, None, None, scale)
    out, lse, moved = blockwise(q[:, 0].double(), k.double(), v.double(), scale, mistake)
    assert moved == 3 * H  # 12 blocks, three levels
    wrong = ((out - r["out"][:, 0]).abs() > r["out_bound"][:, 0]).any(-1)
    off = (lse - r["lse"][:, 0]).abs() > lse_bound
    assert not (wrong | off).any() if mistake == "none" else wrong.all()


# ----------------------------------------------------------------------------- on the GPU
# name, lengths, S, N, Hq, Hkv, d, L, depth level of the first and of the last entry
TREES = [
    # few rows (4 and 16 a tile), transposed products; shares of 8 to 20 steps
    ("rows-1", [2600] * 8 + [1300, 900], 2600, 1, 8, 8, 128, 9, 0, 2),
    ("rows-4", [3000] * 10 + [130, 0], 3000, 1, 32, 8, 128, 24, 0, 0),
    ("rows-4-depth-high", [2000] * 10 + [0], 2000, 2, 16, 8, 128, 300, 0, 5),
    ("rows-16", [2700] * 9 + [255], 2700, 4, 32, 8, 128, 70, 0, 2),
    ("rows-15", [2500] * 9, 2500, 5, 24, 8, 128, 0, 0, 0),
    # one full tile; a pair of tiles
    ("tile-32", [2600] * 9 + [77], 2600, 8, 32, 8, 128, 40, 0, 3),
    ("tile-d64", [2800] * 9, 2800, 13, 16, 8, 64, 24, 0, 2),
    ("tile-128", [2600] * 8, 2600, 128, 8, 8, 64, 3, 0, 1),
    ("pair-d128", [2200] * 8 + [300], 2200, 40, 32, 8, 128, 24, 0, 4),
    ("pair-d64", [2200] * 8, 2200, 61, 24, 8, 64, 12, 0, 3),
    ("pairs-two", [1900] * 6, 1900, 100, 32, 8, 64, 2, 0, 1),
    # one step less than a CTA's share, cut items of a few long caches
    ("long-cut", [4000, 3900], 4000, 20, 4, 1, 128, 8, 0, 2),
    ("long-cut-few", [4000, 3900, 1], 4000, 1, 4, 1, 128, 8, 0, 2),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", TREES, ids=[c[0] for c in TREES])
def test_tree(case, monkeypatch):
    _, lens, S, N, Hq, Hkv, d, L, lo, hi = case
    B, G, scale = len(lens), Hq // Hkv, 1 / math.sqrt(d)
    g = torch.Generator(device="cuda").manual_seed(N + S)
    q = queries(g, d, B, Hq, N)
    # the drafted tokens' own keys lie between the depth entries and the cache
    k = keys(g, levels(S) + (hi + 1) * JUMP, d, B, Hkv)
    kt = keys(g, torch.full((N,), (hi + 0.5) * JUMP), d, B, Hkv)
    v, vt = randn(g, B, Hkv, S, d), randn(g, B, Hkv, N, d)
    kd = vd = None
    if L:
        lv = (torch.arange(L) * (hi - lo + 1) // L + lo).double() * JUMP
        kd, vd = keys(g, lv, d, B, Hkv, N), randn(g, B, Hkv, N, L, d)
    parents = torch.arange(-1, N - 1, device="cuda", dtype=torch.int32).repeat(B, 1)
    lengths = torch.tensor(lens, device="cuda", dtype=torch.int32)
    out, lse = moda.tree_decode(q, k, v, kt, vt, parents, lengths, kd, vd)
    moda.check_device_errors()
    line = torch.ones(N, N, device="cuda", dtype=torch.bool).tril()
    for b, n in enumerate(lens):
        see = torch.cat([torch.ones(N, n, device="cuda", dtype=torch.bool), line], 1)
        for h in range(Hkv):
            rows = slice(h * G, h * G + G)
            kk, vv = torch.cat([k[b, h, :n], kt[b, h]]), torch.cat([v[b, h, :n], vt[b, h]])
            lse_bound = use_error(monkeypatch, logit_error(q[b, rows], kk, scale))
            r = joint_attention(q[b, rows].double(), kk.double(), vv.double(), see,
                                kd[b, h].double() if L else None,
                                vd[b, h].double() if L else None, scale)
            assert_close(out[b, rows], r["out"], r["out_bound"], f"out {b} {h}")
            assert_close(lse[b, rows], r["lse"], lse_bound, f"lse {b} {h}")


# name, lengths, Hq, Hkv, d, L, causal; depth entries at the level `depth` of the keys' last
PACKED = [
    ("prompt-single-d128", [1300, 700], 8, 1, 128, 9, True, 0.0),
    ("prompt-single-d64", [900, 1, 400], 4, 1, 64, 0, True, 0.0),
    ("prompt-single-full", [1000, 129], 4, 1, 128, 3, False, 0.5),
    ("prompt-pair-g3", [2600, 2300, 2200], 6, 2, 128, 24, True, 0.0),
    ("prompt-pair-g3-d64", [3000, 2800, 1500], 6, 2, 64, 5, False, 0.6),
    ("forward-d128", [3100, 1300], 8, 2, 128, 24, True, 0.0),
    ("forward-d128-depth-high", [2900, 1500], 8, 2, 128, 24, True, 0.7),
    ("forward-d64", [2600, 1900, 130], 8, 4, 64, 9, True, 0.3),
    ("forward-full-d64", [2600, 1300], 8, 2, 64, 0, False, 0.0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", PACKED, ids=[c[0] for c in PACKED])
def test_packed(case, monkeypatch):
    _, lens, Hq, Hkv, d, L, causal, depth = case
    N, G, scale = sum(lens), Hq // Hkv, 1 / math.sqrt(d)
    g = torch.Generator(device="cuda").manual_seed(N + d)
    lv = torch.cat([levels(n) for n in lens])
    q, k, v, dout = queries(g, d, Hq, N), keys(g, lv, d, Hkv), randn(g, Hkv, N, d), randn(g, Hq, N, d)
    kd = vd = None
    if L:  # rising from entry to entry; at most `depth` of the way up to the token's own level
        up = depth * lv.max() * torch.arange(1, L + 1) / L
        kd, vd = keys(g, up, d, Hkv, N), randn(g, Hkv, N, L, d)
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    cu = torch.tensor(ends, device="cuda", dtype=torch.int32)
    out, lse = moda.forward_packed(q, k, v, cu, kd, vd, causal=causal)
    grads = moda.backward_packed(q, k, v, cu, kd, vd, out, lse, dout, causal=causal)
    moda.check_device_errors()
    for a, e in zip(ends[:-1], ends[1:]):
        see = torch.ones(e - a, e - a, device="cuda", dtype=torch.bool)
        see = see.tril() if causal else see
        for h in range(Hkv):
            rows = slice(h * G, h * G + G)
            lse_bound = use_error(monkeypatch, logit_error(q[rows, a:e], k[h, a:e], scale))
            r = joint_attention(q[rows, a:e].double(), k[h, a:e].double(), v[h, a:e].double(), see,
                                kd[h, a:e].double() if L else None,
                                vd[h, a:e].double() if L else None, scale,
                                dout[rows, a:e].double())
            assert_close(out[rows, a:e], r["out"], r["out_bound"], f"out {a} {h}")
            assert_close(lse[rows, a:e], r["lse"], lse_bound, f"lse {a} {h}")
            assert_close(grads["dq"][rows, a:e], r["dq"], r["dq_bound"], f"dq {a} {h}")
            for n in ("dk", "dv") + (("dkd", "dvd") if L else ()):
                assert_close(grads[n][h, a:e], r[n], r[n + "_bound"], f"{n} {a} {h}")


@pytest.mark.gpu
@pytest.mark.parametrize("N,Hq,Hkv,d", [(1, 8, 2, 128), (1, 4, 4, 64), (33, 8, 2, 64),
                                        (64, 8, 2, 128), (128, 8, 2, 128)])
def test_scores(N, Hq, Hkv, d):
    lens, S = [3000, 700, 129], 3000
    B, G, scale = len(lens), Hq // Hkv, 1 / math.sqrt(d)
    g = torch.Generator(device="cuda").manual_seed(N + d)
    q, k = queries(g, d, B, Hq, N), keys(g, levels(S), d, B, Hkv)
    score = torch.rand(B, Hkv, S, generator=g, device="cuda")
    lse, ref, added = torch.zeros(B, Hq, N, device="cuda"), score.double(), torch.zeros(B, Hkv, S)
    added = added.double().cuda()
    eps = max(logit_error(q[b], k[b], scale) for b in range(B))
    for b, n in enumerate(lens):
        see = torch.arange(n, device="cuda") <= torch.arange(n - N, n, device="cuda")[:, None]
        for h in range(Hq):
            z = (q[b, h].double() @ k[b, h // G, :n].double().T * scale).masked_fill(~see, -math.inf)
            lse[b, h] = torch.logsumexp(z, -1).float()
            w = torch.exp(z - lse[b, h].double()[:, None])
            added[b, h // G, :n] += torch.where(see, w, 0.0).nan_to_num(0.0).sum(0)
    lengths = torch.tensor(lens, device="cuda", dtype=torch.int32)
    lse = torch.where(lse.isfinite(), lse, -math.inf)
    got = moda.cache_score(q, k, lse, lengths, score).double()
    moda.check_device_errors()
    # weights within 1e-4 and their logits' error; fp32 sums of G * N weights and the old score
    bound = (1e-4 + eps) * added + G * N * 2.0 ** -24 * (ref + added) + 1e-12
    assert ((got - ref - added).abs() <= bound).all(), ((got - ref - added).abs() - bound).max()
