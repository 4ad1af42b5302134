"""What is measured of the operators for ragged batches around mixture-of-depths attention.

Each in a plain form (elementary torch operations in 32 bits) and as the framework's own call:

  packed   attention over whole prompts of different lengths that lie one behind the other,
           each query seeing its own sequence's keys up to itself and its own depth entries
  train    the same forward and then its backward: all gradients for a given upstream one
  tree     attention of N drafted tokens per sequence, a tree given by parents, over a cache
           whose sequences have different lengths (N = 1: one new token per sequence)
  score    the attention weight that the newest N queries give to each cached key, summed
           over the queries and the heads of a group and added to the key's running score
  evict    the cache cut down to its `keep` best entries per KV head: the first `sinks`, the
           last `recent` and the highest scores of the rest, in their old order

`prepare` makes inputs from the seed, `run` is one pass, `exact` gives the same outputs from
the definition in 64 bits.  Lengths are a function of the case alone, so that `work` knows them.
"""
import math
import random

import numpy as np
import torch

own = False

BF = torch.bfloat16


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # a handful of short prompts that arrive together: latency
        dict(name="packed-short", op="packed", nseq=5, total=411, pad=13, Hq=16, Hkv=4, d=128,
             L=24, mix=1),
        # the longest prefill: six documents in 64K tokens
        dict(name="packed-64k", op="packed", nseq=6, total=65536, pad=0, Hq=16, Hkv=4, d=128,
             L=32, mix=3),
        # odd everything: groups of three heads, head size 64, one-token sequences
        dict(name="packed-odd-d64", op="packed", nseq=37, total=5003, pad=6, Hq=6, Hkv=2, d=64,
             L=7, mix=4),
        # a training step's attention: two dozen documents in 16K tokens, the 1.5B layer's shape
        dict(name="train-16k", op="train", nseq=24, total=16384, pad=0, Hq=16, Hkv=4, d=128,
             L=24, mix=2),
        # short odd documents, with rows behind the last one
        dict(name="train-odd-d64", op="train", nseq=11, total=2003, pad=9, Hq=6, Hkv=2, d=64,
             L=5, mix=13),
        # one new token per sequence over short caches: latency
        dict(name="tree-one-token", op="tree", B=4, N=1, S=1000, Hq=16, Hkv=4, d=128, L=24,
             mix=5),
        # one new token per sequence, a full batch of ragged caches
        dict(name="tree-batch32", op="tree", B=32, N=1, S=32768, Hq=16, Hkv=4, d=128, L=48,
             mix=6),
        # a wide tree over the longest caches, head layout of the deep stack
        dict(name="tree-61-drafts-64k", op="tree", B=2, N=61, S=65536, Hq=32, Hkv=8, d=128, L=32,
             mix=8),
        # scores after one decoding step over long caches
        dict(name="score-one-token", op="score", B=8, N=1, S=65536, Hq=16, Hkv=4, d=128, mix=9),
        # scores from a prompt's last 33 queries
        dict(name="score-window", op="score", B=2, N=33, S=5000, Hq=32, Hkv=8, d=64, mix=10),
        # long caches cut to an eighth
        dict(name="evict-64k", op="evict", B=4, S=65536, keep=8192, sinks=4, recent=512, Hkv=4,
             d=128, mix=11),
        # a small odd cache
        dict(name="evict-small", op="evict", B=2, S=2801, keep=1021, sinks=3, recent=65, Hkv=2,
             d=64, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["packed", "train", "tree", "score", "evict"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, Hkv=Hkv, d=d, mix=rng.randrange(1 << 20))
    if op in ("packed", "train"):
        total = _log(rng, 200, 30000 if op == "packed" else 8000)
        c.update(Hq=Hq, total=total, nseq=_log(rng, 1, min(200, total // 4)),
                 pad=rng.randrange(20), L=rng.choice([0, 1, 3, 8, 17, 24, 32]))
    elif op == "tree":
        S = _log(rng, 100, 65536)
        N = rng.choice([1, 1, 2, 5, 8, 13, 16, 31, 32, 64])
        c.update(Hq=Hq, N=N, S=S, L=rng.choice([0, 1, 3, 8, 17, 24, 48]),
                 B=_log(rng, 1, max(1, min(32, 4000000 // (S * Hkv)))))
    elif op == "score":
        S = _log(rng, 100, 65536)
        c.update(Hq=Hq, N=rng.choice([1, 1, 4, 16, 32, 63]), S=S,
                 B=_log(rng, 1, max(1, min(16, 4000000 // (S * Hkv)))))
    else:
        S = _log(rng, 200, 65536)
        keep = max(8, int(S * rng.uniform(0.05, 0.9)))
        sinks = min(rng.randrange(9), keep // 4)
        c.update(S=S, keep=keep, sinks=sinks, recent=rng.randrange(keep // 2),
                 B=_log(rng, 1, max(1, min(16, 4000000 // (S * Hkv)))))
    return c


def _lengths(c):
    """Sequence lengths of a case: a spread of a few long and many short ones."""
    r = random.Random(c["mix"])
    if c["op"] in ("packed", "train"):
        n, total = c["nseq"], c["total"]
        w = [math.exp(r.gauss(0.0, 1.0)) for _ in range(n)]
        lens = [int(total * x / sum(w)) for x in w]
        lens[0] += total - sum(lens)
        return lens
    return [max(1, int(c["S"] * (1.0 if b == 0 else r.uniform(0.3, 1.0)))) for b in range(c["B"])]


def _parents(c):
    """A drafted tree per sequence: parents before children, several children a node, and
    one slot in sixteen left unused (-2) where the tree is not full."""
    r = random.Random(c["mix"] + 1)
    rows = []
    for _ in range(c["B"]):
        p = []
        for i in range(c["N"]):
            live = [j for j in range(i) if p[j] != -2]
            if i and r.random() < 1 / 16:
                p.append(-2)
            else:
                p.append(r.choice(live[-8:] + [-1]) if live else -1)
        rows.append(p)
    return rows


# ---------------------------------------------------------------------------- inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=BF)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + c["mix"])
    lens = _lengths(c)
    s = dict(case=c, lens=lens, scale=1.0 / math.sqrt(c["d"]))
    Hkv, d = c["Hkv"], c["d"]
    zeros = lambda *shape, dtype: torch.zeros(*shape, device="cuda", dtype=dtype)  # noqa: E731
    if c["op"] in ("packed", "train"):
        n, L, Hq = c["total"] + c["pad"], c["L"], c["Hq"]
        s.update(q=_randn(g, Hq, n, d), k=_randn(g, Hkv, n, d), v=_randn(g, Hkv, n, d),
                 kd=_randn(g, Hkv, n, L, d) if L else None,
                 vd=_randn(g, Hkv, n, L, d) if L else None)
        ends = [0]
        for x in lens:
            ends.append(ends[-1] + x)
        s["cu"] = torch.tensor(ends, device="cuda", dtype=torch.int32)
        # rows behind the last sequence are left as they were: zeros here
        s["out"], s["lse"] = zeros(Hq, n, d, dtype=BF), zeros(Hq, n, dtype=torch.float32)
        if c["op"] == "train":
            s["dout"] = _randn(g, Hq, n, d)
            s["grads"] = {"d" + x: zeros(*s[x].shape, dtype=BF) for x in ("q", "k", "v")}
            if L:
                s["grads"].update({"d" + x: zeros(*s[x].shape, dtype=BF) for x in ("kd", "vd")})
        return s
    B, S = c["B"], c["S"]
    s["lengths"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s["k"] = _randn(g, B, Hkv, S, d)
    if c["op"] == "tree":
        N, L, Hq = c["N"], c["L"], c["Hq"]
        s.update(q=_randn(g, B, Hq, N, d), v=_randn(g, B, Hkv, S, d), kt=_randn(g, B, Hkv, N, d),
                 vt=_randn(g, B, Hkv, N, d), kd=_randn(g, B, Hkv, N, L, d) if L else None,
                 vd=_randn(g, B, Hkv, N, L, d) if L else None)
        s["parents"] = torch.tensor(_parents(c), device="cuda", dtype=torch.int32)
        return s
    if c["op"] == "score":
        N, Hq = c["N"], c["Hq"]
        s["q"] = _randn(g, B, Hq, N, d)
        s["score"] = torch.rand(B, Hkv, S, generator=g, device="cuda").pow(8)
        # the queries' own log-sum-exp, some of the weight being on depth entries
        lse = torch.empty(B, Hq, N, device="cuda")
        for b, x in enumerate(lens):
            z = (s["q"][b].float().view(Hkv, Hq // Hkv * N, d)
                 @ s["k"][b, :, :x].float().transpose(1, 2)) * s["scale"]
            lse[b] = torch.logsumexp(z, -1).view(Hq, N)
        s["lse"] = lse + 0.3 * torch.rand(B, Hq, N, generator=g, device="cuda")
        return s
    s["v"] = _randn(g, B, Hkv, S, d)
    # accumulated weights: few large, many small, and a share that is exactly zero (ties)
    w = torch.rand(B, Hkv, S, generator=g, device="cuda").pow(6)
    s["score"] = torch.where(w < 1e-3, torch.zeros_like(w), w)
    keep = c["keep"]
    s["outs"] = dict(k_out=zeros(B, Hkv, keep, d, dtype=BF), v_out=zeros(B, Hkv, keep, d, dtype=BF),
                     score_out=zeros(B, Hkv, keep, dtype=torch.float32),
                     index=zeros(B, Hkv, keep, dtype=torch.int32),
                     lengths_out=zeros(B, dtype=torch.int32))
    return s


# ---------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        import depth_aware_attention_b200 as moda
        if op in ("packed", "train"):
            x = [state[n] for n in ("q", "k", "v", "cu", "kd", "vd")]
            out, lse = moda.forward_packed(*x, out=state["out"], lse=state["lse"])
            if op == "packed":
                return out, lse
            grads = moda.backward_packed(*x, out, lse, state["dout"], grads=state["grads"])
            return out, lse, {n: grads[n] for n in state["grads"]}
        if op == "tree":
            return moda.tree_decode(state["q"], state["k"], state["v"], state["kt"], state["vt"],
                                    state["parents"], state["lengths"], state["kd"], state["vd"])
        if op == "score":
            return moda.cache_score(state["q"], state["k"], state["lse"], state["lengths"],
                                    state["score"])
        return moda.cache_evict(state["k"], state["v"], state["score"], state["lengths"],
                                state["case"]["keep"], state["case"]["sinks"],
                                state["case"]["recent"], **state["outs"])
    return {"packed": _packed, "train": _train, "tree": _tree, "score": _score, "evict": _evict}[op](state)


def _packed(s):
    c, scale = s["case"], s["scale"]
    Hq, Hkv, d, L = c["Hq"], c["Hkv"], c["d"], c["L"]
    G = Hq // Hkv
    n = s["q"].shape[1]
    out = torch.zeros(Hq, n, d, device="cuda", dtype=BF)
    lse = torch.zeros(Hq, n, device="cuda")
    first = 0
    for x in s["lens"]:
        k, v = s["k"][:, first:first + x].float(), s["v"][:, first:first + x].float()
        for a in range(0, x, 2048):
            b = min(x, a + 2048)
            q = s["q"][:, first + a:first + b].float().view(Hkv, G, b - a, d)
            z = torch.einsum("hgtd,hsd->hgts", q, k[:, :b]) * scale
            t = torch.arange(a, b, device="cuda")
            z = z.masked_fill(torch.arange(b, device="cuda")[None, :] > t[:, None], -math.inf)
            top = z.amax(-1, keepdim=True)
            if L:
                kd = s["kd"][:, first + a:first + b].float()
                y = torch.einsum("hgtd,htld->hgtl", q, kd) * scale
                top = torch.maximum(top, y.amax(-1, keepdim=True))
            p = torch.exp(z - top)
            total = p.sum(-1, keepdim=True)
            o = torch.einsum("hgts,hsd->hgtd", p, v[:, :b])
            if L:
                py = torch.exp(y - top)
                total = total + py.sum(-1, keepdim=True)
                o = o + torch.einsum("hgtl,htld->hgtd", py, s["vd"][:, first + a:first + b].float())
            out[:, first + a:first + b] = (o / total).reshape(Hq, b - a, d).to(BF)
            lse[:, first + a:first + b] = (top + torch.log(total)).reshape(Hq, b - a)
        first += x
    return out, lse


def _train(s):
    c, scale = s["case"], s["scale"]
    Hq, Hkv, d, L = c["Hq"], c["Hkv"], c["d"], c["L"]
    G = Hq // Hkv
    out, lse = _packed(s)
    dq, dk, dv = (torch.zeros(s[x].shape, device="cuda") for x in ("q", "k", "v"))
    dkd, dvd = (torch.zeros(s[x].shape, device="cuda", dtype=BF) if L else None
                for x in ("kd", "vd"))
    first = 0
    for x in s["lens"]:
        for a in range(0, x, 2048):
            b = min(x, a + 2048)
            row, key = slice(first + a, first + b), slice(first, first + b)
            q, do = (s[n][:, row].float().view(Hkv, G, b - a, d) for n in ("q", "dout"))
            k, v = s["k"][:, key].float(), s["v"][:, key].float()
            z = torch.einsum("hgtd,hsd->hgts", q, k) * scale
            t = torch.arange(a, b, device="cuda")
            z = z.masked_fill(torch.arange(b, device="cuda")[None, :] > t[:, None], -math.inf)
            top = lse[:, row].view(Hkv, G, b - a, 1)
            p = torch.exp(z - top)
            o = torch.einsum("hgts,hsd->hgtd", p, v)
            if L:
                kd, vd = s["kd"][:, row].float(), s["vd"][:, row].float()
                py = torch.exp(torch.einsum("hgtd,htld->hgtl", q, kd) * scale - top)
                o = o + torch.einsum("hgtl,htld->hgtd", py, vd)
            whole = (o * do).sum(-1, keepdim=True)
            ds = p * (torch.einsum("hgtd,hsd->hgts", do, v) - whole) * scale
            g = torch.einsum("hgts,hsd->hgtd", ds, k)
            dk[:, key] += torch.einsum("hgts,hgtd->hsd", ds, q)
            dv[:, key] += torch.einsum("hgts,hgtd->hsd", p, do)
            if L:
                dy = py * (torch.einsum("hgtd,htld->hgtl", do, vd) - whole) * scale
                g = g + torch.einsum("hgtl,htld->hgtd", dy, kd)
                dkd[:, row] = torch.einsum("hgtl,hgtd->htld", dy, q).to(BF)
                dvd[:, row] = torch.einsum("hgtl,hgtd->htld", py, do).to(BF)
            dq[:, row] = g.reshape(Hq, b - a, d)
        first += x
    grads = dict(dq=dq.to(BF), dk=dk.to(BF), dv=dv.to(BF))
    if L:
        grads.update(dkd=dkd, dvd=dvd)
    return out, lse, grads


def _ancestors(parents):
    """[B, N, N] truth values: j is i itself or an ancestor of i.  Unused slots see nothing."""
    B, N = parents.shape
    step = torch.zeros(B, N, N + 1, device=parents.device)
    step.scatter_(2, torch.where(parents < 0, N, parents).long()[..., None], 1.0)
    reach = step[:, :, :N] + torch.eye(N, device=parents.device)
    for _ in range(max(1, (N - 1).bit_length())):
        reach = ((reach @ reach) > 0).float()
    return (reach > 0) & (parents != -2)[:, :, None] & (parents != -2)[:, None, :]


def _tree(s):
    c, scale = s["case"], s["scale"]
    B, N, S, Hq, Hkv, d, L = (c[x] for x in ("B", "N", "S", "Hq", "Hkv", "d", "L"))
    G = Hq // Hkv
    q = s["q"].float().view(B, Hkv, G, N, d)
    live = (s["parents"] != -2)[:, None, None, :, None]
    z = torch.einsum("bhgnd,bhsd->bhgns", q, s["k"].float()) * scale
    see = torch.arange(S, device="cuda")[None, :] < s["lengths"][:, None]
    z = z.masked_fill(~see[:, None, None, None, :], -math.inf)
    zt = torch.einsum("bhgnd,bhmd->bhgnm", q, s["kt"].float()) * scale
    zt = zt.masked_fill(~_ancestors(s["parents"])[:, None, None], -math.inf)
    top = torch.maximum(z.amax(-1, keepdim=True), zt.amax(-1, keepdim=True))
    if L:
        y = torch.einsum("bhgnd,bhnld->bhgnl", q, s["kd"].float()) * scale
        top = torch.maximum(top, y.amax(-1, keepdim=True))
    p, pt = torch.exp(z - top), torch.exp(zt - top)
    total = p.sum(-1, keepdim=True) + pt.sum(-1, keepdim=True)
    o = (torch.einsum("bhgns,bhsd->bhgnd", p, s["v"].float())
         + torch.einsum("bhgnm,bhmd->bhgnd", pt, s["vt"].float()))
    if L:
        py = torch.exp(y - top)
        total = total + py.sum(-1, keepdim=True)
        o = o + torch.einsum("bhgnl,bhnld->bhgnd", py, s["vd"].float())
    out = torch.where(live, o / total, torch.zeros_like(o))
    lse = torch.where(live, top + torch.log(total), torch.full_like(total, -math.inf))
    return out.view(B, Hq, N, d).to(BF), lse.view(B, Hq, N)


def _score(s):
    c, scale = s["case"], s["scale"]
    B, N, S, Hq, Hkv, d = (c[x] for x in ("B", "N", "S", "Hq", "Hkv", "d"))
    G = Hq // Hkv
    z = torch.einsum("bhgnd,bhsd->bhgns", s["q"].float().view(B, Hkv, G, N, d), s["k"].float())
    w = torch.exp(z * scale - s["lse"].view(B, Hkv, G, N, 1))
    pos = s["lengths"][:, None] - N + torch.arange(N, device="cuda")[None, :]
    see = torch.arange(S, device="cuda")[None, None, :] <= pos[:, :, None]
    return s["score"] + w.masked_fill(~see[:, None, None], 0.0).sum((2, 3))


def _evict(s):
    c = s["case"]
    B, S, Hkv, d, keep = (c[x] for x in ("B", "S", "Hkv", "d", "keep"))
    lens = s["lengths"].long()
    at = torch.arange(S, device="cuda")
    safe = (at < c["sinks"]) | (at >= lens[:, None] - c["recent"])
    rank = s["score"].masked_fill(safe[:, None], math.inf)
    rank = rank.masked_fill((at >= lens[:, None])[:, None], -math.inf)
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    left = torch.clamp(lens, max=keep)
    got = torch.arange(keep, device="cuda") < left[:, None]  # [B, keep]
    index = torch.sort(best.masked_fill(~got[:, None], S), dim=-1).values
    index = index.masked_fill(~got[:, None], 0)
    rows = index[..., None].expand(B, Hkv, keep, d)
    none = ~got[:, None, :, None]
    return dict(k_out=torch.gather(s["k"], 2, rows).masked_fill(none, 0.0),
                v_out=torch.gather(s["v"], 2, rows).masked_fill(none, 0.0),
                score_out=torch.gather(s["score"], 2, index).masked_fill(~got[:, None], 0.0),
                index=index.int(), lengths_out=left.int())


# ---------------------------------------------------------------------------- work
def work(case):
    c, lens = case, _lengths(case)
    Hkv, d = c["Hkv"], c["d"]
    tokens = sum(lens)
    if c["op"] in ("packed", "train"):
        Hq, L = c["Hq"], c["L"]
        pairs = sum(x * (x + 1) // 2 for x in lens) + tokens * L
        both = c["op"] == "train"  # dout in, every gradient out; ten more products than four
        return dict(bytes=tokens * (Hq * (4 * d + 4) + Hkv * 4 * d * (1 + L)
                                    + (Hq * 4 * d + Hkv * 4 * d * (1 + L) if both else 0)),
                    flops=(14 if both else 4) * Hq * d * pairs)
    if c["op"] == "tree":
        Hq, L, N, B = c["Hq"], c["L"], c["N"], c["B"]
        pairs = N * tokens + B * N * (L + (N + 1) / 2)
        return dict(bytes=Hkv * 4 * d * (tokens + B * N * (1 + L)) + B * N * Hq * (4 * d + 4),
                    flops=4 * Hq * d * pairs)
    if c["op"] == "score":
        return dict(bytes=Hkv * tokens * (2 * d + 8) + c["B"] * c["N"] * c["Hq"] * (2 * d + 4),
                    flops=2 * c["Hq"] * c["N"] * d * tokens)
    kept = sum(min(x, c["keep"]) for x in lens)
    return dict(bytes=Hkv * (4 * tokens + kept * (8 * d + 8)), flops=0)


# ---------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"packed": _exact_packed, "train": _exact_train, "tree": _exact_tree, "score": _exact_score,
            "evict": _exact_evict}[case["op"]](s)


def _softmax_row_block(logits, values):
    """Joint softmax of several [..., rows, keys] blocks over their values, in 64 bits."""
    z = torch.cat(logits, -1)
    lse = torch.logsumexp(z, -1)
    out = 0.0
    for y, v in zip(logits, values):  # v: [keys, d], or [rows, keys, d]
        w = torch.exp(y - lse[..., None])
        out = out + ((w[..., None] * v).sum(-2) if v.dim() > w.dim() else w @ v)
    return out, lse


def _exact_packed(s):
    c = s["case"]
    G, L, d = c["Hq"] // c["Hkv"], c["L"], c["d"]
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.zeros(s["q"].shape[:2], device="cuda", dtype=torch.float64)
    ends = s["cu"].tolist()
    for a, e in zip(ends[:-1], ends[1:]):
        for g in range(c["Hkv"]):
            key, val = s["k"][g, a:e].double(), s["v"][g, a:e].double()
            for t in range(a, e, 1024):
                u = min(e, t + 1024)
                hide = torch.ones(u - t, u - a, device="cuda").triu(t - a + 1).bool()
                for h in range(g * G, g * G + G):
                    q = s["q"][h, t:u].double() * s["scale"]
                    z = (q @ key[:u - a].T).masked_fill(hide, -math.inf)
                    logits, values = [z], [val[:u - a]]
                    if L:
                        logits.append((s["kd"][g, t:u].double() @ q[..., None])[..., 0])
                        values.append(s["vd"][g, t:u].double())
                    out[h, t:u], lse[h, t:u] = _softmax_row_block(logits, values)
    return out, lse


def _exact_train(s):
    c = s["case"]
    G, L = c["Hq"] // c["Hkv"], c["L"]
    names = ("q", "k", "v") + (("kd", "vd") if L else ())
    grads = {"d" + n: torch.zeros(s[n].shape, device="cuda", dtype=torch.float64) for n in names}
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.zeros(s["q"].shape[:2], device="cuda", dtype=torch.float64)
    ends = s["cu"].tolist()
    for a, e in zip(ends[:-1], ends[1:]):
        hide = torch.ones(e - a, e - a, device="cuda").triu(1).bool()
        for g in range(c["Hkv"] if e > a else 0):
            leaf = {n: s[n][g, a:e].double().requires_grad_() for n in names[1:]}
            for h in range(g * G, g * G + G):
                q = s["q"][h, a:e].double().requires_grad_()
                logits = [(q @ leaf["k"].T * s["scale"]).masked_fill(hide, -math.inf)]
                values = [leaf["v"]]
                if L:
                    logits.append((leaf["kd"] @ q[..., None])[..., 0] * s["scale"])
                    values.append(leaf["vd"])
                o, lse_h = _softmax_row_block(logits, values)
                (o * s["dout"][h, a:e].double()).sum().backward()
                out[h, a:e], lse[h, a:e] = o.detach(), lse_h.detach()
                grads["dq"][h, a:e] = q.grad
            for n, x in leaf.items():
                grads["d" + n][g, a:e] = x.grad
    return out, lse, grads


def _exact_tree(s):
    c = s["case"]
    G, N, L = c["Hq"] // c["Hkv"], c["N"], c["L"]
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full(s["q"].shape[:3], -math.inf, device="cuda", dtype=torch.float64)
    for b, x in enumerate(s["lens"]):
        parents = s["parents"][b].tolist()
        path = np.zeros((N, N), dtype=bool)
        for i, p in enumerate(parents):
            if p != -2:
                path[i] = path[p] if p >= 0 else False
                path[i, i] = True
        rows = [i for i in range(N) if parents[i] != -2]
        hide = torch.from_numpy(~path).cuda()[rows]
        for h in range(c["Hq"]):
            g = h // G
            q = s["q"][b, h, rows].double() * s["scale"]
            logits = [q @ s["k"][b, g, :x].double().T,
                      (q @ s["kt"][b, g].double().T).masked_fill(hide, -math.inf)]
            values = [s["v"][b, g, :x].double(), s["vt"][b, g].double()]
            if L:
                logits.append((s["kd"][b, g, rows].double() @ q[..., None])[..., 0])
                values.append(s["vd"][b, g, rows].double())
            out[b, h, rows], lse[b, h, rows] = _softmax_row_block(logits, values)
    return out, lse


def _exact_score(s):
    c = s["case"]
    G, N = c["Hq"] // c["Hkv"], c["N"]
    total = s["score"].double().clone()
    for b, x in enumerate(s["lens"]):
        for h in range(c["Hq"]):
            key = s["k"][b, h // G, :x].double()
            for i in range(N):
                end = x - N + i + 1
                if end > 0:
                    w = torch.exp(key[:end] @ s["q"][b, h, i].double() * s["scale"]
                                  - s["lse"][b, h, i].double())
                    total[b, h // G, :end] += w
    return total


def _exact_evict(s):
    c = s["case"]
    B, Hkv, keep, d = c["B"], c["Hkv"], c["keep"], c["d"]
    score = s["score"].cpu().numpy().astype(np.float64)
    k, v = s["k"].double().cpu().numpy(), s["v"].double().cpu().numpy()
    r = dict(k_out=np.zeros((B, Hkv, keep, d)), v_out=np.zeros((B, Hkv, keep, d)),
             score_out=np.zeros((B, Hkv, keep)), index=np.zeros((B, Hkv, keep), np.int32),
             lengths_out=np.array([min(x, keep) for x in s["lens"]], np.int32))
    for b, x in enumerate(s["lens"]):
        n = min(x, keep)
        for g in range(Hkv):
            must = np.zeros(x, dtype=bool)
            must[:c["sinks"]] = True
            must[max(0, x - c["recent"]):] = True
            order = np.lexsort((np.arange(x), -score[b, g, :x], ~must))
            at = np.sort(order[:n])
            r["index"][b, g, :n] = at
            r["k_out"][b, g, :n], r["v_out"][b, g, :n] = k[b, g, at], v[b, g, at]
            r["score_out"][b, g, :n] = score[b, g, at]
    return r
