"""The ragged-batch operators on tensors of more than 2^31 elements, where an offset held in 32 bits
would wrap: caches of 1.1 million keys and more than a million packed tokens.  The last rows, which lie
behind the border, are held against 64 bits."""
import math

import pytest
import torch

import depth_aware_attention_b200 as moda
from ragged_util import BF, LSE_BOUND, assert_close, joint_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=BF)


def test_caches():
    B, Hkv, G, S, d, keep = 2, 8, 2, 1_100_003, 128, 1_060_007
    assert B * Hkv * keep * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = randn(g, B, Hkv, S, d), randn(g, B, Hkv, S, d)
    lengths = torch.tensor([5, S - 1], device="cuda", dtype=torch.int32)
    for N in (1, 40):  # the few-row form, a full tile
        q, kt, vt = randn(g, B, Hkv * G, N, d), randn(g, B, Hkv, N, d), randn(g, B, Hkv, N, d)
        line = torch.arange(-1, N - 1, device="cuda", dtype=torch.int32).repeat(B, 1)
        out, lse = moda.tree_decode(q, k, v, kt, vt, line, lengths)
        moda.check_device_errors()
        for b, h in ((0, Hkv - 1), (1, 0), (1, Hkv - 1)):
            n, rows = int(lengths[b]), slice(G * h, G * h + G)
            see = torch.cat([torch.ones(N, n, device="cuda", dtype=torch.bool),
                             torch.ones(N, N, device="cuda", dtype=torch.bool).tril()], 1)
            r = joint_attention(q[b, rows].double(), torch.cat([k[b, h, :n], kt[b, h]]).double(),
                                torch.cat([v[b, h, :n], vt[b, h]]).double(), see, None, None,
                                1 / math.sqrt(d))
            assert_close(out[b, rows], r["out"], r["out_bound"], f"out N={N} {b} {h}")
            assert_close(lse[b, rows], r["lse"], LSE_BOUND, f"lse N={N} {b} {h}")
    # scores of the newest token, then the eviction
    q, b, h = randn(g, B, Hkv * G, 1, d), 1, Hkv - 1
    n, rows = S - 1, slice(G * h, G * h + G)
    z = q[b, rows, 0].double() @ k[b, h, :n].double().T / math.sqrt(d)
    lse = torch.full((B, Hkv * G, 1), 14.0, device="cuda")
    score = torch.rand(B, Hkv, S, generator=g, device="cuda")
    new = moda.cache_score(q, k, lse, lengths, score)
    moda.check_device_errors()
    added = torch.exp(z - 14.0).sum(0)
    err = (new[b, h, :n].double() - score[b, h, :n].double() - added).abs()
    assert (err <= 1e-4 * added + 8 * 2.0 ** -24 * (1 + added)).all()
    assert torch.equal(new[b, h, n:], score[b, h, n:])
    r = moda.cache_evict(k, v, new, lengths, keep, sinks=4, recent=512)
    moda.check_device_errors()
    assert r["lengths_out"].tolist() == [5, keep]
    key = new[b, h, :n].clone()
    key[:4] = key[n - 512:] = math.inf
    want = torch.sort(key, descending=True, stable=True).indices[:keep].sort().values
    assert torch.equal(r["index"][b, h].long(), want)
    assert torch.equal(r["k_out"][b, h], k[b, h, want]) and torch.equal(r["v_out"][b, h], v[b, h, want])
    assert torch.equal(r["score_out"][b, h], new[b, h, want])


@pytest.mark.parametrize("d,Hq,Hkv,L", [(128, 16, 4, 4), (64, 24, 8, 4)])
def test_packed(d, Hq, Hkv, L):
    N = 1 + 2 ** 31 // (d * min(Hq, Hkv * L))
    g = torch.Generator(device="cuda").manual_seed(d)
    ends = list(range(0, N - 1500, 1009)) + [N - 3]
    q, dout, k, v = (randn(g, H, N, d) for H in (Hq, Hq, Hkv, Hkv))
    kd, vd = randn(g, Hkv, N, L, d), randn(g, Hkv, N, L, d)
    cu = torch.tensor(ends, device="cuda", dtype=torch.int32)
    out, lse = moda.forward_packed(q, k, v, cu, kd, vd)
    grads = moda.backward_packed(q, k, v, cu, kd, vd, out, lse, dout)
    moda.check_device_errors()
    G = Hq // Hkv
    for s, h in ((0, 0), (len(ends) // 2, Hkv - 1), (len(ends) - 2, 0), (len(ends) - 2, Hkv - 1)):
        a, e, rows = ends[s], ends[s + 1], slice(h * G, h * G + G)
        see = torch.ones(e - a, e - a, device="cuda", dtype=torch.bool).tril()
        r = joint_attention(q[rows, a:e].double(), k[h, a:e].double(), v[h, a:e].double(), see,
                            kd[h, a:e].double(), vd[h, a:e].double(), 1 / math.sqrt(d),
                            dout[rows, a:e].double())
        assert_close(out[rows, a:e], r["out"], r["out_bound"], f"out {a} {h}")
        assert_close(lse[rows, a:e], r["lse"], LSE_BOUND, f"lse {a} {h}")
        assert_close(grads["dq"][rows, a:e], r["dq"], r["dq_bound"], f"dq {a} {h}")
        for n in ("dk", "dv", "dkd", "dvd"):
            assert_close(grads[n][h, a:e], r[n], r[n + "_bound"], f"{n} {a} {h}")
