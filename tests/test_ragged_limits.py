"""The ragged-batch operators at their edges: nothing to do, one of everything, very many
sequences, captured and replayed training steps, calls from several threads and streams."""
import math
import threading

import pytest
import torch

import depth_aware_attention_b200 as moda
from ragged_util import BF, LSE_BOUND, assert_close, joint_attention, randn

pytestmark = pytest.mark.gpu


def ints(*v):
    return torch.tensor(v, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("cu", [[0, 0], [5, 5, 5], [0, 0, 0, 0, 0], [7, 7]])
def test_no_tokens_at_all(cu):
    g = torch.Generator(device="cuda").manual_seed(1)
    N, Hq, Hkv, d, L = 7, 4, 1, 64, 2
    x = [randn(g, Hq, N, d), randn(g, Hkv, N, d), randn(g, Hkv, N, d), ints(*cu),
         randn(g, Hkv, N, L, d), randn(g, Hkv, N, L, d)]
    out, lse = torch.full_like(x[0], 3.0), torch.full((Hq, N), 3.0, device="cuda")
    moda.forward_packed(*x, out=out, lse=lse)
    grads = {"d" + n: torch.full_like(t, 3.0) for n, t in
             zip(("q", "k", "v", "kd", "vd"), x[:3] + x[4:])}
    moda.backward_packed(*x, out, lse, torch.randn_like(x[0]), grads=grads)
    moda.check_device_errors()
    assert (out == 3).all() and (lse == 3).all()
    assert all((t == 3).all() for t in grads.values())


@pytest.mark.parametrize("d", [64, 128])
def test_one_of_everything(d):
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = randn(g, 1, 1, d), randn(g, 1, 1, d), randn(g, 1, 1, d)
    out, lse = moda.forward_packed(q, k, v, ints(0, 1))
    assert torch.equal(out, v)  # one visible key: its value
    z = (q.double() * k.double()).sum() / math.sqrt(d)
    assert (lse.double() - z).abs().max() <= LSE_BOUND
    r = moda.backward_packed(q, k, v, ints(0, 1), None, None, out, lse, torch.ones_like(q))
    # dv = dout exactly; the softmax of one key has no slope: dS = P (dP - D) is the rounding of
    # D alone, |D - dP| <= d * U * |v|, times scale and the other factor
    assert torch.equal(r["dv"], torch.ones_like(v))
    slack = d * 2.0 ** -8 * v.double().abs().max() / math.sqrt(d)
    assert r["dq"].double().abs().max() <= slack * k.double().abs().max() + 1e-6
    assert r["dk"].double().abs().max() <= slack * q.double().abs().max() + 1e-6
    o2, l2 = moda.tree_decode(q[None], k[None], v[None], k[None], v[None], ints(-1)[None], ints(0))
    assert torch.equal(o2[0], v) and (l2.double() - z).abs().max() <= LSE_BOUND
    s = moda.cache_score(q[None], k[None], l2, ints(1), torch.zeros(1, 1, 1, device="cuda"))
    assert (s - 1).abs().max() <= 1e-3
    e = moda.cache_evict(k[None], v[None], s, ints(1), 1)
    assert torch.equal(e["k_out"], k[None]) and e["index"].item() == 0
    moda.check_device_errors()


def test_empty_caches():
    g = torch.Generator(device="cuda").manual_seed(3)
    B, Hq, Hkv, S, N, d, L = 3, 8, 2, 50, 4, 128, 2
    k = torch.full((B, Hkv, S, d), float("nan"), device="cuda", dtype=BF)
    q, kt, vt = randn(g, B, Hq, N, d), randn(g, B, Hkv, N, d), randn(g, B, Hkv, N, d)
    kd, vd = randn(g, B, Hkv, N, L, d), randn(g, B, Hkv, N, L, d)
    zero, line = ints(0, 0, 0), ints(-1, 0, 1, 2).repeat(B, 1)
    out, lse = moda.tree_decode(q, k, k, kt, vt, line, zero, kd, vd)
    moda.check_device_errors()
    see = torch.ones(N, N, device="cuda", dtype=torch.bool).tril()
    for b in range(B):
        for h in range(Hkv):
            r = joint_attention(q[b, 4 * h:4 * h + 4].double(), kt[b, h].double(),
                                vt[b, h].double(), see, kd[b, h].double(), vd[b, h].double(),
                                1 / math.sqrt(d))
            assert_close(out[b, 4 * h:4 * h + 4], r["out"], r["out_bound"], "empty cache")
    score = torch.rand(B, Hkv, S, generator=g, device="cuda")
    assert torch.equal(moda.cache_score(q, k, lse, zero, score), score)
    r = moda.cache_evict(k, k, score, zero, 8, index=torch.full((B, Hkv, 8), 9, device="cuda",
                                                               dtype=torch.int32))
    moda.check_device_errors()
    assert r["lengths_out"].tolist() == [0, 0, 0] and (r["index"] == 9).all()


@pytest.mark.parametrize("d,Hq,Hkv,L", [(128, 4, 1, 3), (64, 3, 1, 2), (128, 2, 2, 0)])
def test_thousands_of_sequences(d, Hq, Hkv, L):
    # lengths 0 to 6, more sequences than a CTA's item list or a warp's registers hold
    lens = [(5 * i * i + i) % 7 for i in range(6000)]
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    N = ends[-1]
    g = torch.Generator(device="cuda").manual_seed(d + L)
    q, k, v = randn(g, Hq, N, d), randn(g, Hkv, N, d), randn(g, Hkv, N, d)
    kd, vd = (randn(g, Hkv, N, L, d) if L else None for _ in range(2))
    dout = randn(g, Hq, N, d)
    out, lse = moda.forward_packed(q, k, v, ints(*ends), kd, vd)
    grads = moda.backward_packed(q, k, v, ints(*ends), kd, vd, out, lse, dout)
    moda.check_device_errors()
    G = Hq // Hkv
    for a, e in [(x, y) for x, y in zip(ends[:-1], ends[1:]) if y > x][::97]:
        see = torch.ones(e - a, e - a, device="cuda", dtype=torch.bool).tril()
        for h in range(Hkv):
            rows = slice(h * G, h * G + G)
            r = joint_attention(q[rows, a:e].double(), k[h, a:e].double(), v[h, a:e].double(), see,
                                kd[h, a:e].double() if L else None,
                                vd[h, a:e].double() if L else None, 1 / math.sqrt(d),
                                dout[rows, a:e].double())
            assert_close(out[rows, a:e], r["out"], r["out_bound"], f"out [{a},{e})")
            assert_close(grads["dq"][rows, a:e], r["dq"], r["dq_bound"], f"dq [{a},{e})")
            for n in ("dk", "dv") + (("dkd", "dvd") if L else ()):
                assert_close(grads[n][h, a:e], r[n], r[n + "_bound"], f"{n} [{a},{e})")


@pytest.mark.parametrize("d", [64, 128])
def test_captured_training_step(d):
    # forward and backward in one graph; replayed on new inputs, lengths and gradients while the
    # eager results of the same tensors are alive
    Hq, Hkv, L, N = 8, 2, 4, 400
    g = torch.Generator(device="cuda").manual_seed(d)
    x = dict(q=randn(g, Hq, N, d), k=randn(g, Hkv, N, d), v=randn(g, Hkv, N, d),
             cu=ints(0, 100, 330, 400), kd=randn(g, Hkv, N, L, d), vd=randn(g, Hkv, N, L, d))
    dout = randn(g, Hq, N, d)

    def step():
        out, lse = moda.forward_packed(*x.values())
        return out, lse, moda.backward_packed(*x.values(), out, lse, dout)

    first = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, grads = step()
    for cu in ([0, 100, 330, 400], [0, 7, 8, 400], [0, 390, 390, 400]):
        for n in ("q", "kd", "v"):
            x[n].copy_(randn(g, *x[n].shape))
        x["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        graph.replay()
        o, ls, gr = step()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(ls, lse)
        for n in gr:  # dq, dk, dv are summed in the order of arrival: their last bits may differ
            a, b = gr[n].float(), grads[n].float()
            if n in ("dkd", "dvd"):
                assert torch.equal(a, b), n
            else:
                # two fp32 sums of the same terms, each then rounded to bf16: one step apart
                assert ((a - b).abs() <= 2.0 ** -7 * a.abs().clamp(min=1e-3)).all(), n
    moda.check_device_errors()
    del first


def test_calls_from_several_threads_and_streams():
    g = torch.Generator(device="cuda").manual_seed(4)
    jobs = []
    for i, (S, keep) in enumerate([(500, 100), (30000, 4000), (9000, 50), (150000, 20000)]):
        k, v = randn(g, 1, 2, S, 64), randn(g, 1, 2, S, 64)
        score = torch.rand(1, 2, S, generator=g, device="cuda")
        q, kt, vt = randn(g, 1, 8, 5, 64), randn(g, 1, 2, 5, 64), randn(g, 1, 2, 5, 64)
        jobs.append((k, v, score, q, kt, vt, ints(S - i), keep))
    line = ints(-1, 0, 0, 1, 2)[None]

    def run(job):
        k, v, score, q, kt, vt, lengths, keep = job
        out, lse = moda.tree_decode(q, k, v, kt, vt, line, lengths)
        new = moda.cache_score(q, k, lse, lengths, score)
        return (out, lse, new, moda.cache_evict(k, v, new, lengths, keep, 4, 16))

    want = [run(j) for j in jobs]
    torch.cuda.synchronize()
    got, errors = [None] * len(jobs), []

    def worker(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[i] = run(jobs[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 (reported by the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    moda.check_device_errors()
    assert not errors
    for w, r, job in zip(want, got, jobs):
        n = int(job[6])
        assert torch.equal(w[0], r[0]) and torch.equal(w[1], r[1])
        assert torch.equal(w[2][..., :n], r[2][..., :n])
        for name in ("k_out", "v_out", "score_out", "index", "lengths_out"):
            assert torch.equal(w[3][name], r[3][name]), name


def test_more_items_than_ctas():
    # 3 x 60 KV heads of short caches, and their trees: pieces that begin and end inside a CTA
    B, Hkv, G, S, N, d = 3, 60, 2, 333, 3, 64
    g = torch.Generator(device="cuda").manual_seed(6)
    k, v = randn(g, B, Hkv, S, d), randn(g, B, Hkv, S, d)
    q, kt, vt = randn(g, B, Hkv * G, N, d), randn(g, B, Hkv, N, d), randn(g, B, Hkv, N, d)
    lens = [333, 1, 129]
    out, lse = moda.tree_decode(q, k, v, kt, vt, ints(-1, 0, 0).repeat(B, 1), ints(*lens))
    moda.check_device_errors()
    see = torch.tensor([[1, 0, 0], [1, 1, 0], [1, 0, 1]], device="cuda", dtype=torch.bool)
    for b, n in enumerate(lens):
        all_see = torch.cat([torch.ones(N, n, device="cuda", dtype=torch.bool), see], 1)
        for h in range(Hkv):
            r = joint_attention(q[b, G * h:G * h + G].double(),
                                torch.cat([k[b, h, :n], kt[b, h]]).double(),
                                torch.cat([v[b, h, :n], vt[b, h]]).double(), all_see, None, None,
                                1 / math.sqrt(d))
            assert_close(out[b, G * h:G * h + G], r["out"], r["out_bound"], f"{b} {h}")
            assert_close(lse[b, G * h:G * h + G], r["lse"], LSE_BOUND, f"lse {b} {h}")
