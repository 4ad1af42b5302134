"""The ragged-batch entry points refuse bad calls before anything is launched (CPU only).

At the C ABI the addresses are fake and never dereferenced: on a machine with a GPU a call with
valid arguments would launch a kernel on them, so every call here must fail an argument check
(or, where there is no GPU, the injected launch failure).  At the torch wrappers CPU tensors
with consistent metadata get as far as the device check.
"""
import pytest
import torch

import depth_aware_attention_b200 as moda

A = 1 << 24  # fake addresses 16 MiB apart
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
BAD, NO = moda.MODA_ERR_INVALID_ARGUMENT, moda.MODA_ERR_UNSUPPORTED

FORWARD = dict(q=A, k=A * 2, v=A * 3, kd=A * 4, vd=A * 5, cu_seqlens=A * 6, out=A * 7, lse=A * 8,
               Hq=4, Hkv=2, N=64, nseq=3, L=2, d=64, scale=0.125, causal=1, stream=None)
BACKWARD = dict(q=A, k=A * 2, v=A * 3, kd=A * 4, vd=A * 5, cu_seqlens=A * 6, out=A * 7, lse=A * 8,
                dout=A * 9, dq=A * 10, dk=A * 11, dv=A * 12, dkd=A * 13, dvd=A * 14,
                workspace=A * 15, workspace_bytes=1 << 24, Hq=4, Hkv=2, N=64, nseq=3, L=2, d=64,
                scale=0.125, causal=1, stream=None)
TREE = dict(q=A, k=A * 2, v=A * 3, kt=A * 4, vt=A * 5, kd=A * 6, vd=A * 7, parents=A * 8,
            lengths=A * 9, out=A * 10, lse=A * 11, workspace=A * 16, workspace_bytes=1 << 28, B=2,
            Hq=4, Hkv=2, S=100, N=8, L=2, d=64, scale=0.125, stream=None)
SCORE = dict(q=A, k=A * 2, lse=A * 3, lengths=A * 4, score=A * 5, score_out=A * 6, B=2, Hq=4,
             Hkv=2, S=100, N=8, d=64, scale=0.125, stream=None)
EVICT = dict(k=A, v=A * 2, score=A * 3, lengths=A * 4, k_out=A * 5, v_out=A * 6, score_out=A * 7,
             index=A * 8, lengths_out=A * 9, B=2, Hkv=2, S=100, keep=20, sinks=2, recent=5, d=64,
             stream=None)
CALLS = {"moda_forward_packed": FORWARD, "moda_backward_packed": BACKWARD,
         "moda_tree_decode": TREE, "moda_cache_score": SCORE, "moda_cache_evict": EVICT}

NAN, INF = float("nan"), float("inf")
REFUSED = [
    ("moda_forward_packed", dict(N=0), BAD), ("moda_forward_packed", dict(nseq=0), BAD),
    ("moda_forward_packed", dict(Hq=3), BAD), ("moda_forward_packed", dict(L=-1), BAD),
    ("moda_forward_packed", dict(d=96), NO), ("moda_forward_packed", dict(Hq=130, Hkv=1), NO),
    ("moda_forward_packed", dict(cu_seqlens=None), BAD),
    ("moda_forward_packed", dict(cu_seqlens=A * 6 + 2), BAD),
    ("moda_forward_packed", dict(kd=None), BAD), ("moda_forward_packed", dict(q=A + 8), BAD),
    ("moda_forward_packed", dict(scale=0.0), BAD), ("moda_forward_packed", dict(scale=-1.0), BAD),
    ("moda_forward_packed", dict(scale=NAN), BAD), ("moda_forward_packed", dict(scale=INF), BAD),
    ("moda_forward_packed", dict(out=A * 2), BAD),  # out over k
    ("moda_forward_packed", dict(cu_seqlens=A * 7 + 64), BAD),  # out over cu_seqlens
    ("moda_forward_packed", dict(N=(1 << 30) + 1), NO),
    ("moda_forward_packed", dict(Hkv=2, Hq=2, N=1 << 30, nseq=1 << 30), NO),
    ("moda_backward_packed", dict(N=0), BAD), ("moda_backward_packed", dict(nseq=0), BAD),
    ("moda_backward_packed", dict(cu_seqlens=None), BAD),
    ("moda_backward_packed", dict(dq=None), BAD), ("moda_backward_packed", dict(dvd=None), BAD),
    ("moda_backward_packed", dict(workspace_bytes=1000), BAD),
    ("moda_backward_packed", dict(workspace=A * 15 + 16), BAD),
    ("moda_backward_packed", dict(scale=0.0), BAD), ("moda_backward_packed", dict(scale=INF), BAD),
    ("moda_backward_packed", dict(dk=A * 3), BAD),  # dk over v
    ("moda_backward_packed", dict(cu_seqlens=A * 12 + 64), BAD),  # dv over cu_seqlens
    ("moda_backward_packed", dict(dkd=A * 10), BAD),  # dkd over dq
    ("moda_tree_decode", dict(B=0), BAD), ("moda_tree_decode", dict(S=0), BAD),
    ("moda_tree_decode", dict(N=0), BAD), ("moda_tree_decode", dict(N=129), NO),
    ("moda_tree_decode", dict(Hq=5), BAD), ("moda_tree_decode", dict(d=32), NO),
    ("moda_tree_decode", dict(Hq=130, Hkv=2), NO), ("moda_tree_decode", dict(L=65536), NO),
    ("moda_tree_decode", dict(B=70000, Hkv=1), NO), ("moda_tree_decode", dict(kt=None), BAD),
    ("moda_tree_decode", dict(vd=None), BAD), ("moda_tree_decode", dict(parents=None), BAD),
    ("moda_tree_decode", dict(lengths=A * 9 + 1), BAD), ("moda_tree_decode", dict(k=A * 2 + 8), BAD),
    ("moda_tree_decode", dict(workspace_bytes=64), BAD),
    ("moda_tree_decode", dict(workspace=None), BAD),
    ("moda_tree_decode", dict(workspace=A * 16 + 128), BAD),
    ("moda_tree_decode", dict(scale=0.0), BAD), ("moda_tree_decode", dict(scale=INF), BAD),
    ("moda_tree_decode", dict(out=A * 4), BAD), ("moda_tree_decode", dict(lse=A * 10), BAD),
    ("moda_cache_score", dict(S=0), BAD), ("moda_cache_score", dict(N=200), NO),
    ("moda_cache_score", dict(d=80), NO), ("moda_cache_score", dict(q=None), BAD),
    ("moda_cache_score", dict(lse=None), BAD), ("moda_cache_score", dict(score=None), BAD),
    ("moda_cache_score", dict(score=None, score_out=None), BAD),
    ("moda_cache_score", dict(score_out=A * 5 + 64), BAD),  # overlaps score, but is not score
    ("moda_cache_score", dict(score_out=A * 2), BAD), ("moda_cache_score", dict(scale=-0.5), BAD),
    ("moda_cache_evict", dict(keep=0), BAD), ("moda_cache_evict", dict(sinks=-1), BAD),
    ("moda_cache_evict", dict(recent=-1), BAD), ("moda_cache_evict", dict(recent=19), BAD),
    ("moda_cache_evict", dict(keep=20, sinks=1 << 30, recent=1 << 30), BAD),
    ("moda_cache_evict", dict(d=96), NO), ("moda_cache_evict", dict(k_out=A), BAD),  # in place
    ("moda_cache_evict", dict(lengths_out=A * 4), BAD), ("moda_cache_evict", dict(index=None), BAD),
    ("moda_cache_evict", dict(v_out=A * 6 + 8), BAD), ("moda_cache_evict", dict(score=None), BAD),
]


@pytest.mark.parametrize("name,change,status", REFUSED,
                         ids=[f"{n[5:]}-{i}" for i, (n, _, _) in enumerate(REFUSED)])
def test_c_entry_points_refuse(name, change, status):
    assert getattr(moda, name)(**{**CALLS[name], **change}) == status
    assert moda.moda_last_error_message()


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses: CPU-only test")
@pytest.mark.parametrize("name", sorted(CALLS))
def test_fault_injection(name, monkeypatch):
    monkeypatch.setenv("MODA_FAULT_INJECT", "validate")
    assert getattr(moda, name)(**CALLS[name]) == BAD
    assert "MODA_FAULT_INJECT=validate" in moda.moda_last_error_message()
    monkeypatch.setenv("MODA_FAULT_INJECT", "launch")
    assert getattr(moda, name)(**CALLS[name]) == moda.MODA_ERR_CUDA
    assert "MODA_FAULT_INJECT=launch" in moda.moda_last_error_message()


def test_workspace_sizes():
    size = moda.moda_tree_decode_workspace_size
    assert size(2, 16, 4, 1000, 1, 24, 128) > 0
    assert size(2, 16, 4, 1000, 0, 24, 128) == 0 and size(2, 16, 5, 1000, 1, 24, 128) == 0
    # it depends on the rows of a tile, not on the cache or the batch
    assert size(1, 16, 4, 1000, 8, 0, 128) == size(64, 16, 4, 65536, 8, 48, 128)


# ------------------------------------------------------------------------------- torch wrappers
def _t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


B, Hq, Hkv, N, S, L, d = 2, 4, 2, 6, 40, 3, 64


def wrappers():
    p = dict(q=_t(Hq, S, d), k=_t(Hkv, S, d), v=_t(Hkv, S, d), cu_seqlens=_t(4, dtype=I32),
             kd=_t(Hkv, S, L, d), vd=_t(Hkv, S, L, d))
    return {
        "forward_packed": p,
        "backward_packed": dict(p, out=_t(Hq, S, d), lse=_t(Hq, S, dtype=F32), dout=_t(Hq, S, d)),
        "tree_decode": dict(q=_t(B, Hq, N, d), k=_t(B, Hkv, S, d), v=_t(B, Hkv, S, d),
                            kt=_t(B, Hkv, N, d), vt=_t(B, Hkv, N, d), parents=_t(B, N, dtype=I32),
                            lengths=_t(B, dtype=I32), kd=_t(B, Hkv, N, L, d),
                            vd=_t(B, Hkv, N, L, d)),
        "cache_score": dict(q=_t(B, Hq, N, d), k=_t(B, Hkv, S, d), lse=_t(B, Hq, N, dtype=F32),
                            lengths=_t(B, dtype=I32), score=_t(B, Hkv, S, dtype=F32)),
        "cache_evict": dict(k=_t(B, Hkv, S, d), v=_t(B, Hkv, S, d),
                            score=_t(B, Hkv, S, dtype=F32), lengths=_t(B, dtype=I32), keep=10),
    }


@pytest.mark.parametrize("name", sorted(wrappers()))
def test_consistent_cpu_tensors_stop_at_the_device_check(name):
    with pytest.raises(ValueError, match="runs on CUDA tensors"):
        getattr(moda, name)(**wrappers()[name])


@pytest.mark.parametrize("name,change,err,match", [
    ("forward_packed", dict(k=_t(Hkv, S - 1, d)), ValueError, "k has shape"),
    ("forward_packed", dict(cu_seqlens=_t(4, dtype=torch.int64)), TypeError, "cu_seqlens has dtype"),
    ("forward_packed", dict(cu_seqlens=_t(1, dtype=I32)), ValueError, "nseq"),
    ("forward_packed", dict(q=_t(1, Hq, S, d)), ValueError, "q must be a 3-D tensor"),
    ("forward_packed", dict(vd=None), ValueError, "vd is required"),
    ("forward_packed", dict(v=_t(Hkv, d, S).transpose(1, 2)), ValueError, "v must be contiguous"),
    ("forward_packed", dict(out=_t(Hq, S + 1, d)), ValueError, "out has shape"),
    ("backward_packed", dict(lse=_t(Hq, S)), TypeError, "lse has dtype"),
    ("backward_packed", dict(grads=dict(dk=_t(Hkv, S + 1, d))), ValueError, "dk has shape"),
    ("backward_packed", dict(dout=_t(Hq, S, d, dtype=F32)), TypeError, "dout has dtype"),
    ("tree_decode", dict(kt=_t(B, Hkv, N + 1, d)), ValueError, "kt has shape"),
    ("tree_decode", dict(parents=_t(B, N + 1, dtype=I32)), ValueError, "parents has shape"),
    ("tree_decode", dict(lengths=_t(B, dtype=torch.int64)), TypeError, "lengths has dtype"),
    ("tree_decode", dict(kd=_t(B, Hkv, N, d)), ValueError, "kd must be a 5-D tensor"),
    ("tree_decode", dict(workspace=torch.zeros(64, dtype=torch.uint8, device="meta")), ValueError,
     "workspace must be"),
    ("cache_score", dict(lse=_t(B, Hq, N + 1, dtype=F32)), ValueError, "lse has shape"),
    ("cache_score", dict(score=_t(B, Hkv, S)), TypeError, "score has dtype"),
    ("cache_score", dict(out=_t(B, Hkv, S + 1, dtype=F32)), ValueError, "out has shape"),
    ("cache_evict", dict(keep=0), ValueError, "keep must be"),
    ("cache_evict", dict(v=_t(B, Hkv, S + 1, d)), ValueError, "v has shape"),
    ("cache_evict", dict(index=_t(B, Hkv, 10, dtype=torch.int64)), TypeError, "index has dtype"),
])
def test_wrappers_refuse(name, change, err, match):
    with pytest.raises(err, match=match):
        getattr(moda, name)(**{**wrappers()[name], **change})
