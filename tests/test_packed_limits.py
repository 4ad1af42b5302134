"""Packed batches at the ends of what their bounds can say: more sequences than the kernels count,
and bounds that go back and forth, so that sequences overlap."""
import pytest
import torch

import depth_aware_attention_b200 as moda
from ragged_util import BF, LSE_BOUND, assert_close, joint_attention, randn

A = 1 << 24  # fake addresses 16 MiB apart, never dereferenced: the calls fail before a launch


@pytest.mark.parametrize("nseq,status", [((1 << 30) + 1, moda.MODA_ERR_UNSUPPORTED),
                                         ((1 << 31) - 1, moda.MODA_ERR_UNSUPPORTED),
                                         (-1, moda.MODA_ERR_INVALID_ARGUMENT)])
def test_more_sequences_than_are_counted(nseq, status):
    # (the loops over the sequences step by 32 in 32 bits)
    sizes = dict(Hq=4, Hkv=2, N=64, nseq=nseq, L=2, d=64, scale=0.125, causal=1, stream=None)
    ins = dict(q=A, k=A * 2, v=A * 3, kd=A * 4, vd=A * 5, cu_seqlens=A * 4000, out=A * 7, lse=A * 8)
    grads = dict(dout=A * 9, dq=A * 10, dk=A * 11, dv=A * 12, dkd=A * 13, dvd=A * 14,
                 workspace=A * 15, workspace_bytes=1 << 24)
    assert moda.moda_forward_packed(**ins, **sizes) == status
    assert moda.moda_backward_packed(**ins, **grads, **sizes) == status


@pytest.mark.gpu
@pytest.mark.parametrize("d,G,L", [(64, 1, 0), (128, 4, 3)])
@pytest.mark.parametrize("N,nseq", [(300, 9), (4000, 64), (700, 5000)])
def test_sequences_that_overlap(N, nseq, d, G, L):
    # 0, N, 0, N, ...: every other sequence is all rows, and they add up to many times N.  What is
    # computed of them is not said, but all of it stays in range, is reported, and a good call
    # after it is as it was.
    g = torch.Generator(device="cuda").manual_seed(N)
    q, dout = randn(g, G, N, d), randn(g, G, N, d)
    k, v = randn(g, 1, N, d), randn(g, 1, N, d)
    kd, vd = (randn(g, 1, N, L, d) if L else None for _ in range(2))
    one = torch.tensor([0, N], device="cuda", dtype=torch.int32)
    want = moda.forward_packed(q, k, v, one, kd, vd)
    cu = torch.zeros(nseq + 1, device="cuda", dtype=torch.int32)
    cu[1::2] = N
    out, lse = moda.forward_packed(q, k, v, cu, kd, vd)
    assert moda.moda_check_device_errors() == (moda.MODA_ERR_INTERNAL, 2)
    moda.backward_packed(q, k, v, cu, kd, vd, out, lse, dout)
    assert moda.moda_check_device_errors() == (moda.MODA_ERR_INTERNAL, 2)
    again = moda.forward_packed(q, k, v, one, kd, vd)
    moda.check_device_errors()
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])


@pytest.mark.gpu
def test_good_bounds_with_as_many_sequences():
    # the same number of sequences, all but one empty: as that one alone
    N, d, nseq = 700, 64, 1 << 15
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (randn(g, 1, N, d) for _ in range(3))
    cu = torch.full((nseq + 1,), N, device="cuda", dtype=torch.int32)
    cu[:1000] = 0
    out, lse = moda.forward_packed(q, k, v, cu)
    moda.check_device_errors()
    see = torch.ones(N, N, device="cuda", dtype=torch.bool).tril()
    r = joint_attention(q.double(), k[0].double(), v[0].double(), see, None, None, d ** -0.5)
    assert_close(out, r["out"], r["out_bound"], "out")
    assert_close(lse, r["lse"], LSE_BOUND, "lse")


@pytest.mark.gpu
@pytest.mark.parametrize("N", [127, 128, 255, 257])
@pytest.mark.parametrize("d,G,Hkv", [(128, 4, 64), (64, 2, 64), (64, 1, 75)])
def test_one_sequence_about_a_block_long_with_many_heads(N, d, G, Hkv):
    # around the counts of blocks at which CTAs share a walk, and tiles are cut smaller
    g = torch.Generator(device="cuda").manual_seed(N + d)
    q, dout = randn(g, G * Hkv, N, d), randn(g, G * Hkv, N, d)
    k, v = randn(g, Hkv, N, d), randn(g, Hkv, N, d)
    cu = torch.tensor([0, N], device="cuda", dtype=torch.int32)
    out, lse = moda.forward_packed(q, k, v, cu)
    grads = moda.backward_packed(q, k, v, cu, None, None, out, lse, dout)
    moda.check_device_errors()
    see = torch.ones(N, N, device="cuda", dtype=torch.bool).tril()
    for h in range(0, Hkv, 7):
        rows = slice(h * G, h * G + G)
        r = joint_attention(q[rows].double(), k[h].double(), v[h].double(), see, None, None,
                            d ** -0.5, dout[rows].double())
        assert_close(out[rows], r["out"], r["out_bound"], f"out {h}")
        assert_close(lse[rows], r["lse"], LSE_BOUND, f"lse {h}")
        assert_close(grads["dq"][rows], r["dq"], r["dq_bound"], f"dq {h}")
        assert_close(grads["dk"][h], r["dk"], r["dk_bound"], f"dk {h}")
        assert_close(grads["dv"][h], r["dv"], r["dv_bound"], f"dv {h}")
