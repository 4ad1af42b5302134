"""Shared helpers of the ragged-batch tests: the operators written out in 64 bits, and error
bounds derived from the roundings the kernels make.

Rounding to bf16 is off by at most U = 2^-8 of the value (finfo(bf16).eps / 2), taken as
uniform in +-U: variance U^2 / 3 relative to the value.  The kernels round, in the forward,
each softmax weight P to bf16 before its product with V (the normaliser sums unrounded
weights), and in the backward P and dS; the backward also takes its row term D = <dO, out>
from the rounded out.  The errors of different terms are independent, so an element's error
has the variance of the sum of its terms' errors, and SIGMAS standard deviations bound every
one of up to 10^7 elements (6 sigma: 2e-9 each).  On top come
  - half a step of the output's own type,
  - FP32 relative to the sum of the absolute terms, for the fp32 sums, the exponentials
    (2^-22 by the exponent unit, 7.5e-5 for a quarter of them by polynomial) and the
    products' fp32 accumulation.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8
SIGMAS = 6.0
FP32 = 1e-4
BF = torch.bfloat16


def rounded_bound(var, terms, value, out_u=U):
    """Bound of one output: 6 sigma of its terms' roundings, the fp32 part, its own step."""
    return SIGMAS * torch.sqrt(var) + FP32 * terms + out_u * value.abs() + 1e-6


def assert_close(got, ref, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    over = (got - ref).abs() - bound
    assert (over <= 0).all(), (
        f"{what}: error {(got - ref).abs().max().item():.3e}, worst excess over its bound "
        f"{over.max().item():.3e} at {tuple(int(i) for i in (over == over.max()).nonzero()[0])}")


def joint_attention(q, k, v, see, kd, vd, scale, dout=None):
    """q [H,T,d] (one KV head's group), k/v [S,d], see [T,S] truth values, kd/vd [T,L,d] or
    None, all in 64 bits.  Rows that see nothing give out 0 and lse -inf.  Returns a dict of
    out, lse and their bounds, and with dout of the gradients and theirs."""
    z = (q @ k.T * scale).masked_fill(~see, -math.inf)
    y = None if kd is None else torch.einsum("htd,tld->htl", q, kd) * scale
    lse = torch.logsumexp(z if y is None else torch.cat([z, y], -1), -1)
    safe = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None]
    p = torch.exp(z - safe)
    out, var, tot = p @ v, (p ** 2) @ (v ** 2), p @ v.abs()
    if y is not None:
        py = torch.exp(y - safe)
        out = out + torch.einsum("htl,tld->htd", py, vd)
        var = var + torch.einsum("htl,tld->htd", py ** 2, vd ** 2)
        tot = tot + torch.einsum("htl,tld->htd", py, vd.abs())
    r = dict(out=out, lse=lse, out_bound=rounded_bound(var * U * U / 3, tot, out))
    if dout is None:
        return r
    D = (dout * out).sum(-1, keepdim=True)
    # variance of D from out's rounding, one error per row
    dvar = ((U * dout * out) ** 2).sum(-1, keepdim=True) / 3
    ds = p * (dout @ v.T - D) * scale
    # fp32 errors of D and of the products: relative to their own sums of absolute terms
    dabs = p * ((dout.abs() @ v.abs().T) + (dout * out).abs().sum(-1, keepdim=True)) * scale
    dq, qvar, qtot = ds @ k, (ds ** 2) @ (k ** 2), dabs @ k.abs()
    qshift = (p * scale) @ k
    if y is not None:
        dy = py * (torch.einsum("htd,tld->htl", dout, vd) - D) * scale
        dyabs = py * (torch.einsum("htd,tld->htl", dout.abs(), vd.abs())
                      + (dout * out).abs().sum(-1, keepdim=True)) * scale
        dq = dq + torch.einsum("htl,tld->htd", dy, kd)
        qtot = qtot + torch.einsum("htl,tld->htd", dyabs, kd.abs())
        qshift = qshift + torch.einsum("htl,tld->htd", py * scale, kd)
        r.update(dkd=torch.einsum("htl,htd->tld", dy, q),
                 dvd=torch.einsum("htl,htd->tld", py, dout))
        # (the depth gradients' P and dS stay in fp32; D's shift remains)
        sv = torch.einsum("htl,htd->tld", (py * scale) ** 2 * dvar, q ** 2)
        r["dkd_bound"] = rounded_bound(sv, torch.einsum("htl,htd->tld", dyabs, q.abs()), r["dkd"])
        r["dvd_bound"] = rounded_bound(torch.zeros_like(sv),
                                       torch.einsum("htl,htd->tld", py, dout.abs()), r["dvd"])
    r["dq"] = dq
    r["dq_bound"] = rounded_bound(qvar * U * U / 3 + qshift ** 2 * dvar, qtot, dq)
    r["dk"] = torch.einsum("hts,htd->sd", ds, q)
    kvar = torch.einsum("hts,htd->sd", (U * ds) ** 2 / 3 + (p * scale) ** 2 * dvar, q ** 2)
    r["dk_bound"] = rounded_bound(kvar, torch.einsum("hts,htd->sd", dabs, q.abs()), r["dk"])
    r["dv"] = torch.einsum("hts,htd->sd", p, dout)
    vvar = torch.einsum("hts,htd->sd", (U * p) ** 2 / 3, dout ** 2)
    r["dv_bound"] = rounded_bound(vvar, torch.einsum("hts,htd->sd", p, dout.abs()), r["dv"])
    return r


# lse: fp32 sums of weights whose relative error is at most FP32, then a logarithm; the
# logits are fp32 sums of exact products (error below 2^-20 of sum |q k| scale, < 1e-4 here)
LSE_BOUND = 3e-4


def randn(gen, *shape, device="cuda"):
    return torch.randn(*shape, generator=gen, device=device).to(BF)
