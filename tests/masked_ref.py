"""Attention under any mask in fp64, with bounds on what the kernels may be off by.

For one set of rows: q [..., n, d], k, v [..., m, d], seen [..., n, m] (True where the row sees the key).
The bounds follow the kernels' roundings.  With u = eps / 2 of the 16-bit type (half a step):

  * a score's fp32 products and sums: ds <= scale (d + 2) 2^-24 sum_c |q_c k_c|, and a further 2^-22 |s| for the
    scaling to base 2 and the running reference (m, lse);
  * an unnormalised p: relative error e = ds + 4e-6 (the exponential: 3.6e-6 on the FMA pipe, less on the MUFU);
    normalised, numerator and denominator both: 2 e_max, e_max over the row's keys;
  * P and dS enter their products rounded to 16 bits (u); outputs are rounded once (u); sums of n terms in fp32
    add n 2^-24 of the terms' absolute values;
  * below the type's smallest normal value 2^-14 (fp16) the step no longer shrinks with the value: half a step is
    then 2^-14 2^-10 / 2 = 2^-25, an absolute term for every rounded P, dS and output (for bf16 it is 2^-134).
"""
import math

import torch


def u_of(dtype):
    return torch.finfo(dtype).eps / 2


class Ref:
    """Forward (and, with dout, backward) in fp64 on the tensors' device, and the bounds."""

    def __init__(self, q, k, v, seen, scale=None, dout=None):
        self.u = u_of(q.dtype)
        sub = torch.finfo(q.dtype).smallest_normal * self.u
        q, k, v = q.double(), k.double(), v.double()
        d, m = q.shape[-1], k.shape[-2]
        self.scale = scale = 1.0 / math.sqrt(d) if scale is None else scale
        seen = seen.expand(q.shape[:-1] + (m,))
        # what masked keys hold does not count
        any_seen = seen.flatten(0, -2).any(0) if k.dim() == 2 else seen.any(-2)
        k = torch.where(any_seen.unsqueeze(-1), k, 0.0)
        v = torch.where(any_seen.unsqueeze(-1), v, 0.0)
        s = torch.matmul(q, k.transpose(-1, -2)) * scale
        s = torch.where(seen, s, -math.inf)
        self.lse = torch.logsumexp(s, -1)
        base = torch.where(torch.isinf(self.lse), 0.0, self.lse).unsqueeze(-1)
        self.p = p = torch.where(seen, torch.exp(s - base), 0.0)
        self.o = torch.matmul(p, v)
        ds = torch.matmul(q.abs(), k.abs().transpose(-1, -2)) * (scale * (d + 2) * 2.0 ** -24)
        ds = torch.where(seen, ds + 2.0 ** -22 * s.abs().nan_to_num(0.0, posinf=0.0), 0.0)
        e = ds.amax(-1, keepdim=True) + 4e-6           # relative error of a p of the row
        small = m * 2.0 ** -24
        pv = torch.matmul(p, v.abs())
        # the kernels' unnormalised p = exp(s - m) is the normalised one times l >= 1 (the running reference m is
        # at most the row's largest score), so an absolute error of `sub` in it is at most `sub` in P
        pv_sub = sub * torch.matmul(seen.double(), v.abs())
        self.o_tol = self.u * self.o.abs() + (self.u + 2 * e + small) * pv * (1 + self.u) + pv_sub + sub
        # log2 of the sum: approximate to 2^-22 near 1, times ln 2; scaling back to natural units
        self.lse_tol = e.squeeze(-1) + small + 2.0 ** -22 * (1 + self.lse.abs().nan_to_num(0.0, posinf=0.0))
        self.w = p.sum(-2)
        n = q.shape[-2]
        self.w_tol = (p * (ds + self.lse_tol.unsqueeze(-1) + 4e-6 + n * 2.0 ** -24)).sum(-2) + 1e-30
        if dout is None:
            return
        do = dout.double()
        dp = torch.matmul(do, v.transpose(-1, -2))
        delta = (do * self.o).sum(-1, keepdim=True)
        g = p * (dp - delta)
        self.dq = torch.matmul(g, k) * scale
        self.dk = torch.matmul(g.transpose(-1, -2), q) * scale
        self.dv = torch.matmul(p.transpose(-1, -2), do)
        ep = ds + self.lse_tol.unsqueeze(-1) + 4e-6     # P from the saved lse
        ddp = torch.matmul(do.abs(), v.abs().transpose(-1, -2)) * (d * 2.0 ** -24)
        ddelta = (do.abs() * self.o_tol).sum(-1, keepdim=True) + (do.abs() * self.o.abs()).sum(-1, keepdim=True) * d * 2.0 ** -24
        dg = (self.u + ep) * g.abs() + p * (1 + ep) * (ddp + ddelta) + sub
        dg = torch.where(seen, dg, 0.0)
        acc_n, acc_m = n * 2.0 ** -24, m * 2.0 ** -24
        a = (self.u + 2.0 ** -23)
        self.dq_tol = a * self.dq.abs() + scale * torch.matmul(dg + acc_m * g.abs(), k.abs()) + sub
        self.dk_tol = a * self.dk.abs() + scale * torch.matmul((dg + acc_n * g.abs()).transpose(-1, -2), q.abs()) + sub
        self.dv_tol = a * self.dv.abs() + torch.matmul((p * (self.u + ep + acc_n) + sub * seen).transpose(-1, -2), do.abs()) + sub


def close(got, ref, tol, what):
    """got within tol of ref, element by element; infinities equal."""
    got = got.double().reshape(ref.shape)
    assert torch.isfinite(got[torch.isfinite(ref)]).all(), f"{what}: values that are not finite"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    if ref[~inf].numel():
        over = (got - ref).abs()[~inf] / tol.expand_as(ref)[~inf]
        assert over.max() <= 1.0, f"{what}: {over.max():.3f} of the bound, {int((over > 1).sum())} values over it"


def window_seen(nq, nk, window, sinks, device):
    """[nq, nk]: key j is seen from position x = i + nk - nq iff j <= x and (j > x - window or j < sinks)."""
    x = (torch.arange(nq, device=device) + nk - nq).unsqueeze(1)
    j = torch.arange(nk, device=device)
    return (j <= x) & ((j > x - window) | (j < sinks))
