"""The definition of attention over given keys in 64 bits, with its gradients and, beside each result, how far the
kernels may be from it.

The bounds count the kernels' roundings (u = 2^-8 is bf16's half step, relative):
  O    each weight P is rounded to bf16 before P V (u), the row's sum is not, and O is rounded once (u):
       u sum_j p_ij |v_j| + u |o_i|.
  P    before that rounding: scores are fp32 sums of d products (at most d 2^-24 sum |q k| scale, 1.1e-4 for d = 128 and
       N(0,1) inputs), the exponential is at most 8.6e-5 off (one pair in eight; 2^-22 otherwise) and LSE carries the same
       again: rho = 2^-11 in all, relative; LSE itself, absolute: rho.
  dV   sum_i p_ij (u + rho) |do_i| + u |dv_j|.
  dS   = p (dP - D): its rounding u |dS|, rho |dS|, and D_i = do_i . o_i taken from the bf16 O:
       p_ij sum_c |do_ic| e_ic with e the error of O above; fp32 sums of dP and D: p_ij 2^-15 sum |do v|.
  dQ   scale sum_j e(dS_ij) |k_j| + u |dq_i|;   dK   scale sum_i e(dS_ij) |q_i| + u |dk_j|.
"""
import math

import torch

U = 2.0 ** -8
RHO = 2.0 ** -11


def attend(q, k, v, scale, do=None, z=None):
    """q, do [I, Hq, d], k, v [J, Hkv, d] -> dict name -> (value, bound), 64 bits; z [Hq]: learned sink logits."""
    q, k, v = q.double(), k.double(), v.double()
    I, Hq, d = q.shape
    J, Hkv, _ = k.shape
    g = Hq // Hkv
    kk, vv = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    s = torch.einsum("ihd,jhd->hij", q, kk) * scale
    if z is not None:
        s = torch.cat([s, z.double()[:, None, None].expand(Hq, I, 1)], -1)
    if s.shape[-1] == 0:
        s = torch.full((Hq, I, 1), -math.inf, dtype=torch.float64)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isfinite(lse), lse, 0.0)[..., None])[..., :J]
    o = torch.einsum("hij,jhd->ihd", p, vv)
    e_o = 1.01 * (U + RHO) * torch.einsum("hij,jhd->ihd", p, vv.abs()) + U * o.abs() + 1e-6
    out = {"o": (o, e_o), "lse": (lse, torch.full_like(lse, RHO))}
    if do is None:
        return out
    do = do.double()
    dp = torch.einsum("ihd,jhd->hij", do, vv)
    ds = p * (dp - torch.einsum("ihd,ihd->hi", do, o)[..., None])
    e_ds = 1.01 * ((U + RHO) * ds.abs() + p * (torch.einsum("ihd,ihd->hi", do.abs(), e_o)[..., None] +
                                               2.0 ** -15 * torch.einsum("ihd,jhd->hij", do.abs(), vv.abs())))
    dq = scale * torch.einsum("hij,jhd->ihd", ds, kk)
    e_dq = scale * torch.einsum("hij,jhd->ihd", e_ds, kk.abs()) + U * dq.abs() + 1e-6

    def fold(x):
        return x.view(J, Hkv, g, d).sum(2)
    dk = fold(scale * torch.einsum("hij,ihd->jhd", ds, q))
    e_dk = fold(scale * torch.einsum("hij,ihd->jhd", e_ds, q.abs())) + U * dk.abs() + 1e-6
    dv = fold(torch.einsum("hij,ihd->jhd", p, do))
    e_dv = fold(1.01 * (U + RHO) * torch.einsum("hij,ihd->jhd", p, do.abs())) + U * dv.abs() + 1e-6
    out.update(dq=(dq, e_dq), dk=(dk, e_dk), dv=(dv, e_dv))
    return out


def check(got, want, what):
    """got (a tensor) against want = (value, bound)."""
    ref, tol = want
    x = got.detach().double().cpu()
    assert x.shape == ref.shape, (what, x.shape, ref.shape)
    inf = torch.isneginf(ref)
    assert torch.equal(torch.isneginf(x), inf), f"{what}: -inf pattern"
    err = torch.where(inf, 0.0, (x - torch.where(inf, 0.0, ref)).abs())
    assert torch.isfinite(err).all(), f"{what}: not finite"
    if err.numel():
        assert (err <= tol).all(), f"{what}: {(err / tol).max().item():.3f} of its bound"
