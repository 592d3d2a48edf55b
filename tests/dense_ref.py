"""Dense attention of packed sequences in 64 bits, with bounds on what bf16
kernels may differ by.

Bounds (derived, not fitted).  u = 2^-8 is half a bf16 step relative to the
value, the most one rounding changes it by.  A probability carries a relative
error of at most PEXP = 8e-5 (the polynomial exponential; the special-function
unit's is below it) plus the error of its logit, at most
ELOG = 2 D 2^-23 scale max sum_d |q_d k_d| (fp32 products and sums), so
e = PEXP + 2 ELOG relative, numerator and normaliser.
* out = sum_j p_j v_j with p_j rounded to bf16 and the result rounded once:
  |err| <= (u + 2 e) sum_j p_j |v_j| + u |out|, plus the second order.
* lse: |err| <= PEXP + ELOG + 2^-21 |lse|.
* gradients: p and ds are rounded to bf16 before their products, the result
  once; delta = sum_d dout out takes out rounded to bf16, an error of at most
  u sum_d |dout_d out_d| =: u E, plus the out kernel's own (u + 2 e)
  sum_d |dout_d| A_d with A = sum_j p_j |v_j|; so with
  F = E + sum_d |dout_d| A_d,  |err(ds_j)| <= p_j ((2 u + 2 e) F +
  (u + 2 e) |dp_j - delta| + ELOG-sized error of dp_j), and
  |err(dq)| <= scale sum_j |err(ds_j)| |k_j| + u |dq|; dk likewise over rows,
  |err(dv)| <= (u + 2 e) sum_r p_rj |dout_r| + u |dv|.
The second order is covered by the factor 1.02.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8
PEXP = 8e-5
SLACK = 1.02


def visible(lq, lk, causal):
    if not causal:
        return torch.ones(lq, lk, dtype=torch.bool)
    return torch.arange(lk)[None, :] < torch.arange(lq)[:, None] + 1 + lk - lq


def attend(q, k, v, scale, seen):
    """One head of one sequence: (probabilities, out, lse, out bound, lse bound), fp64."""
    s = scale * (q @ k.T)
    s = torch.where(seen, s, -math.inf)
    lse = torch.logsumexp(s, -1) if s.shape[1] else torch.full((s.shape[0],), -math.inf, dtype=q.dtype)
    p = torch.where(seen, torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[:, None]), 0.0)
    out = p @ v
    mags = scale * (q.abs() @ k.abs().T)
    mags = torch.where(seen, mags, 0.0)
    elog = 2 * q.shape[1] * 2.0 ** -23 * (mags.amax(-1) if mags.shape[1] else mags.sum(-1))
    e = PEXP + 2 * elog
    a = p @ v.abs()
    tol = SLACK * ((U + 2 * e)[:, None] * a + U * out.abs()) + 1e-30
    tol_lse = SLACK * (PEXP + elog + 2.0 ** -21 * torch.where(torch.isinf(lse), 0.0, lse).abs())
    return p, out, lse, tol, tol_lse, e, a


def forward(q, k, v, cu_q, cu_kv, causal=True, scale=None):
    """(out, lse, tol_out, tol_lse) fp64 on the CPU for [H, rows, D] inputs; rows
    past the last sequence are NaN (not defined by the operator)."""
    q, k, v = (x.detach().double().cpu() for x in (q, k, v))
    scale = 1.0 / math.sqrt(q.shape[2]) if scale is None else scale
    g = q.shape[0] // k.shape[0]
    out = torch.full_like(q, math.nan)
    tol = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float64)
    tol_lse = torch.zeros_like(lse)
    for i in range(len(cu_q) - 1):
        a, b = slice(cu_q[i], cu_q[i + 1]), slice(cu_kv[i], cu_kv[i + 1])
        seen = visible(cu_q[i + 1] - cu_q[i], cu_kv[i + 1] - cu_kv[i], causal)
        for h in range(q.shape[0]):
            _, out[h, a], lse[h, a], tol[h, a], tol_lse[h, a], _, _ = attend(
                q[h, a], k[h // g, b], v[h // g, b], scale, seen)
    return out, lse, tol, tol_lse


def backward(q, k, v, dout, cu_q, cu_kv, causal=True, scale=None):
    """((dq, dk, dv), (their bounds)) fp64 on the CPU."""
    q, k, v, dout = (x.detach().double().cpu() for x in (q, k, v, dout))
    scale = 1.0 / math.sqrt(q.shape[2]) if scale is None else scale
    g = q.shape[0] // k.shape[0]
    grads = [torch.zeros_like(x) for x in (q, k, v)]
    tols = [torch.zeros_like(x) for x in (q, k, v)]
    for i in range(len(cu_q) - 1):
        a, b = slice(cu_q[i], cu_q[i + 1]), slice(cu_kv[i], cu_kv[i + 1])
        seen = visible(cu_q[i + 1] - cu_q[i], cu_kv[i + 1] - cu_kv[i], causal)
        for h in range(q.shape[0]):
            qq, kk, vv, do = q[h, a], k[h // g, b], v[h // g, b], dout[h, a]
            p, out, _, _, _, e, am = attend(qq, kk, vv, scale, seen)
            dp = do @ vv.T
            delta = (do * out).sum(-1, keepdim=True)
            ds = p * (dp - delta)
            grads[0][h, a] = scale * ds @ kk
            grads[1][h // g, b] += scale * ds.T @ qq
            grads[2][h // g, b] += p.T @ do
            e = e[:, None]
            f = (do * out).abs().sum(-1, keepdim=True) + (do.abs() * am).sum(-1, keepdim=True)
            edp = 2 * q.shape[2] * 2.0 ** -23 * (do.abs() @ vv.abs().T)
            eds = p * ((2 * U + 2 * e) * f + (U + 2 * e) * (dp - delta).abs() + edp)
            tols[0][h, a] = scale * eds @ kk.abs()
            tols[1][h // g, b] += scale * eds.T @ qq.abs()
            tols[2][h // g, b] += ((U + 2 * e) * p).T @ do.abs()
    return tuple(grads), tuple(SLACK * (t + U * x.abs()) + 1e-30 for t, x in zip(tols, grads))


def decode(q, kp, vp, ks, vs, lens, scale=None):
    """(out, lse, tol_out, tol_lse) fp64 on the CPU of shared-prefix decoding;
    partial results and their joining stay in fp32 (PEXP covers the weights),
    so the bounds are the forward's."""
    lens = [int(n) for n in lens]
    q, kp, vp, ks, vs = (x.detach().double().cpu() for x in (q, kp, vp, ks, vs))
    scale = 1.0 / math.sqrt(q.shape[3]) if scale is None else scale
    b, hq, t, _ = q.shape
    p, g = kp.shape[1], hq // kp.shape[0]
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    lse, tol_lse = torch.zeros(q.shape[:3], dtype=q.dtype), torch.zeros(q.shape[:3], dtype=q.dtype)
    for i in range(b):
        seen = torch.arange(p + lens[i])[None, :] < (p + (lens[i] - t + 1 + torch.arange(t)).clamp_min(0))[:, None]
        for h in range(hq):
            k = torch.cat([kp[h // g], ks[i, h // g, :lens[i]]])
            v = torch.cat([vp[h // g], vs[i, h // g, :lens[i]]])
            _, out[i, h], lse[i, h], tol[i, h], tol_lse[i, h], _, _ = attend(q[i, h], k, v, scale, seen)
    return out, lse, tol, tol_lse


def assert_within(got, want, tol, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    same = (got == want) | (torch.isnan(want))
    err = torch.where(same, 0.0, (got - want).abs())
    bad = ~(err <= torch.where(same, 1.0, tol))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{bad.nonzero()[0].tolist()}, worst ratio {(err / tol)[bad].max()}")


def rel_rms(got, want):
    got = got.detach().double().cpu()
    ok = torch.isfinite(want)
    return float(((got - want)[ok].norm() / want[ok].norm().clamp_min(1e-300)))


def cumulative(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def normal(shape, seed, device="cuda", mult=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * mult).to(torch.bfloat16).to(device)
