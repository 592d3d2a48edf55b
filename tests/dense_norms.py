"""Relative errors of the dense entries' results over blocks of them.

The elementwise bounds of dense_ref add worst cases over keys or rows, so on
long sequences they exceed the results themselves.  A block's error norm does
not add up like that: each element of a correct result is off by a handful of
independent roundings to bf16 (its terms', out's within delta, its own), of
U / sqrt(3) RMS each at most, some 0.002 to 0.004 of the block's norm.  LIMIT
is 4 U = 0.016: a result that lacks a head of a group, a tile or a share of a
sum is off by more (test_dense_norms_cpu.py).  For logits of ordinary size and
blocks whose results do not cancel (rows that see one key have dq = 0).
"""
import math

import torch

from . import dense_ref as R

LIMIT = 4 * R.U


def attention64(q, k, v, cu_q, cu_kv, causal, dout=None, drop=None):
    """fp64 out, or with dout (dq, dk, dv), on the inputs' device.  `drop(h, p, ds)`
    may change a head's probabilities and ds (rows x keys) on the way."""
    q, k, v = (x.detach().double() for x in (q, k, v))
    g = q.shape[0] // k.shape[0]
    scale = 1.0 / math.sqrt(q.shape[2])
    out = torch.zeros_like(q)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for i in range(len(cu_q) - 1):
        a, b = slice(cu_q[i], cu_q[i + 1]), slice(cu_kv[i], cu_kv[i + 1])
        if a.start == a.stop or b.start == b.stop:
            continue
        seen = R.visible(a.stop - a.start, b.stop - b.start, causal).to(q.device)
        for h in range(q.shape[0]):
            s = torch.where(seen, scale * (q[h, a] @ k[h // g, b].T), -math.inf)
            lse = torch.logsumexp(s, -1, keepdim=True)
            p = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse))
            if dout is None:
                out[h, a] = (drop(h, p, None)[0] if drop else p) @ v[h // g, b]
                continue
            do = dout[h, a].double()
            ds = p * (do @ v[h // g, b].T - (do * (p @ v[h // g, b])).sum(-1, keepdim=True))
            if drop:
                p, ds = drop(h, p, ds)
            dq[h, a] = scale * ds @ k[h // g, b]
            dk[h // g, b] += scale * ds.T @ q[h, a]
            dv[h // g, b] += p.T @ do
    return out if dout is None else (dq, dk, dv)


def worst_block(got, want, cu):
    """The largest relative error norm over the whole, every sequence and head and
    every 128-row tile of one; a block that should be 0 counts as infinite if it is not."""
    got = got.detach().double().to(want.device)
    blocks = [(slice(None), slice(0, cu[-1]))]
    for i in range(len(cu) - 1):
        for h in range(want.shape[0]):
            blocks.append((slice(h, h + 1), slice(cu[i], cu[i + 1])))
            blocks += [(slice(h, h + 1), slice(r, min(r + 128, cu[i + 1]))) for r in range(cu[i], cu[i + 1], 128)]
    worst = 0.0
    for b in blocks:
        norm, err = want[b].norm(), (got[b] - want[b]).norm()
        worst = max(worst, float(err / norm) if norm > 0 else (0.0 if err == 0 else math.inf))
    return worst


def assert_close(got, want, cu, what):
    worst = worst_block(got, want, cu)
    assert worst <= LIMIT, f"{what}: a block is off by {worst} of its norm"
