"""NaN and infinities inside a sequence's own rows: the gradients that the
formulas make NaN are, those of other sequences have the bits they had; rows
whose logits are all -inf take no part."""
import math

import pytest
import torch

from . import dense_ref as R
from .test_gpu_dense import make, vsa
from .test_gpu_dense_nonfinite import HEADS, inputs, seeing_rows

pytestmark = pytest.mark.gpu


def gradients(q, k, v, cu_q, cu_kv, causal, dout):
    out, lse = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv, causal=causal, return_lse=True)
    res = vsa().dense_attn_varlen_backward(q, k, v, out, dout, lse, cu_q, cu_kv, causal=causal)
    vsa().check_device_status()
    return out, lse, res


def check_nan(got, clean, rows, cu_q, cu_kv, causal, hkv):
    """`rows` [Hq, q rows]: rows whose log-sum-exp is NaN.  Their dq, and dk and dv
    of every key that one of them sees, are NaN."""
    dq, dk, dv = got
    assert rows.any() and torch.isnan(dq[rows]).all()
    n, lk = cu_q[2] - cu_q[1], cu_kv[2] - cu_kv[1]
    vis = R.visible(n, lk, causal).double().cuda()
    per_head = rows[:, cu_q[1]:cu_q[2]].double() @ vis
    keys = per_head.view(hkv, -1, lk).sum(1) > 0
    for x in (dk, dv):
        assert torch.isnan(x[:, cu_kv[1]:cu_kv[2]][keys]).all()
    for x, y, cu in ((dq, clean[0], cu_q), (dk, clean[1], cu_kv), (dv, clean[2], cu_kv)):
        for i in (0, 2):
            assert torch.equal(x[:, cu[i]:cu[i + 1]], y[:, cu[i]:cu[i + 1]])


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("d", [64, 128])
def test_nan_logits_of_a_key(d, heads, causal, value):
    q, k, v, cu_q, cu_kv = inputs(heads, d, seed=d + heads[0] + 5)
    dout = R.normal(q.shape, d)
    clean = gradients(q, k, v, cu_q, cu_kv, causal, dout)[2]
    for start in (0, 97, 388):
        keys = [start + h for h in range(heads[1])]
        kb = k.clone()
        for h, j in enumerate(keys):
            kb[h, cu_kv[1] + j, 0] = value
        got = gradients(q, kb, v, cu_q, cu_kv, causal, dout)[2]
        check_nan(got, clean, seeing_rows(heads[0], cu_q, cu_kv, causal, keys), cu_q, cu_kv, causal, heads[1])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_query_rows(d, heads, causal):
    """One bad row to a head, the heads together at every place of a tile's columns."""
    q, k, v, cu_q, cu_kv = inputs(heads, d, seed=d + heads[0] + 6)
    dout = R.normal(q.shape, d)
    clean = gradients(q, k, v, cu_q, cu_kv, causal, dout)[2]
    for start in (0, 100, 236):
        qb = q.clone()
        bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
        for h in range(heads[0]):
            bad[h, cu_q[1] + start + h] = True
        qb[bad, d - 1] = math.nan
        check_nan(gradients(qb, k, v, cu_q, cu_kv, causal, dout)[2], clean, bad, cu_q, cu_kv, causal, heads[1])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(4, 4), (4, 2), (8, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_whose_logits_are_all_minus_infinity(d, heads, causal):
    """Finite inputs whose logits leave fp32's range: such a row's output is 0, its
    log-sum-exp -inf, and its share of every gradient 0."""
    lens = [(65, 65), (300, 420), (1500, 1500)] if heads == (8, 1) else [(65, 65), (300, 420), (40, 33)]
    q, k, v, cu_q, cu_kv = make(*heads, d, lens, seed=d + heads[0] + 7)
    dout = R.normal(q.shape, d)
    q[..., 0] = 0
    k[..., 0] = -2.0 ** 100
    dead = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    dead[:, cu_q[1]:cu_q[2]:7], dead[1, cu_q[2] - 1], dead[0, 10] = True, True, True
    q[dead] = 0
    q[dead, 0] = 2.0 ** 100  # logits of -2^200
    out, lse, got = gradients(q, k, v, cu_q, cu_kv, causal, dout)
    # (in 64 bits, where these logits are numbers, only rows without keys have lse = -inf)
    without_keys = torch.isinf(R.forward(q, k, v, cu_q, cu_kv, causal)[1]).cuda()
    assert (out[dead] == 0).all() and torch.equal(lse == -math.inf, dead | without_keys)
    # in 64 bits the rows take no part where their dout is 0
    dout[dead] = 0
    want, tol = R.backward(q, k, v, dout, cu_q, cu_kv, causal)
    for name, x, y, z in zip(("dq", "dk", "dv"), got, want, tol):
        R.assert_within(x, y, z, name)
