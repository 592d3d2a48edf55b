"""NaN and infinities inside a sequence's own q and k: they reach the rows whose
logits they make, at every key position, and no other row."""
import math

import pytest
import torch

from . import dense_ref as R
from .test_gpu_dense import make, vsa

pytestmark = pytest.mark.gpu

# 32 key heads, the bad key of head h at place START + h: every place a thread's
# registers can hold.  One query head (few tiles: both slots of an item share
# one) and two (items of two tiles); a sequence before and one behind.
HEADS = [(32, 32), (64, 32)]
PAIRS = [(65, 65), (300, 420), (40, 33)]
STARTS = [0, 64, 97, 256, 388]


def inputs(heads, d, seed):
    q, k, v, cu_q, cu_kv = make(*heads, d, PAIRS, seed=seed)
    q[..., 0] = q[..., 0].abs() + 0.25  # logits of an infinite k[0] have its sign
    return q, k, v, cu_q, cu_kv


def forward(q, k, v, cu_q, cu_kv, causal):
    res = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv, causal=causal, return_lse=True)
    vsa().check_device_status()
    return res


def seeing_rows(hq, cu_q, cu_kv, causal, keys):
    """[Hq, rows]: rows of the middle sequence that see the key of their head's key head."""
    n, lk = cu_q[2] - cu_q[1], cu_kv[2] - cu_kv[1]
    sees = torch.zeros((hq, cu_q[-1]), dtype=torch.bool, device="cuda")
    vis = R.visible(n, lk, causal)
    for h in range(hq):
        sees[h, cu_q[1]:cu_q[2]] = vis[:, keys[h * len(keys) // hq]]
    return sees


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("d", [64, 128])
def test_nan_logits_of_a_key(d, heads, causal, value):
    q, k, v, cu_q, cu_kv = inputs(heads, d, seed=d + heads[0])
    clean = forward(q, k, v, cu_q, cu_kv, causal)
    for start in STARTS:
        keys = [start + h for h in range(heads[1])]
        kb = k.clone()
        for h, j in enumerate(keys):
            kb[h, cu_kv[1] + j, 0] = value
        out, lse = forward(q, kb, v, cu_q, cu_kv, causal)
        bad = seeing_rows(heads[0], cu_q, cu_kv, causal, keys)
        assert bad.any() and torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
        assert torch.equal(out[~bad], clean[0][~bad]) and torch.equal(lse[~bad], clean[1][~bad])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_query_rows(d, heads, causal):
    q, k, v, cu_q, cu_kv = inputs(heads, d, seed=d + heads[0] + 1)
    clean = forward(q, k, v, cu_q, cu_kv, causal)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    bad[::3, cu_q[1] + 5], bad[1::3, cu_q[2] - 1], bad[::2, cu_q[3] - 1] = True, True, True
    q[bad, d - 1] = math.nan
    out, lse = forward(q, k, v, cu_q, cu_kv, causal)
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(out[~bad], clean[0][~bad]) and torch.equal(lse[~bad], clean[1][~bad])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("d", [64, 128])
def test_logits_of_minus_infinity(d, heads, causal):
    """Keys whose logit is -inf weigh nothing: those of the first tiles (nothing is
    seen at first), of the last, and one in four; a row of nothing else gives 0
    and -inf."""
    q, k, v, cu_q, cu_kv = inputs(heads, d, seed=d + heads[0] + 2)
    n, lk, g = cu_q[2] - cu_q[1], cu_kv[2] - cu_kv[1], heads[0] // heads[1]
    cut = {0: slice(0, 256), 1: slice(256, lk), 2: slice(0, lk, 4), 3: slice(0, lk)}
    kb = k.clone()
    for h, which in cut.items():
        kb[h, cu_kv[1]:cu_kv[2]][which, 0] = -math.inf
    out, lse = forward(q, kb, v, cu_q, cu_kv, causal)
    rows, keys = slice(cu_q[1], cu_q[2]), slice(cu_kv[1], cu_kv[2])
    for h, which in cut.items():
        seen = R.visible(n, lk, causal).clone()
        seen[:, which] = False
        for i in range(h * g, h * g + g):
            x, y, z = (t.double().cpu() for t in (q[i, rows], k[h, keys], v[h, keys]))
            _, want, wlse, tol, tlse, _, _ = R.attend(x, y, z, d ** -0.5, seen)
            R.assert_within(out[i, rows], want, tol, f"out {h}")
            R.assert_within(lse[i, rows], wlse, tlse, f"lse {h}")
    none = 3 * g
    assert (out[none:none + g, rows] == 0).all() and (lse[none:none + g, rows] == -math.inf).all()
