"""NaN and infinities inside what a row of shared_prefix_attn reads: they reach
that row, whatever share of the line they fell to, and no other row."""
import math

import pytest
import torch

from . import dense_ref as R
from .test_gpu_prefix import make, vsa

pytestmark = pytest.mark.gpu

# (requests, query heads, key heads, tokens, prefix, capacity): one share of the
# prefix, several, one per SM; blocks of few, of up to 128 and of more rows
SHAPES = [(1, 4, 2, 1, 100, 40), (3, 8, 2, 1, 128, 300), (5, 8, 2, 3, 700, 300), (2, 6, 1, 2, 9000, 2000),
          (40, 16, 2, 1, 700, 180), (40, 16, 1, 1, 1500, 180)]


def inputs(shape, d, seed):
    b, hq, hkv, t, prefix, cap = shape
    args = make(b, hq, hkv, t, d, prefix, cap, [t + (53 * i) % (cap - t + 1) for i in range(b)], seed=seed)
    args[0][..., 0] = args[0][..., 0].abs() + 0.25  # logits of an infinite k[0] have its sign
    return args


def call(args):
    out, lse = vsa().shared_prefix_attn(*args, return_lse=True)
    vsa().check_device_status()
    return out, lse


def check(got, clean, bad):
    """Rows in `bad` [B, Hq, T] are NaN throughout, the others as if nothing had happened."""
    out, lse = got
    assert bad.any()
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(out[~bad], clean[0][~bad]) and torch.equal(lse[~bad], clean[1][~bad])


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_a_query_row(shape, d):
    args = inputs(shape, d, seed=d)
    clean = call(args)
    b, hq, hkv, t, _, _ = shape
    bad = torch.zeros((b, hq, t), dtype=torch.bool, device="cuda")
    bad[b // 2, hq - 1, t - 1] = bad[0, 0, 0] = True
    args[0][bad, d // 2] = math.nan
    check(call(args), clean, bad)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_nan_logits_of_a_prefix_key(shape, d, value):
    """One key of the prefix, in the first, a middle and the last share: every
    row of its key head is NaN (an infinite logit's weight is inf - inf)."""
    args = inputs(shape, d, seed=d + 1)
    clean = call(args)
    b, hq, hkv, t, prefix, _ = shape
    for key in (0, 5, prefix // 2, prefix - 1):
        kp = args[1].clone()
        kp[hkv - 1, key, 0] = value
        bad = torch.zeros((b, hq, t), dtype=torch.bool, device="cuda")
        bad[:, (hkv - 1) * (hq // hkv):] = True
        check(call((args[0], kp, *args[2:])), clean, bad)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_nan_logits_of_a_suffix_key(shape, d, value):
    """A key of one request's own: the rows of that request that see it."""
    args = inputs(shape, d, seed=d + 2)
    clean = call(args)
    b, hq, hkv, t, _, _ = shape
    i = b // 2
    n = int(args[5][i])
    for key in {0, n // 2, n - 1}:
        ks = args[3].clone()
        ks[i, 0, key, 0] = value
        bad = torch.zeros((b, hq, t), dtype=torch.bool, device="cuda")
        sees = n - t + 1 + torch.arange(t, device="cuda") > key
        bad[i, :hq // hkv] = sees
        check(call((*args[:3], ks, *args[4:])), clean, bad)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_logits_of_minus_infinity(shape, d):
    """Keys whose logit is -inf weigh nothing; a row of nothing else gives 0 and -inf."""
    args = inputs(shape, d, seed=d + 3)
    b, hq, hkv, t, prefix, _ = shape
    kp, ks = args[1].clone(), args[3].clone()
    # key head 0: the first half of the prefix weighs nothing (whole shares of it, where there are several)
    half = (prefix + 1) // 2
    kp[0, :half, 0] = -math.inf
    got, lse = call((args[0], kp, args[2], ks, *args[4:]))
    want, wlse, tol, tlse = R.decode(args[0][:, :hq // hkv], args[1][:1, half:], args[2][:1, half:], ks[:, :1],
                                     args[4][:, :1], args[5])
    R.assert_within(got[:, :hq // hkv], want, tol, "out")
    R.assert_within(lse[:, :hq // hkv], wlse, tlse, "lse")
    kp[0, :, 0] = -math.inf
    ks[:, 0, :, 0] = -math.inf
    got, lse = call((args[0], kp, args[2], ks, *args[4:]))
    assert (got[:, :hq // hkv] == 0).all() and (lse[:, :hq // hkv] == -math.inf).all()
    assert torch.isfinite(got).all() and torch.isfinite(lse[:, hq // hkv:]).all()


def test_pieces_that_a_token_does_not_see():
    """A NaN in v of a key tile that an earlier drafted token sees nothing of:
    that token's partial result there weighs nothing, not 0 * NaN."""
    args = make(60, 4, 2, 3, 64, 300, 300, [258] * 60, seed=9)
    clean = call(args)
    vs = args[4].clone()
    vs[:, :, 256:258] = math.nan  # the keys of the two last tokens begin a tile of their own
    out, lse = call((*args[:4], vs, args[5]))
    assert torch.isnan(out[:, :, 1:]).all()
    # where the tile is a share of its own token 0 is whole; it may be NaN elsewhere (0 * NaN in one product)
    whole = torch.isfinite(out[:, :, 0]).all(-1)
    assert whole.any()
    assert torch.equal(out[:, :, 0][whole], clean[0][:, :, 0][whole])
    assert torch.equal(lse, clean[1])
