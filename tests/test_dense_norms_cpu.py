"""The comparison of dense_norms lets correctly rounded results pass and rejects
plausible mistakes, planted in the reference, that the elementwise bounds of
dense_ref may let through."""
import pytest
import torch

from . import dense_norms as N
from . import dense_ref as R

PAIRS = [(700, 700), (300, 420)]


def inputs(hq, hkv, d, pairs, seed):
    cu_q, cu_kv = R.cumulative([a for a, _ in pairs]), R.cumulative([b for _, b in pairs])
    q, dout = (R.normal((hq, cu_q[-1], d), seed + i, "cpu") for i in range(2))
    k, v = (R.normal((hkv, cu_kv[-1], d), seed + 2 + i, "cpu") for i in range(2))
    return q, k, v, dout, cu_q, cu_kv


def without_head(h, p, ds):
    return (p * 0, ds * 0) if h == 3 else (p, ds)


def without_last_query_tile(h, p, ds):
    keep = (torch.arange(p.shape[0]) < (p.shape[0] - 1) // 128 * 128).double()[:, None]
    return p * keep, ds * keep


def without_a_share(h, p, ds):
    """One of 12 shares of the walk over all heads' query tiles: half a head's rows."""
    keep = (torch.arange(p.shape[0]) >= p.shape[0] // 2).double()[:, None]
    return (p * keep, ds * keep) if h == 5 else (p, ds)


def without_a_key_tile(h, p, ds):
    keep = ((torch.arange(p.shape[1]) < 128) | (torch.arange(p.shape[1]) >= 256)).double()
    return p * keep, ds if ds is None else ds * keep


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("mistake", [without_head, without_last_query_tile, without_a_share, without_a_key_tile])
def test_mistakes_in_the_gradients(mistake, causal):
    q, k, v, dout, cu_q, cu_kv = inputs(8, 1, 64, PAIRS, 1)
    want = N.attention64(q, k, v, cu_q, cu_kv, causal, dout)
    wrong = N.attention64(q, k, v, cu_q, cu_kv, causal, dout, mistake)
    for name, x, y, cu in zip(("dq", "dk", "dv"), want, wrong, (cu_q, cu_kv, cu_kv)):
        N.assert_close(x.to(torch.bfloat16), x, cu, name)
        with pytest.raises(AssertionError):
            N.assert_close(y.to(torch.bfloat16), x, cu, name)


def test_gradients_without_delta():
    """Off by 0.03 and more of the norm, for one sequence behind many keys."""
    q, k, v, dout, cu_q, cu_kv = inputs(4, 1, 64, [(300, 2000)], 5)
    want = N.attention64(q, k, v, cu_q, cu_kv, True, dout)

    def no_delta(h, p, ds):
        return p, p * (dout[h].double() @ v[0].double().T)

    wrong = N.attention64(q, k, v, cu_q, cu_kv, True, dout, no_delta)
    for name, x, y, cu in zip(("dq", "dk"), want, wrong, (cu_q, cu_kv)):
        with pytest.raises(AssertionError):
            N.assert_close(y.to(torch.bfloat16), x, cu, name)


def test_a_key_tile_of_forty_missing_from_the_output():
    q, k, v, _, cu_q, cu_kv = inputs(2, 1, 64, [(130, 5000)], 9)
    want = N.attention64(q, k, v, cu_q, cu_kv, True)
    N.assert_close(want.to(torch.bfloat16), want, cu_q, "out")
    with pytest.raises(AssertionError):
        N.assert_close(N.attention64(q, k, v, cu_q, cu_kv, True, drop=without_a_key_tile), want, cu_q, "out")


def test_the_reference_is_that_of_the_elementwise_bounds():
    q, k, v, dout, cu_q, cu_kv = inputs(4, 2, 64, [(40, 70), (9, 5), (0, 3), (6, 0)], 11)
    for causal in (True, False):
        out = R.forward(q, k, v, cu_q, cu_kv, causal)[0]
        assert torch.allclose(N.attention64(q, k, v, cu_q, cu_kv, causal), out, rtol=1e-12, atol=1e-14)
        for x, y in zip(N.attention64(q, k, v, cu_q, cu_kv, causal, dout), R.backward(q, k, v, dout, cu_q, cu_kv, causal)[0]):
            assert torch.allclose(x, y, rtol=1e-12, atol=1e-14)
