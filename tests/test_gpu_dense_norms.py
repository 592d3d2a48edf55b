"""The dense entries on the GPU by the error norms of blocks of their results
(dense_norms), where the elementwise bounds of dense_ref are wide: long
sequences, walks shared by several items, items taken over, several launches."""
import pytest
import torch

from . import dense_norms as N
from . import dense_ref as R
from .test_gpu_dense import make, vsa

pytestmark = pytest.mark.gpu


def run(q, k, v, cu_q, cu_kv, causal, dout):
    out, lse = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv, causal=causal, return_lse=True)
    grads = vsa().dense_attn_varlen_backward(q, k, v, out, dout, lse, cu_q, cu_kv, causal=causal)
    vsa().check_device_status()
    return out, grads


def check(q, k, v, cu_q, cu_kv, causal, seed=7):
    dout = R.normal(q.shape, seed)
    out, grads = run(q, k, v, cu_q, cu_kv, causal, dout)
    N.assert_close(out, N.attention64(q, k, v, cu_q, cu_kv, causal), cu_q, "out")
    want = N.attention64(q, k, v, cu_q, cu_kv, causal, dout)
    for name, x, y, cu in zip(("dq", "dk", "dv"), grads, want, (cu_q, cu_kv, cu_kv)):
        N.assert_close(x, y, cu, name)
    return out, grads, dout


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(8, 1), (32, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_key_tiles(d, heads, causal):
    check(*make(*heads, d, [(700, 700)], seed=d), causal)
    check(*make(*heads, d, [(130, 400), (0, 5), (600, 777), (5, 0), (300, 420)], seed=d + 1, extra=7), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(7, 1), (10, 2), (28, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_more_items_than_sms(d, heads, causal):
    check(*make(*heads, d, [(1000, 1000), (130, 400), (700, 700), (513, 640), (900, 1111), (350, 350)], seed=5), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_long(d, causal):
    check(*make(16, 4, d, [(2049, 5000), (300, 300)], seed=9), causal)
    check(*make(4, 4, d, [(4000, 4000)], seed=10), causal)


@pytest.mark.parametrize("d", [64, 128])
def test_shared_key_tiles_in_two_launches(d):
    """More sequences than a launch takes, a long one in each launch: shared walks
    whose partial sums begin at other rows and have other sizes, in one workspace."""
    pairs = [(0, 0)] * 200
    pairs[5], pairs[150] = (700, 700), (650, 650)
    q, k, v, cu_q, cu_kv = make(8, 1, d, pairs, seed=d + 3)
    out, grads, dout = check(q, k, v, cu_q, cu_kv, True)
    for i in (5, 150):
        # alone a sequence is shared by as many items: the same bits
        a, n = slice(cu_q[i], cu_q[i + 1]), pairs[i][0]
        one, one_grads = run(*(x[:, a].contiguous() for x in (q, k, v)), [0, n], [0, n], True, dout[:, a].contiguous())
        assert torch.equal(out[:, a], one)
        assert all(torch.equal(x[:, a], y) for x, y in zip(grads, one_grads))


@pytest.mark.parametrize("d", [64, 128])
def test_two_launches_with_short_sequences(d):
    """The same among sequences of two rows behind 60 keys, and of none."""
    pairs = [(2, 60) if i % 4 == 0 else (0, 7) if i % 4 == 1 else (0, 0) for i in range(290)]
    pairs[20], pairs[140], pairs[280] = (640, 640), (700, 700), (600, 900)
    check(*make(8, 1, d, pairs, seed=d + 4), False)


@pytest.mark.parametrize("prefix", [0, 3000])
@pytest.mark.parametrize("shape", [(5, 8, 2, 1), (40, 16, 2, 1), (16, 20, 4, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode(d, shape, prefix):
    """Each request's rows as a sequence behind its prefix and suffix."""
    b, hq, hkv, t = shape
    cap = 2000
    lens = [200 + (397 * i) % (cap - 200) for i in range(b)]
    q = R.normal((b, hq, t, d), 1)
    kp, vp = R.normal((hkv, prefix, d), 2), R.normal((hkv, prefix, d), 3)
    ks, vs = R.normal((b, hkv, cap, d), 4), R.normal((b, hkv, cap, d), 5)
    out = vsa().shared_prefix_attn(q, kp, vp, ks, vs, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    vsa().check_device_status()
    for i, n in enumerate(lens):
        k, v = torch.cat([kp, ks[i, :, :n]], 1), torch.cat([vp, vs[i, :, :n]], 1)
        want = N.attention64(q[i], k, v, [0, t], [0, prefix + n], True)
        N.assert_close(out[i], want, [0, t], f"request {i}")
