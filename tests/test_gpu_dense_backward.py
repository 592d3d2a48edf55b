"""Gradients of dense packed attention on the GPU against the 64-bit formulas
(bounds in dense_ref), and against differences of the 64-bit loss."""
import pytest
import torch

from . import dense_ref as R
from .test_gpu_dense import LENGTHS, make

pytestmark = pytest.mark.gpu


def vsa():
    from block_sparse_attention_15_b200 import binding
    return binding


def gradients(q, k, v, cu_q, cu_kv, causal, dout, scale=None, **kw):
    out, lse = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv, causal=causal, scale=scale, return_lse=True)
    return vsa().dense_attn_varlen_backward(q, k, v, out, dout, lse, cu_q, cu_kv, causal=causal, scale=scale, **kw)


def check(q, k, v, cu_q, cu_kv, causal, seed=99, scale=None):
    dout = R.normal(q.shape, seed)
    got = gradients(q, k, v, cu_q, cu_kv, causal, dout, scale)
    vsa().check_device_status()
    want, tol = R.backward(q, k, v, dout, cu_q, cu_kv, causal, scale)
    for n, a, b, c in zip(("dq", "dk", "dv"), got, want, tol):
        R.assert_within(a, b, c, n)
    return got, dout


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", list(LENGTHS))
@pytest.mark.parametrize("heads", [(1, 1), (4, 2), (3, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_gradients(d, heads, lens, causal):
    check(*make(*heads, d, LENGTHS[lens], seed=d + heads[0]), causal)


@pytest.mark.parametrize("heads", [(7, 1), (10, 2), (28, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_more_items_than_sms(d, heads):
    pairs = [(1000, 1000), (130, 400), (700, 700), (1, 1), (513, 100), (900, 1111), (350, 350)]
    check(*make(*heads, d, pairs, seed=5), True)
    check(*make(*heads, d, pairs, seed=6), False)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(8, 1), (32, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_key_tiles(d, heads, causal):
    """Fewer key tiles than SMs: their walks are shared out, some shares empty,
    beside sequences without rows or keys."""
    check(*make(*heads, d, [(700, 700)], seed=d), causal)
    check(*make(*heads, d, [(130, 400), (0, 5), (600, 777), (5, 0), (1, 200), (300, 20)], seed=d + 1, extra=7), causal)


def test_long():
    """2049 rows behind 5000 keys."""
    check(*make(16, 4, 128, [(2049, 5000), (3, 3)], seed=9), True)


def test_many_sequences():
    pairs = [(1 + i % 3, 1 + (i * 7) % 40) for i in range(300)]
    check(*make(4, 2, 64, pairs, seed=11), True)


def test_peaked_logits_and_scale():
    check(*make(4, 2, 128, [(300, 900), (65, 65)], seed=20, mult=4.0), True)
    check(*make(2, 1, 64, [(70, 200)], seed=31), True, scale=0.5)


@pytest.mark.parametrize("causal", [True, False])
def test_against_differences(causal):
    """The 64-bit formulas, which the kernels are held to, against central
    differences of sum(out * dout); and the kernels' directional derivative."""
    pairs = [(40, 70), (9, 9)]
    q, k, v, cu_q, cu_kv = make(4, 2, 64, pairs, seed=70)
    got, dout = check(q, k, v, cu_q, cu_kv, causal)
    want, _ = R.backward(q, k, v, dout, cu_q, cu_kv, causal)
    gen = torch.Generator().manual_seed(1)
    base = [x.double().cpu() for x in (q, k, v)]
    loss = lambda xs: (R.forward(*xs, cu_q, cu_kv, causal)[0] * dout.double().cpu()).sum()  # noqa: E731
    for i in range(3):
        step = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        plus, minus = list(base), list(base)
        plus[i], minus[i] = base[i] + h * step, base[i] - h * step
        slope = (loss(plus) - loss(minus)) / (2 * h)
        # the difference quotient is off by O(h^2) and by rounding of the loss over h
        assert abs(slope - (want[i] * step).sum()) <= 1e-6 * (1 + want[i].abs().mul(step.abs()).sum())
        # each element is off by at most a few bf16 half steps of its largest terms (check());
        # a direction mixes them with random signs
        err = (got[i].double().cpu() - want[i]).norm() / want[i].norm()
        assert err < 4 * R.U


def test_neighbours_do_not_matter():
    pairs = [(100, 100), (60, 60), (200, 333), (1, 5)]
    q, k, v, cu_q, cu_kv = make(4, 2, 128, pairs, seed=40, extra=9)
    dout = R.normal(q.shape, 41)
    out, lse = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv, return_lse=True)
    want = vsa().dense_attn_varlen_backward(q, k, v, out, dout, lse, cu_q, cu_kv)
    for bad in (float("nan"), float("inf")):
        rows, keys = [x.clone() for x in (q, out, dout, lse)], [x.clone() for x in (k, v)]
        for x, cu in [(x, cu_q) for x in rows] + [(x, cu_kv) for x in keys]:
            for i in (1, 3):
                x[:, cu[i]:cu[i + 1]] = bad
            x[:, cu[-1]:] = bad
        got = vsa().dense_attn_varlen_backward(rows[0], *keys, rows[1], rows[2], rows[3], cu_q, cu_kv)
        for a, b, cu in zip(got, want, (cu_q, cu_kv, cu_kv)):
            for i in (0, 2):
                assert torch.equal(a[:, cu[i]:cu[i + 1]], b[:, cu[i]:cu[i + 1]])


def test_views_and_rows_behind():
    """Token-major and fused views of every tensor give the contiguous result bit
    for bit; rows behind the last sequence keep what they held."""
    pairs = [(130, 130), (77, 77), (300, 300)]
    cu = R.cumulative([a for a, _ in pairs])
    hq, hkv, d, rows = 6, 2, 128, cu[-1] + 20
    fused = R.normal((rows, (hq + 2 * hkv) * d), 50).view(rows, hq + 2 * hkv, d)
    parts = ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv))
    q, k, v = (fused[:, a:b].transpose(0, 1) for a, b in parts)
    want, dout = check(q.contiguous(), k.contiguous(), v.contiguous(), cu, cu, True)
    grads = torch.full_like(fused, 7.0)
    dq, dk, dv = (grads[:, a:b].transpose(0, 1) for a, b in parts)
    got = gradients(q, k, v, cu, cu, True, dout.transpose(0, 1).contiguous().transpose(0, 1), dq=dq, dk=dk, dv=dv)
    for a, b, c in zip(got, want, (dq, dk, dv)):
        assert a is c and torch.equal(a[:, :cu[-1]], b[:, :cu[-1]])
    assert (grads[cu[-1]:] == 7).all()


def test_stream_and_graph():
    pairs = [(300, 300), (5, 150)]
    args = make(4, 2, 64, pairs, seed=60)
    dout = R.normal(args[0].shape, 61)
    want = gradients(*args, True, dout)
    out, lse = vsa().dense_attn_varlen(*args, return_lse=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = vsa().dense_attn_varlen_backward(*args[:3], out, dout, lse, *args[3:], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gradients(*args, True, dout)
    gradients(*make(4, 2, 64, [(400, 400), (1, 1), (9, 9)], seed=63), True, R.normal((4, 410, 64), 64))
    new = make(4, 2, 64, pairs, seed=65)
    want = gradients(*new, True, dout)
    for a, b in zip(args[:3], new[:3]):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_repeats_are_equal():
    args = make(12, 4, 128, [(900, 900), (33, 400), (512, 512)], seed=70)
    dout = R.normal(args[0].shape, 71)
    first = gradients(*args, True, dout)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(gradients(*args, True, dout), first))


def test_refusals():
    B = vsa()
    q, k, v, cu_q, cu_kv = make(4, 2, 64, [(10, 10)], seed=80)
    out, lse = B.dense_attn_varlen(q, k, v, cu_q, cu_kv, return_lse=True)
    f = B.dense_attn_varlen_backward
    with pytest.raises(ValueError):
        f(q, k, v, out, out[:2], lse, cu_q, cu_kv)
    with pytest.raises(ValueError):
        f(q, k, v, out, q, lse[:, :5].contiguous(), cu_q, cu_kv)
    with pytest.raises(TypeError):
        f(q, k, v, out, q, lse.double(), cu_q, cu_kv)
    with pytest.raises(TypeError):
        f(q, k, v, out, q.float(), lse, cu_q, cu_kv)
    with pytest.raises(ValueError):
        f(q, k, v, out, q, lse, cu_q, cu_kv, dk=torch.empty_like(q))
    with pytest.raises(ValueError):
        f(q, k, v, out, q[:1].expand(4, -1, -1), lse, cu_q, cu_kv)
    with pytest.raises(B.VSAError):
        f(q, k, v, out, q, lse, [0, 11], cu_kv)
    with pytest.raises(B.VSAError):
        f(q, k, v, out, q, lse, cu_q, cu_kv, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert B.get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_no_keys_or_no_rows_at_all(d):
    B = vsa()
    q, dout = R.normal((4, 50, d), 90), R.normal((4, 50, d), 91)
    none = torch.empty((2, 0, d), dtype=torch.bfloat16, device="cuda")
    out, lse = B.dense_attn_varlen(q, none, none, [0, 20, 50], [0, 0, 0], return_lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()
    dq, dk, dv = B.dense_attn_varlen_backward(q, none, none, out, dout, lse, [0, 20, 50], [0, 0, 0])
    assert (dq == 0).all() and dk.shape == dv.shape == none.shape
    rows = torch.empty((4, 0, d), dtype=torch.bfloat16, device="cuda")
    k, v = R.normal((2, 300, d), 92), R.normal((2, 300, d), 93)
    out, lse = B.dense_attn_varlen(rows, k, v, [0, 0], [0, 300], return_lse=True)
    dq, dk, dv = B.dense_attn_varlen_backward(rows, k, v, out, out, lse, [0, 0], [0, 300])
    assert dq.shape == rows.shape and (dk == 0).all() and (dv == 0).all()
    B.check_device_status()


def test_calls_side_by_side():
    """Forward and gradients on two streams at once, each with more items than
    SMs and waiting for the other's: the results of the calls alone."""
    sets = []
    for seed, lens in ((95, [(700, 700), (900, 1111)]), (96, [(1000, 1000), (130, 400), (5, 0)])):
        args = make(28, 4, 128, lens, seed=seed)
        dout = R.normal(args[0].shape, seed)
        sets.append((args, dout, gradients(*args, True, dout), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for args, dout, want, stream in sets:
            with torch.cuda.stream(stream):
                got.append((gradients(*args, True, dout), want))
    torch.cuda.synchronize()
    vsa().check_device_status()
    for a, b in got:
        assert all(torch.equal(x, y) for x, y in zip(a, b))
