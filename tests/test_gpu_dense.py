"""Dense packed attention on the GPU against the 64-bit reference (bounds in dense_ref)."""
import math

import pytest
import torch

from . import dense_ref as R

pytestmark = pytest.mark.gpu


def vsa():
    from block_sparse_attention_15_b200 import binding
    return binding


def make(hq, hkv, d, pairs, seed=0, mult=1.0, extra=0):
    cu_q, cu_kv = R.cumulative([a for a, _ in pairs]), R.cumulative([b for _, b in pairs])
    q = R.normal((hq, cu_q[-1] + extra, d), seed, mult=mult)
    k = R.normal((hkv, cu_kv[-1] + extra, d), seed + 1, mult=mult)
    v = R.normal((hkv, cu_kv[-1] + extra, d), seed + 2)
    return q, k, v, cu_q, cu_kv


def check(q, k, v, cu_q, cu_kv, causal, scale=None):
    out, lse = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv, causal=causal, scale=scale, return_lse=True)
    vsa().check_device_status()
    want, wlse, tol, tlse = R.forward(q, k, v, cu_q, cu_kv, causal, scale)
    R.assert_within(out, want, tol, "out")
    R.assert_within(lse, wlse, tlse, "lse")
    return out, lse


LENGTHS = {
    "one": [(1, 1)],
    "edges": [(127, 127), (128, 128), (129, 129), (255, 255), (257, 257)],
    "ragged": [(1, 300), (300, 77), (64, 64), (16, 17), (15, 15), (200, 513)],
    "empty": [(0, 5), (5, 0), (33, 33), (0, 0), (300, 100), (7, 7)],
    "decode": [(1, 1025), (2, 640), (3, 129)],
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", list(LENGTHS))
@pytest.mark.parametrize("heads", [(1, 1), (4, 2), (3, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_forward(d, heads, lens, causal):
    check(*make(*heads, d, LENGTHS[lens], seed=d + heads[0]), causal)


@pytest.mark.parametrize("heads", [(7, 1), (10, 2), (16, 16), (28, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_forward_two_tiles_per_item(d, heads):
    """More row tiles than SMs: items of two slots, odd and even groups, and
    more items than SMs."""
    pairs = [(1000, 1000), (130, 400), (700, 700), (1, 1), (513, 100), (900, 1111), (350, 350)]
    check(*make(*heads, d, pairs, seed=5), True)
    check(*make(*heads, d, pairs, seed=6), False)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(64, 64), (63, 9), (96, 12)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_heads(d, heads, causal):
    """Items of two slots with the small and empty sequences of test_forward."""
    pairs = [p for lens in LENGTHS.values() for p in lens]
    check(*make(*heads, d, pairs, seed=90 + heads[0]), causal)


def test_many_heads_repeat_and_neighbours():
    pairs = [(300, 300), (5, 150), (129, 60), (1, 1)]
    q, k, v, cu_q, cu_kv = make(96, 8, 64, pairs, seed=95, extra=3)
    want = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv)
    for bad in (float("nan"), float("inf")):
        for i in (1, 3):
            q[:, cu_q[i]:cu_q[i + 1]] = bad
            k[:, cu_kv[i]:cu_kv[i + 1]] = bad
            v[:, cu_kv[i]:cu_kv[i + 1]] = bad
        q[:, cu_q[-1]:], k[:, cu_kv[-1]:], v[:, cu_kv[-1]:] = bad, bad, bad
        for _ in range(3):
            got = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv)
            for i in (0, 2):
                assert torch.equal(got[:, cu_q[i]:cu_q[i + 1]], want[:, cu_q[i]:cu_q[i + 1]])


def test_forward_long():
    """2049 rows behind 5000 keys (several waves of long items)."""
    check(*make(16, 4, 128, [(2049, 5000), (3, 3)], seed=9), True)


def test_many_sequences():
    """More sequences than one launch takes."""
    pairs = [(1 + i % 3, 1 + (i * 7) % 40) for i in range(300)]
    check(*make(4, 2, 64, pairs, seed=11), True)


def test_peaked_logits():
    """Large logits: the reference max moves often, and far-off keys vanish."""
    for seed in range(3):
        q, k, v, cu_q, cu_kv = make(4, 2, 128, [(300, 900), (65, 65)], seed=20 + seed, mult=4.0)
        check(q, k, v, cu_q, cu_kv, True)
    # keys that grow along the sequence: every tile raises the max
    q, k, v, cu_q, cu_kv = make(2, 2, 64, [(256, 1000)], seed=30)
    k = (k.float() * torch.linspace(0.1, 12, 1000, device="cuda")[None, :, None]).to(torch.bfloat16)
    check(q, k, v, cu_q, cu_kv, True)
    check(q, k, v, cu_q, cu_kv, False)


def test_scale_and_constant_inputs():
    q, k, v, cu_q, cu_kv = make(2, 1, 64, [(70, 200)], seed=31)
    check(q, k, v, cu_q, cu_kv, True, scale=0.5)
    out, lse = check(torch.zeros_like(q), k, v, cu_q, cu_kv, False)
    assert torch.allclose(lse, torch.full_like(lse, math.log(200.0)), atol=2e-4)


def test_neighbours_do_not_matter():
    """NaN and infinities in other sequences' rows, and past the last one."""
    pairs = [(100, 100), (60, 60), (200, 333), (1, 5)]
    q, k, v, cu_q, cu_kv = make(4, 2, 128, pairs, seed=40, extra=9)
    want = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv)
    for bad in (float("nan"), float("inf")):
        qb, kb, vb = q.clone(), k.clone(), v.clone()
        for i in (1, 3):
            qb[:, cu_q[i]:cu_q[i + 1]] = bad
            kb[:, cu_kv[i]:cu_kv[i + 1]] = bad
            vb[:, cu_kv[i]:cu_kv[i + 1]] = bad
        qb[:, cu_q[-1]:], kb[:, cu_kv[-1]:], vb[:, cu_kv[-1]:] = bad, bad, bad
        got = vsa().dense_attn_varlen(qb, kb, vb, cu_q, cu_kv)
        for i in (0, 2):
            assert torch.equal(got[:, cu_q[i]:cu_q[i + 1]], want[:, cu_q[i]:cu_q[i + 1]])


def test_views_and_rows_behind():
    """Token-major and fused-QKV views give the contiguous result bit for bit;
    rows behind the last sequence keep what they held."""
    pairs = [(130, 130), (77, 77), (300, 300)]
    cu = R.cumulative([a for a, _ in pairs])
    hq, hkv, d, rows = 6, 2, 128, cu[-1] + 20
    fused = R.normal((rows, (hq + 2 * hkv) * d), 50).view(rows, hq + 2 * hkv, d)
    q, k, v = (fused[:, a:b].transpose(0, 1) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    want, wlse = check(q.contiguous(), k.contiguous(), v.contiguous(), cu, cu, True)
    got, glse = vsa().dense_attn_varlen(q, k, v, cu, cu, return_lse=True)
    assert torch.equal(got, want) and torch.equal(glse, wlse)
    wide = torch.full((rows, hq, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    vsa().dense_attn_varlen(q, k, v, cu, cu, out=wide[:, :, :d].transpose(0, 1))
    assert torch.equal(wide[:cu[-1], :, :d].transpose(0, 1), want[:, :cu[-1]])
    assert (wide[cu[-1]:] == 7).all() and (wide[:, :, d:] == 7).all()


def test_stream_and_graph():
    """A side stream, and a captured call replayed on new inputs after other
    calls with other lengths."""
    pairs = [(300, 300), (5, 150)]
    q, k, v, cu_q, cu_kv = make(4, 2, 64, pairs, seed=60)
    want = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv, out=out)
    vsa().dense_attn_varlen(*make(4, 2, 64, [(400, 400), (1, 1), (9, 9)], seed=61))
    q2, k2, v2, _, _ = make(4, 2, 64, pairs, seed=62)
    want2 = vsa().dense_attn_varlen(q2, k2, v2, cu_q, cu_kv)
    q.copy_(q2), k.copy_(k2), v.copy_(v2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)


def test_repeats_are_equal():
    q, k, v, cu_q, cu_kv = make(12, 4, 128, [(900, 900), (33, 400), (512, 512)], seed=70)
    first = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv)
    for _ in range(5):
        assert torch.equal(vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv), first)


def test_refusals():
    B = vsa()
    q, k, v, cu_q, cu_kv = make(4, 2, 64, [(10, 10)], seed=80)
    with pytest.raises(B.VSAError):
        B.dense_attn_varlen(q, k, v, [0, 11], cu_kv)          # past the rows
    with pytest.raises(B.VSAError):
        B.dense_attn_varlen(q, k, v, [1, 10], cu_kv)          # not from 0
    with pytest.raises(B.VSAError):
        B.dense_attn_varlen(q[:3], k, v, cu_q, cu_kv)         # 3 heads over 2
    with pytest.raises(ValueError):
        B.dense_attn_varlen(q, k, v, cu_q, [0, 5, 10])        # counts differ
    with pytest.raises(TypeError):
        B.dense_attn_varlen(q.half(), k, v, cu_q, cu_kv)
    with pytest.raises(ValueError):
        B.dense_attn_varlen(q.cpu(), k, v, cu_q, cu_kv)
    with pytest.raises(ValueError):
        B.dense_attn_varlen(q, k[:, :, :32], v, cu_q, cu_kv)  # another head dim
    with pytest.raises(ValueError):
        B.dense_attn_varlen(q[:, :, ::2], k[:, :, ::2], v[:, :, ::2], cu_q, cu_kv)
    with pytest.raises(B.VSAError):
        B.dense_attn_varlen(q[:, :, :32], k[:, :, :32], v[:, :, :32], cu_q, cu_kv)
    assert B.get_device_status() == 0
