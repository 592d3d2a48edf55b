"""Decoding over a shared prefix on the GPU against the 64-bit reference (bounds in dense_ref)."""
import pytest
import torch

from . import dense_ref as R

pytestmark = pytest.mark.gpu


def vsa():
    from block_sparse_attention_15_b200 import binding
    return binding


def make(b, hq, hkv, t, d, prefix, cap, lens, seed=0, mult=1.0):
    q = R.normal((b, hq, t, d), seed, mult=mult)
    kp, vp = R.normal((hkv, prefix, d), seed + 1, mult=mult), R.normal((hkv, prefix, d), seed + 2)
    ks, vs = R.normal((b, hkv, cap, d), seed + 3, mult=mult), R.normal((b, hkv, cap, d), seed + 4)
    return q, kp, vp, ks, vs, torch.tensor(lens, dtype=torch.int32, device="cuda")


def check(args, scale=None):
    out, lse = vsa().shared_prefix_attn(*args, scale=scale, return_lse=True)
    vsa().check_device_status()
    want, wlse, tol, tlse = R.decode(*args, scale=scale)
    R.assert_within(out, want, tol, "out")
    R.assert_within(lse, wlse, tlse, "lse")
    return out, lse


@pytest.mark.parametrize("prefix", [0, 1, 128, 129, 700])
@pytest.mark.parametrize("t", [1, 3])
@pytest.mark.parametrize("heads", [(1, 1), (10, 2), (7, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode(d, heads, t, prefix):
    check(make(6, *heads, t, d, prefix, 300, [t, 300, 127, 128, 129, 200], seed=d + t + prefix))


@pytest.mark.parametrize("prefix", [0, 640])
@pytest.mark.parametrize("shape", [(40, 16, 1, 1), (9, 16, 1, 10), (3, 16, 2, 20), (2, 8, 1, 40), (33, 8, 2, 1)])
def test_row_blocks(shape, prefix):
    """More than 128 and 256 rows of a prefix block or of one request."""
    b, hq, hkv, t = shape
    check(make(b, hq, hkv, t, 128, prefix, 180, [t + (37 * i) % (180 - t) for i in range(b)], seed=b))


@pytest.mark.parametrize("rows", [(8, 1), (9, 1), (31, 1), (32, 1), (33, 1), (8, 4), (11, 3), (16, 4), (13, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_a_request(d, rows):
    """Around the 8 rows of a warp and the 32 that four warps share; logits that
    move the reference max, and rows that see nothing of their last tile."""
    hq, t = rows
    check(make(3, hq, 1, t, d, 260, 400, [t, 129 + t // 2, 400], seed=70 + hq, mult=3.0))
    check(make(30, hq, 1, t, d, 0, 300, [(53 * i) % 301 for i in range(30)], seed=71 + hq))


def test_short_pieces_and_row_blocks_in_turn():
    """Many requests of one key tile, and of none, around blocks of a prefix."""
    check(make(33, 8, 1, 1, 128, 640, 180, [(37 * i) % 181 for i in range(33)], seed=79))  # 256 + 8 rows
    check(make(200, 4, 2, 1, 128, 500, 130, [(i * 7) % 131 for i in range(200)], seed=80))
    check(make(150, 8, 4, 1, 64, 1300, 20, [1 + i % 20 if i % 3 else 0 for i in range(150)], seed=81))


@pytest.mark.parametrize("prefix", [0, 5, 256])
def test_lengths_that_leave_rows_empty(prefix):
    """No suffix, fewer suffix keys than new tokens, no keys at all."""
    check(make(5, 4, 2, 4, 64, prefix, 9, [0, 1, 3, 4, 9], seed=prefix))
    check(make(3, 4, 2, 2, 128, prefix, 0, [0, 0, 0], seed=prefix))
    check(make(1, 4, 2, 1, 128, prefix, 1, [1], seed=prefix))
    check(make(40, 4, 2, 1, 128, prefix, 300, [300 if i in (3, 36) else 0 for i in range(40)], seed=prefix))


def test_long_and_uneven():
    """Splits over all SMs: a long prefix, one long suffix among short ones."""
    check(make(5, 4, 1, 1, 128, 9000, 7000, [7000, 1, 30, 500, 0], seed=3))
    check(make(70, 4, 4, 1, 64, 1000, 400, [1 + (91 * i) % 400 for i in range(70)], seed=4))


def test_peaked_logits_and_scale():
    check(make(4, 8, 2, 2, 128, 500, 600, [600, 2, 301, 77], seed=5, mult=4.0))
    check(make(4, 8, 2, 2, 64, 500, 600, [600, 2, 301, 77], seed=6), scale=0.4)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_lies_past_the_lengths(bad):
    args = make(4, 8, 2, 2, 128, 200, 260, [2, 260, 130, 17], seed=7)
    want = vsa().shared_prefix_attn(*args)
    q, kp, vp, ks, vs, lens = args
    for i, n in enumerate(lens.tolist()):
        ks[i, :, n:] = bad
        vs[i, :, n:] = bad
    # the prefix is a slice of a longer cache
    kl, vl = (torch.full((2, 300, 128), bad, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kl[:, :200], vl[:, :200] = kp, vp
    got = vsa().shared_prefix_attn(q, kl[:, :200], vl[:, :200], ks, vs, lens)
    assert torch.equal(got, want)


def test_views():
    """Token-major caches and queries give the contiguous result bit for bit."""
    args = make(5, 10, 2, 3, 128, 300, 200, [3, 200, 100, 64, 5], seed=8)
    want, wlse = check(args)
    q, kp, vp, ks, vs, lens = args
    swap = lambda x: x.transpose(-3, -2).contiguous().transpose(-3, -2)  # noqa: E731
    fused = torch.cat([swap(ks).transpose(1, 2), swap(vs).transpose(1, 2)], 2)
    out = torch.full((5, 3, 10, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    got, glse = vsa().shared_prefix_attn(swap(q), swap(kp), swap(vp), fused[:, :, :2].transpose(1, 2),
                                         fused[:, :, 2:].transpose(1, 2), lens, return_lse=True,
                                         out=out[..., :128].transpose(1, 2))
    assert torch.equal(got, want) and torch.equal(glse, wlse)
    assert (out[..., 128:] == 7).all()


def test_stream_graph_and_lengths_at_replay():
    args = make(6, 8, 2, 1, 128, 300, 256, [10, 20, 30, 40, 50, 60], seed=9)
    want = vsa().shared_prefix_attn(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = vsa().shared_prefix_attn(*args, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(args[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vsa().shared_prefix_attn(*args, out=out)
    vsa().shared_prefix_attn(*make(9, 8, 2, 2, 64, 77, 50, [50] * 9, seed=10))
    for step in (1, 60, 190):
        args[5].add_(step) if step < 190 else args[5].fill_(256)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, vsa().shared_prefix_attn(*args))
        want, _, tol, _ = R.decode(*args)
        R.assert_within(out, want, tol, "out")


def test_repeats_are_equal():
    args = make(17, 20, 4, 1, 128, 2000, 900, [1 + (71 * i) % 900 for i in range(17)], seed=11)
    first = vsa().shared_prefix_attn(*args)
    for _ in range(5):
        assert torch.equal(vsa().shared_prefix_attn(*args), first)


def test_prompt_then_decode():
    """A prompt through the packed attention, then tokens one at a time over its
    cache, against the packed attention of the whole text; and the same rows as
    drafted tokens checked in one call."""
    n, new, hq, hkv, d = 333, 5, 8, 2, 128
    q, k, v = (R.normal((n + new, h, d), 12 + i).transpose(0, 1) for i, h in enumerate((hq, hkv, hkv)))
    want, wlse, tol, tlse = R.forward(q, k, v, [0, n + new], [0, n + new])
    got = vsa().dense_attn_varlen(q[:, :n], k[:, :n], v[:, :n], [0, n], [0, n])
    R.assert_within(got, want[:, :n], tol[:, :n], "prompt")
    ks, vs = (torch.zeros((2, 16, hkv, d), dtype=torch.bfloat16, device="cuda").transpose(1, 2) for _ in range(2))
    for i in range(new):
        ks[:, :, i], vs[:, :, i] = k[:, n + i], v[:, n + i]
        lens = torch.full((2,), i + 1, dtype=torch.int32, device="cuda")
        row = q[None, :, n + i:n + i + 1].expand(2, -1, -1, -1).contiguous()
        out, lse = vsa().shared_prefix_attn(row, k[:, :n], v[:, :n], ks, vs, lens, return_lse=True)
        for b in range(2):
            R.assert_within(out[b], want[:, n + i:n + i + 1], tol[:, n + i:n + i + 1], "token")
            R.assert_within(lse[b], wlse[:, n + i:n + i + 1], tlse[:, n + i:n + i + 1], "token lse")
    lens = torch.full((1,), new, dtype=torch.int32, device="cuda")
    out = vsa().shared_prefix_attn(q[None, :, n:], k[:, :n], v[:, :n], ks[:1], vs[:1], lens)
    R.assert_within(out[0], want[:, n:], tol[:, n:], "drafts")
    vsa().check_device_status()


def test_refusals():
    B = vsa()
    q, kp, vp, ks, vs, lens = make(3, 4, 2, 1, 64, 20, 10, [1, 2, 3], seed=13)
    with pytest.raises(TypeError):
        B.shared_prefix_attn(q, kp, vp, ks, vs, lens.long())
    with pytest.raises(ValueError):
        B.shared_prefix_attn(q, kp, vp, ks, vs, lens.cpu())
    with pytest.raises(ValueError):
        B.shared_prefix_attn(q, kp, vp, ks, vs, lens[:2])
    with pytest.raises(ValueError):
        B.shared_prefix_attn(q, kp, vp, ks[:2], vs[:2], lens)
    with pytest.raises(ValueError):
        B.shared_prefix_attn(q, kp, vp, ks[:1].expand(3, -1, -1, -1), vs, lens)
    with pytest.raises(ValueError):
        B.shared_prefix_attn(q, kp[:, :, :32], vp[:, :, :32], ks, vs, lens)
    with pytest.raises(TypeError):
        B.shared_prefix_attn(q.half(), kp, vp, ks, vs, lens)
    with pytest.raises(B.VSAError):
        B.shared_prefix_attn(q[:, :3], kp, vp, ks, vs, lens)            # 3 heads over 2
    with pytest.raises(B.VSAError):
        B.shared_prefix_attn(q, kp, vp, ks, vs, lens, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert B.get_device_status() == 0
    # a length past the capacity counts as 0 and is reported
    want = B.shared_prefix_attn(q, kp, vp, ks, vs, torch.tensor([1, 0, 3], dtype=torch.int32, device="cuda"))
    for n in (11, -1, 2 ** 31 - 1):
        got = B.shared_prefix_attn(q, kp, vp, ks, vs, torch.tensor([1, n, 3], dtype=torch.int32, device="cuda"))
        assert B.get_device_status() == 6 and torch.equal(got, want)
    assert B.get_device_status() == 0


def test_calls_side_by_side():
    """Two streams at once, each call with a workspace of its own."""
    sets = []
    for seed, shape in ((14, (17, 20, 4, 1, 128, 2000, 900)), (15, (9, 16, 2, 5, 64, 700, 600))):
        cap, t = shape[-1], shape[3]
        args = make(*shape, [t + (71 * i) % (cap - t) for i in range(shape[0])], seed=seed)
        sets.append((args, vsa().shared_prefix_attn(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for args, want, stream in sets:
            got.append((vsa().shared_prefix_attn(*args, stream=stream), want))
    torch.cuda.synchronize()
    vsa().check_device_status()
    for a, b in got:
        assert torch.equal(a, b)
