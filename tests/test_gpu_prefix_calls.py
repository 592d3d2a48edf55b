"""Forms of the shared_prefix_attn call beside those of test_gpu_prefix."""
import pytest
import torch

from .test_gpu_prefix import check, make, vsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_no_prefix_given(d):
    q, kp, vp, ks, vs, lens = make(5, 8, 2, 2, d, 0, 300, [2, 300, 128, 1, 0], seed=d)
    want, wlse = check((q, kp, vp, ks, vs, lens))
    got, lse = vsa().shared_prefix_attn(q, None, None, ks, vs, lens, return_lse=True)
    assert torch.equal(got, want) and torch.equal(lse, wlse)
    for a, b in ((kp, None), (None, vp)):
        with pytest.raises(TypeError):
            vsa().shared_prefix_attn(q, a, b, ks, vs, lens)
    with pytest.raises(vsa().VSAError):
        vsa().shared_prefix_attn(q[:, :7], None, None, ks, vs, lens)  # 7 heads over 2


@pytest.mark.parametrize("prefix", [0, 130])
@pytest.mark.parametrize("b", [511, 512, 1025, 2100])
@pytest.mark.parametrize("d", [64, 128])
def test_many_requests(d, b, prefix):
    """Around the number of requests from which on their tiles are counted by a
    kernel of its own, and past its block of 1024; runs of requests without keys."""
    t = 1 + b % 2
    lens = [0 if i % 64 > 50 or i > b - 20 else (37 * i) % 301 for i in range(b)]
    check(make(b, 2, 1, t, d, prefix, 300, lens, seed=b + d))


def test_many_requests_behind_a_long_block():
    """Blocks of the prefix and of a request's rows that count twice."""
    check(make(600, 16, 1, 9, 64, 300, 140, [(11 * i) % 141 for i in range(600)], seed=21))


def test_lengths_of_many_requests_at_replay():
    args = make(700, 4, 2, 1, 64, 50, 200, [1 + i % 200 for i in range(700)], seed=22)
    out = torch.zeros_like(args[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vsa().shared_prefix_attn(*args, out=out)
    for step in (3, 50):
        args[5].copy_((args[5] * step) % 201)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, vsa().shared_prefix_attn(*args))
    check(args)


def test_time_grows_with_the_batch_not_with_its_square():
    """65536 short requests may cost three times as much each as 4096 of them (they
    did eight times when every warp added up all lengths)."""
    per_request = []
    for b in (4096, 65536):
        q = torch.zeros((b, 8, 1, 64), dtype=torch.bfloat16, device="cuda")
        kv = torch.zeros((b, 1, 100, 64), dtype=torch.bfloat16, device="cuda")
        lens = torch.full((b,), 100, dtype=torch.int32, device="cuda")
        times = []
        for _ in range(7):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            vsa().shared_prefix_attn(q, None, None, kv, kv, lens)
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end))
        per_request.append(sorted(times)[3] / b)
    assert per_request[1] < 3 * per_request[0], per_request
