"""Rows and keys whose offsets pass 2^31 elements (a few GB a tensor)."""
import pytest
import torch

from . import dense_norms as N
from . import dense_ref as R
from .test_gpu_dense import vsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("token_major", [True, False])
def test_packed_rows_far_out(token_major):
    """A long sequence without keys, whose rows become 0, before one with."""
    hq, hkv, d, far, n, keys = 32, 8, 128, 560000, 200, 300
    assert hq * far * d > 2 ** 31

    def rows(h, count, filled):
        x = torch.empty((count, h, d) if token_major else (h, count, d), dtype=torch.bfloat16, device="cuda")
        x = x.transpose(0, 1) if token_major else x
        x[:, count - filled:] = R.normal((h, filled, d), h + filled)
        return x

    q, dout = rows(hq, far, n), rows(hq, far, n)
    dout[:, far - n:] = R.normal((hq, n, d), 77)
    k, v = rows(hkv, keys, keys), rows(hkv, keys, keys)
    v[:] = R.normal((hkv, keys, d), 78)
    cu_q, cu_kv = [0, far - n, far], [0, 0, keys]
    out, lse = vsa().dense_attn_varlen(q, k, v, cu_q, cu_kv, return_lse=True)
    grads = vsa().dense_attn_varlen_backward(q, k, v, out, dout, lse, cu_q, cu_kv)
    vsa().check_device_status()
    tail = slice(far - n, far)
    small = (q[:, tail], k, v, [0, n], [0, keys], True)
    N.assert_close(out[:, tail], N.attention64(*small), [0, n], "out")
    want = N.attention64(*small, dout[:, tail])
    for name, x, y, cu in zip(("dq", "dk", "dv"), (grads[0][:, tail], *grads[1:]), want, ([0, n], [0, keys], [0, keys])):
        N.assert_close(x, y, cu, name)
    for x in (out, grads[0]):
        assert not x[:, :far - n].any()
    assert (lse[:, :far - n] == -float("inf")).all()


@pytest.mark.parametrize("token_major", [True, False])
def test_caches_far_out(token_major):
    b, hq, hkv, d, cap = 4, 16, 8, 128, 600000
    assert b * hkv * cap * d > 2 ** 31
    lens = [5, 599990, 0, 20000]

    def cache(seed):
        x = torch.empty((b, cap, hkv, d) if token_major else (b, hkv, cap, d), dtype=torch.bfloat16, device="cuda")
        x = x.transpose(1, 2) if token_major else x
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for i, n in enumerate(lens):
            for h in range(hkv):
                x[i, h, :n] = torch.randn((n, d), generator=gen, device="cuda").to(torch.bfloat16)
        return x

    q, ks, vs = R.normal((b, hq, 1, d), 5), cache(6), cache(7)
    kp, vp = R.normal((hkv, 130, d), 8), R.normal((hkv, 130, d), 9)
    out = vsa().shared_prefix_attn(q, kp, vp, ks, vs, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    vsa().check_device_status()
    for i, n in enumerate(lens):
        k, v = torch.cat([kp, ks[i, :, :n]], 1), torch.cat([vp, vs[i, :, :n]], 1)
        N.assert_close(out[i], N.attention64(q[i], k, v, [0, 1], [0, 130 + n], True), [0, 1], f"request {i}")
