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
