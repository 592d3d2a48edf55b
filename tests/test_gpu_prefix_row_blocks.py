"""shared_prefix_attn where blocks of 256 rows and smaller ones follow each other
in one CTA's work: requests of more than 256 rows to a key head, behind prefixes
and not, whose smaller blocks have one, two or three key tiles.  Results are
compared with the reference and, over many calls, with themselves: a tile of
query rows given free too early shows in some calls only."""
import pytest
import torch

from . import dense_ref as R
from .test_gpu_prefix import check, make, vsa

pytestmark = pytest.mark.gpu

# (requests, query heads, key heads, tokens, prefix, capacity)
SHAPES = {
    "256_and_44_rows": (37, 12, 2, 50, 0, 250),
    "5_blocks_and_120_rows": (14, 28, 4, 200, 1, 316),
    "12_blocks_and_128_rows": (20, 32, 2, 200, 0, 539),
    "prefix_256_and_64_rows": (64, 40, 8, 1, 700, 250),
    "prefix_and_own_blocks": (9, 16, 2, 33, 300, 200),
}


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("d", [64, 128])
def test_row_blocks(d, shape):
    b, hq, hkv, t, prefix, cap = SHAPES[shape]
    # one, two and three key tiles, two most often; now and then fewer keys than tokens, or none
    lens = [0 if i % 13 == 12 else min(cap, (130 + 31 * i % 120, 30 + 7 * i % 90, 140 + 17 * i % 110, 257 + i)[i % 4])
            for i in range(b)]
    args = make(b, hq, hkv, t, d, prefix, cap, lens, seed=d + b)
    first, _ = vsa().shared_prefix_attn(*args, return_lse=True)
    for _ in range(60):
        assert torch.equal(vsa().shared_prefix_attn(*args), first)
    got, _ = check(args)
    assert torch.equal(got, first)


def test_row_blocks_beside_other_work():
    """The same while another stream streams through memory."""
    b, hq, hkv, t, prefix, cap = SHAPES["5_blocks_and_120_rows"]
    args = make(b, hq, hkv, t, 64, prefix, cap, [130 + 31 * i % 120 for i in range(b)], seed=3)
    want, _, tol, _ = R.decode(*args)
    a = torch.zeros(1 << 28, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(40):
        with torch.cuda.stream(side):
            a.add_(1.0)
        got.append(vsa().shared_prefix_attn(*args))
    torch.cuda.synchronize()
    vsa().check_device_status()
    R.assert_within(got[0], want, tol, "out")
    assert all(torch.equal(x, got[0]) for x in got)
