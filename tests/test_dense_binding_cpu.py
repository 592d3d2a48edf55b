"""Host checks of the dense entries' binding (no GPU)."""
import numpy as np
import pytest
import torch

from block_sparse_attention_15_b200 import binding as B


@pytest.mark.parametrize("xs", [[0, 5, 12], (0, 5, 12), np.array([0, 5, 12]), np.array([0, 5, 12], dtype=np.uint8),
                                torch.tensor([0, 5, 12]), torch.tensor([0, 5, 12], dtype=torch.int32),
                                [np.int64(0), torch.tensor(5), 12], range(0, 3)])
def test_cumulative_lengths(xs):
    got = B._cumulative(xs, "cu")
    assert got.typecode == "i" and list(got) == ([0, 1, 2] if isinstance(xs, range) else [0, 5, 12])


@pytest.mark.parametrize("xs", [[0, 10.7], (0, 5.0), np.array([0.0, 10.7]), torch.tensor([0.0, 10.7]),
                                [torch.tensor(0), torch.tensor(10.7)], np.array([False, True])])
def test_cumulative_lengths_that_are_no_integers(xs):
    with pytest.raises(TypeError):
        B._cumulative(xs, "cu")


@pytest.mark.parametrize("xs", [[0, 2 ** 32 + 10], np.array([0, 2 ** 32 + 10]), torch.tensor([0, 2 ** 32 + 10]),
                                np.array([0, 2 ** 31]), np.array([0, 2 ** 64 - 1], dtype=np.uint64), [[0, 5]],
                                np.zeros((1, 2), dtype=np.int32)])
def test_cumulative_lengths_out_of_range(xs):
    """64-bit values must not wrap into valid ones."""
    with pytest.raises(ValueError):
        B._cumulative(xs, "cu")


def test_stream_of_another_device():
    """Refused before anything is allocated or launched."""
    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    calls = []
    with pytest.raises(ValueError):
        B._on(0, Stream(), calls.append)
    assert not calls


def test_workspace_must_be_contiguous():
    """The bytes of an expanded or strided view are not all there."""
    like = torch.empty(1)
    for bad in (torch.empty(1, dtype=torch.uint8).expand(1 << 20), torch.empty(64, 64)[:, ::2]):
        with pytest.raises(ValueError):
            B._workspace(bad, 0, like)
    ws = torch.empty(100, dtype=torch.float32)
    assert B._workspace(ws, 0, like) == (ws, ws.data_ptr(), 400)
