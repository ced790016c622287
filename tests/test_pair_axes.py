"""What the binding takes for the axes of channel pairs: bytes or a sequence of numbers, not a number of zeros."""
import ctypes

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from query_aware_sparse_append_gb300 import build
    build.build()
    from query_aware_sparse_append_gb300 import binding
    return binding


POS = torch.zeros((2, 1, 2), dtype=torch.int32)


@pytest.mark.parametrize("axes", [32, np.int64(32), torch.tensor(32), True, 1.5, "0" * 32, ["0"] * 32, [0.0] * 32, [None] * 32,
                                  [300] + [0] * 31, torch.zeros(32)])
def test_refused(lib, axes):
    with pytest.raises(ValueError, match="pair_axes"):
        lib._positions(POS, axes, 1, 2, 32, -1)


@pytest.mark.parametrize("axes", [[0, 1] * 16, (0, 1) * 16, bytes([0, 1] * 16), bytearray([0, 1] * 16), iter([0, 1] * 16),
                                  np.array([0, 1] * 16), np.array([0, 1] * 16, dtype=np.uint8), torch.tensor([0, 1] * 16),
                                  torch.tensor([0, 1] * 16, dtype=torch.uint8)])
def test_taken(lib, axes):
    got = lib._positions(POS, axes, 1, 2, 32, -1)
    at = ctypes.c_void_p.from_buffer(got, lib._Positions.pair_axes.offset).value
    assert ctypes.string_at(at, 32) == bytes([0, 1] * 16) and got.num_axes == 2
