"""A caller's workspace is memory of the tensors' device in one piece: anything else
is refused before its address reaches a kernel (the device is only a name here)."""

import pytest
import torch

from paged_recurrent_state_amd import _lib

GPU = torch.device("cuda", 0)


def test_memory_of_another_device():
    for n in (64, 1 << 20):
        with pytest.raises(ValueError, match="expected cuda:0"):
            _lib._workspace(torch.empty(n, dtype=torch.uint8), 64, GPU)


def test_not_a_tensor():
    for ws in (b"\0" * 4096, 4096, [0] * 4096):
        with pytest.raises(TypeError):
            _lib._workspace(ws, 64, GPU)


def test_pieces_and_sizes():
    cpu = torch.device("cpu")
    ws = torch.empty(64, 64, dtype=torch.float32)
    assert _lib._workspace(ws, 64 * 64 * 4, cpu) is ws
    for bad in (ws[:, :32], ws.t(), ws[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            _lib._workspace(bad, 64, cpu)
    with pytest.raises(ValueError, match="needs"):
        _lib._workspace(ws, 64 * 64 * 4 + 1, cpu)
