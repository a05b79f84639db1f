"""The Python side of the dense-layer and gradient operators, with a library and tensors that stand in for the GPU's."""
import types

import pytest
import torch

from linear_bound_propagation_b200 import vf


class Tensor:
    """Counts the streams it is recorded on."""

    def __init__(self):
        self.streams = []

    def record_stream(self, s):
        self.streams.append(s)


def test_tensors_are_recorded_on_the_stream_that_is_given():
    a, b = Tensor(), Tensor()
    vf._used_on(None, a, None, b)
    assert a.streams == b.streams == []
    vf._used_on("s", a, None, b)
    assert a.streams == b.streams == ["s"]


def test_a_stream_of_another_device_is_refused():
    """It would be left for the tensors' device, and the call would run on that device's current stream."""
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        vf._On(0, other)
