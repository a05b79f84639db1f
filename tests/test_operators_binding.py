"""The Python side of the dense-layer and gradient operators, with a library and tensors that stand in for the GPU's."""
import os
import subprocess
import sys
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


def test_workspace_sizes_are_kept_for_each_device(monkeypatch):
    """Plans depend on the number of SMs: a size asked on one device is not another's."""
    on = [0]

    class Lib:
        def vf_linear_workspace(self, dtype, M, N, K, grad, n):
            n._obj.value = 1000 + on[0]
            return vf.VF_OK

    monkeypatch.setattr(vf, "lib", lambda: Lib())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: on[0])
    sizes = (0, 123457, 11, 13, 1)  # asked nowhere else
    assert vf._linear_work(*sizes) == 1000
    on[0] = 1
    assert vf._linear_work(*sizes) == 1001
    on[0] = 0
    assert vf._linear_work(*sizes) == 1000
    vf._linear_work_on.cache_clear()


def test_running_out_of_host_memory_is_an_error_with_a_message():
    """A list of gradients whose table does not fit into what the process may still allocate."""
    code = """
import ctypes, resource
from linear_bound_propagation_b200 import vf
L, n = vf.lib(), 4_000_000
ptrs = (ctypes.c_void_p * n)(*range(1 << 20, (1 << 20) + 16 * n, 16))
sizes, types = (ctypes.c_longlong * n)(*([4] * n)), (ctypes.c_int * n)()
args = (ptrs, ptrs, sizes, types, 1.0, 1.0, 1 << 20, None, 0, None)
assert L.vf_clip_grad_norm(-1, *args) == vf.VF_ERR_ARG  # leaves a message of its own
now = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (now + (48 << 20), resource.RLIM_INFINITY))
rc = L.vf_clip_grad_norm(n, *args)
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
assert rc == vf.VF_ERR_CUDA, rc
assert b"alloc" in L.vf_last_error(), L.vf_last_error()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("M,N,K", [(1, (1 << 32) + 8, 1), (1, 8, (1 << 32) + 8), (2, 1 << 31, 4)])
def test_sizes_that_a_c_int_would_wrap_are_refused(M, N, K):
    """2^32 + 8 rows of W would arrive as 8: the rest of the output would be left as it was."""

    class OnGpu(torch.Tensor):
        def get_device(self):
            return 0

    x, W = (torch.empty(s, device="meta", dtype=torch.bfloat16).as_subclass(OnGpu) for s in ((M, K), (N, K)))
    with pytest.raises(ValueError, match="below 2.31"):
        vf._layer(x, W, "none")
    if N <= 8:
        with pytest.raises(ValueError, match="below 2.31"):
            vf._layer(W, x, "relu")
    x, W = (torch.empty(s, device="meta", dtype=torch.bfloat16).as_subclass(OnGpu) for s in ((1 << 33, 3), (vf.MAX_EXTENT, 3)))
    assert vf._layer(x, W, "none")[4:] == (1 << 33, vf.MAX_EXTENT, 3)  # rows are a long long: left to the library
