"""The attention kernels' bounded waits: a ring whose consumer gets stuck ends by itself, with no copy
issued into a place that was not handed back, and leaves the GPU as usable as before."""
import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_linear_09_gb300 import build as gbuild
    os.makedirs(os.path.join(HERE, "_build"), exist_ok=True)
    so = os.path.join(HERE, "_build", "libattnwaits.so")
    subprocess.run([gbuild.nvcc()] + gbuild.flags() + ["-shared", "-o", so, os.path.join(HERE, "csrc", "attn_wait_selftest.cu")],
                   check=True)
    l = ctypes.CDLL(so)
    l.attn_ring.restype = ctypes.c_int
    l.attn_ring.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    return l


@pytest.mark.parametrize("stuck_at,issued,sums", [(-1, 8, 32), (3, 5, 18), (0, 2, 6)])
def test_a_stuck_ring_ends(lib, stuck_at, issued, sums):
    """A warp that stops at tile t keeps its stage: tiles up to t + 1 are issued and, by the other three, read."""
    src = torch.arange(8, device="cuda").repeat_interleave(256).float()
    for _ in range(2):
        status, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
        assert lib.attn_ring(src.data_ptr(), 8, stuck_at, status.data_ptr(), out.data_ptr()) == 0
        assert int(status.item()) == (0 if stuck_at < 0 else 4)
        assert out.tolist() == [issued, 0 if stuck_at < 0 else 4, sums]
