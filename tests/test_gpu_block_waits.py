"""The block norm's bounded wait: a row whose copy never comes leaves NaN in that row and the CTA's later ones, the other
rows as ever, and the GPU as usable as before."""
import ctypes
import os
import subprocess

import pytest
import torch

from gated_deltanet_linear_09_gb300 import build as gbuild
from gated_deltanet_linear_09_gb300 import gdn, runtime

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib():
    os.makedirs(os.path.join(HERE, "_build"), exist_ok=True)
    so = os.path.join(HERE, "_build", "libblockwaits.so")
    subprocess.run([gbuild.nvcc()] + gbuild.flags() + ["-shared", "-o", so, os.path.join(HERE, "csrc", "block_wait_selftest.cu")],
                   check=True)
    l = ctypes.CDLL(so)
    l.block_rows.restype = ctypes.c_int
    l.block_rows.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_ulonglong, ctypes.c_void_p]
    return l


@pytest.mark.parametrize("lost,parts", [(None, "all"), (0, "all"), (11, "all"), (38, "all"), (11, "total"), (11, "y")])
def test_a_lost_row(lib, lost, parts):
    rows, n = 40, 1032
    g = torch.Generator().manual_seed(rows)
    x, r = ((torch.randn((rows, n), generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    w = (0.1 * torch.randn(n, generator=g)).to(torch.bfloat16).cuda()
    pre = None if parts == "total" else w
    post = None if parts == "y" else w
    want = [t.clone() if t is not None else None for t in runtime.block_norm(x, post, residual=r, pre=pre, weight_offset=1.0)]
    outs = [torch.zeros_like(x) if keep else None for keep in (parts != "y", parts != "total")]
    ptrs = [None if t is None else t.data_ptr() for t in outs]
    a = gdn.gdn_block_args(x=x.data_ptr(), residual=r.data_ptr(), post=None if post is None else post.data_ptr(),
                           pre=None if pre is None else pre.data_ptr(), x_ld=n, residual_ld=n, total=ptrs[0], y=ptrs[1], scale=1.0,
                           weight_offset=1.0, eps=1e-6, group=n)
    ctas = ctypes.c_int(0)
    torch.cuda.synchronize()
    assert lib.block_rows(ctypes.byref(a), rows, n, 0 if lost is None else x[lost].data_ptr(), ctypes.byref(ctas)) == 0
    gone = torch.zeros(rows, dtype=torch.bool)
    if lost is not None:
        gone[lost::ctas.value] = True
    for got, exp in zip(outs, want):
        if got is not None:
            assert bool(got[gone.cuda()].isnan().all())
            assert torch.allclose(got[~gone.cuda()].float(), exp[~gone.cuda()].float(), rtol=2.0 ** -7, atol=1e-6)
    assert bool(runtime.block_norm(x, w)[0].isfinite().all())
