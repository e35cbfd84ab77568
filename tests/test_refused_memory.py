"""A call whose workspace the device has no memory for is refused, and leaves nothing behind: the next calls are judged by
their own launches alone.  The workspaces asked for are terabytes, more than the device has, so nothing is launched by the refused
calls; their tensors are addresses that no kernel sees."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
WORKSPACE, BF16, FP32 = 6, 0, 1


def P(i):
    return ctypes.c_void_p(i << 44)   # far enough apart for tensors of terabytes


def test_calls_behind_a_refused_one(cuda_lib):
    na = cuda_lib
    lib, rows = na.load(), 2 ** 31 - 256
    assert na.na_glu_bwd_workspace_size(rows, 8, 256) > 2 << 40
    x, y = torch.randn(64, 256, device="cuda"), torch.empty(64, 256, device="cuda")
    w = torch.randn(64, 256, device="cuda")
    h, want = torch.empty(64, 64, device="cuda"), torch.empty(64, 64, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    na.na_glu(x, w, w, want)
    refused = {
        "na_glu_bwd": lambda: lib.na_glu_bwd(*(P(i) for i in range(1, 7)), P(7), P(8), P(9), P(10), P(11), rows, 8, 256, 0, BF16, None, 0, stream),
        "na_glu": lambda: lib.na_glu(*(P(i) for i in range(1, 7)), rows, 511, 1, 0, BF16, stream),   # copies of the tokens
    }
    for name, call in refused.items():
        assert call() == WORKSPACE, name
        na.na_glu(x, w, w, h)           # raises where the launch is reported as failed
        assert torch.equal(h, want)
        assert call() == WORKSPACE, name
        na.na_layernorm(x, None, None, y)
    torch.cuda.synchronize()
    st, raw = na.na_device_status()
    assert st == 0, hex(raw)
