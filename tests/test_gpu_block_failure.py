"""Expired waits of the decode block's kernels: the test hook makes every wait for an asynchronous copy give
up at once. The kernel must say so (the error word, or NaN rows where the call has no workspace), return
soon, and leave the next call as ever."""
import time

import numpy as np
import pytest
import torch

from tests.block_util import bf16
from tests.layer_util import ftmoe
from tests.test_gpu_block_linear import matrix, on_gpu
from tests.test_gpu_block_norm import cuda, inputs

pytestmark = pytest.mark.gpu
FT_ERR_TIMEOUT = 7


def zeroed(n):
    ws = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    return ws[(-ws.data_ptr()) % 256:][:n]


def without_waits(m, call):
    """call() with the hook set; the seconds until the GPU is done."""
    torch.cuda.synchronize()
    try:
        m.debug_set_wait_limit(0)
        begin = time.perf_counter()
        got = call()
        torch.cuda.synchronize()
        return got, time.perf_counter() - begin
    finally:
        m.debug_set_wait_limit(None)


@pytest.mark.parametrize("T", [12, 30, 48, 64])
def test_dense_product(T):
    m = ftmoe()
    rng = np.random.default_rng(T)
    lin, x = on_gpu(m, *matrix(rng, 12011, 4096)), bf16(rng.standard_normal((T, 4096))).cuda()
    ws = zeroed(m.nvfp4_linear_workspace_bytes(T, 4096))
    want = m.nvfp4_linear(x, lin, workspace=ws)
    assert m.get_error(ws) == 0
    _, seconds = without_waits(m, lambda: m.nvfp4_linear(x, lin, workspace=ws))
    assert seconds < 1 and m.get_error(ws) == FT_ERR_TIMEOUT and m.get_error(ws) == 0
    assert torch.equal(m.nvfp4_linear(x, lin, workspace=ws), want) and m.get_error(ws) == 0


@pytest.mark.parametrize("T,H,res", [(2600, 4096, torch.float32), (1300, 8192, torch.bfloat16), (700, 16384, torch.float32)])
@pytest.mark.parametrize("post", [True, False])
def test_norm(T, H, res, post):
    m = ftmoe()
    d = {n: cuda(t) for n, t in inputs(np.random.default_rng(T), T, H, res, post, True, "none").items()}
    call = lambda: m.residual_norm(d["y"], d["r"], w_post=d["w_post"], w_pre=d["w_pre"])  # noqa: E731
    want = call()
    got, seconds = without_waits(m, call)
    assert seconds < 1 and all(torch.isnan(t).all() for t in got)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))


@pytest.mark.parametrize("T,H,res,gate", [(9001, 504, torch.bfloat16, "none"), (3000, 1032, torch.float32, "token"),
                                          (1500, 4096, torch.bfloat16, "channel"), (700, 8192, torch.float32, "element"),
                                          (400, 16384, torch.float32, "element")])
@pytest.mark.parametrize("pre", [True, False])
def test_gradient(T, H, res, gate, pre):
    m = ftmoe()
    d = {n: cuda(t) for n, t in inputs(np.random.default_rng(T), T, H, res, True, pre, gate).items()}
    ws = zeroed(m.lib().ft_residual_norm_backward_workspace_bytes(T, H))

    def call():
        return m.residual_norm_backward(d["y"], d["r"], d["dr"], d["dx"] if pre else None, w_post=d["w_post"],
                                        w_pre=d["w_pre"], gate=d["gate"], workspace=ws)

    want = call()
    assert m.get_error(ws) == 0
    _, seconds = without_waits(m, call)
    assert seconds < 1 and m.get_error(ws) == FT_ERR_TIMEOUT
    for a, b in zip(call(), want):
        assert (a is None and b is None) or torch.equal(a, b)
    assert m.get_error(ws) == 0
