"""The decode block's C entry points in forms that the binding does not use."""
import ctypes

import numpy as np
import pytest
import torch

from tests.layer_util import ftmoe
from tests.test_gpu_block_norm import cuda, inputs

pytestmark = pytest.mark.gpu
KIND = {"none": 0, "channel": 1, "token": 2, "element": 3}


def workspace(m, T, H):
    n = m.lib().ft_residual_norm_backward_workspace_bytes(T, H)
    ws = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    return ws[(-ws.data_ptr()) % 256:][:n]


def backward(m, d, gate, dy, dres, dw_post, dw_pre, dgate, d_x, scale=0.7, eps=1e-5):
    """ft_residual_norm_backward on tensors; None is NULL."""
    T, H = d["y"].shape
    p = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    ws = workspace(m, T, H)
    st = m.lib().ft_residual_norm_backward(
        p(d["y"]), p(d["r"]), p(d["w_post"]), p(d["w_pre"]), p(d["gate"]), KIND[gate], p(d["dr"]), p(d_x), T, H,
        int(dres.dtype == torch.float32), ctypes.c_float(scale), ctypes.c_float(eps), p(dy), p(dres), p(dw_post),
        p(dw_pre), p(dgate), p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert m.get_error(ws) == 0


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,gate", [(64, "token"), (256, "channel"), (264, "none"), (520, "element"), (1032, "token"),
                                    (4096, "channel"), (8192, "none"), (16384, "element")])
def test_a_gradient_of_x_without_its_weight_is_ignored(H, gate, res):
    m = ftmoe()
    d = {n: cuda(t) for n, t in inputs(np.random.default_rng(H), 331, H, res, True, False, gate).items()}
    want = m.residual_norm_backward(d["y"], d["r"], d["dr"], w_post=d["w_post"], gate=d["gate"], scale=0.7, eps=1e-5)
    got = [torch.full_like(t, float("nan")) for t in (want.dy, want.dresidual, want.dw_post)]
    dgate = None if want.dgate is None else torch.full_like(want.dgate, float("nan"))
    backward(m, d, gate, *got, None, dgate, torch.full_like(d["y"], float("nan")))
    for a, b in zip([*got, dgate], (want.dy, want.dresidual, want.dw_post, want.dgate)):
        assert (a is None and b is None) or torch.equal(a, b)
