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


@pytest.mark.parametrize("H,gate,res,T", [(64, "token", torch.bfloat16, 10037), (128, "element", torch.float32, 9001),
                                          (256, "none", torch.bfloat16, 5003), (504, "channel", torch.float32, 9001),
                                          (520, "element", torch.bfloat16, 4001), (1032, "token", torch.float32, 4001),
                                          (4096, "channel", torch.bfloat16, 1500), (4096, "element", torch.float32, 1500),
                                          (8192, "none", torch.bfloat16, 700), (8192, "element", torch.float32, 700),
                                          (16384, "none", torch.bfloat16, 500), (16384, "element", torch.float32, 500)])
@pytest.mark.parametrize("onto", ["y", "dx"])
def test_gradients_in_place(H, gate, res, T, onto):
    """dresidual over d_r, dy over y or d_x, with several rows a group and one to eight stages of them."""
    m = ftmoe()
    d = {n: cuda(t) for n, t in inputs(np.random.default_rng(H + T), T, H, res, True, True, gate).items()}
    want = m.residual_norm_backward(d["y"], d["r"], d["dr"], d["dx"], w_post=d["w_post"], w_pre=d["w_pre"],
                                    gate=d["gate"], scale=0.7, eps=1e-5)
    sums = [torch.empty_like(t) for t in (want.dw_post, want.dw_pre)]
    dgate = None if want.dgate is None else torch.empty_like(want.dgate)
    backward(m, d, gate, d[onto], d["dr"], *sums, dgate, d["dx"])
    for a, b in zip([d[onto], d["dr"], *sums, dgate], want):
        assert (a is None and b is None) or torch.equal(a, b)
