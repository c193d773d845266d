"""Calls of different kinds on one workspace, one after the other: a prompt and then decode steps, block-FP8
and NVFP4 layers, the decode block's calls between them. Each gives the bits that it gives alone."""
import numpy as np
import pytest
import torch

from synth import LayerSpec, make_layer
from tests.block_util import bf16
from tests.layer_util import bf16_tensor, experts_to_device, ftmoe
from tests.test_gpu_block_linear import matrix, on_gpu
from tests.test_gpu_fp8block import _to_device as fp8_to_device

pytestmark = pytest.mark.gpu


def layer_calls(m):
    """name -> (call(workspace), workspace bytes)."""
    made = {}
    for name, T in (("one", 1), ("few", 24), ("prompt", 90)):
        spec = LayerSpec(f"sw_{name}", seed=140 + T, T=T, E=20, k=5, H=512, I=256, shared=True)
        layer = make_layer(spec)
        ex, sh = experts_to_device(layer)
        x = bf16_tensor(layer.x)
        idx, w = m.route(torch.from_numpy(layer.logits).cuda(), spec.k)
        n = lambda p: m.workspace_bytes(T, spec.k, spec.E, spec.H, spec.I, True, p)  # noqa: E731
        made["prefill " + name] = (lambda ws, a=(x, idx, w, ex, sh): m.prefill(*a, workspace=ws), n(True))
        if T <= 64:
            made["decode " + name] = (lambda ws, a=(x, idx, w, ex, sh): m.decode(*a, workspace=ws), n(False))
    spec = LayerSpec("sw_f8", seed=150, T=7, E=8, k=2, H=256, I=128, fmt="fp8block")
    layer = make_layer(spec)
    ex, sh = fp8_to_device(layer)
    x = bf16_tensor(layer.x)
    idx, w = m.route(torch.from_numpy(layer.logits).cuda(), spec.k)
    made["fp8"] = (lambda ws: m.fp8block_decode(x, idx, w, ex, sh, workspace=ws),
                   m.new_fp8block_workspace(spec.T, spec.k, ex, sh is not None).numel())
    rng = np.random.default_rng(9)
    lin, xl = on_gpu(m, *matrix(rng, 300, 512)), bf16(rng.standard_normal((20, 512))).cuda()
    made["linear"] = (lambda ws: m.nvfp4_linear(xl, lin, workspace=ws), m.nvfp4_linear_workspace_bytes(20, 512))
    return made


def test_calls_of_every_kind_share_a_workspace():
    m = ftmoe()
    calls = layer_calls(m)
    want = {}
    for name, (call, n) in calls.items():
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        want[name] = call(ws).clone()
        assert m.get_error(ws) == 0
    shared = torch.zeros(max(n for _, n in calls.values()), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(3)
    order = [name for first in calls for second in calls for name in (first, second)]
    order += list(rng.permutation(order))
    for ws in (shared, None):
        for i, name in enumerate(order):
            got = calls[name][0](ws)
            assert torch.equal(got.view(torch.int16), want[name].view(torch.int16)), (i, order[max(0, i - 1)], name)
            assert m.get_error(ws) == 0, (i, name)
