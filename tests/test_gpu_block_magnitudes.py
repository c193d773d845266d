"""The norm and its gradient for rows far from magnitude one, as far as a row's squares stay inside float32
(a root mean square of about 1e-18 to 3e17 for rows of 4096).

Tolerance as for the other norm tests: 2^-18 of the sum of magnitudes (2^-17 for column sums), then one
rounding to the output's type.
"""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.block_util import bf16, close, f64
from tests.layer_util import ftmoe
from tests.test_gpu_block_norm import REL

pytestmark = pytest.mark.gpu
F32 = torch.float32


def check(H, size_y, size_r, size_d, eps, gate, seed, res=F32):
    m = ftmoe()
    rng = np.random.default_rng(seed)
    T, n = 7, rng.standard_normal
    shape = {"none": None, "token": (T, 1), "channel": (H,)}[gate]
    a = dict(y=bf16(size_y * n((T, H))), r=torch.from_numpy(size_r * n((T, H))).to(res),
             w_post=bf16(1 + 0.2 * n(H)), w_pre=bf16(1 + 0.2 * n(H)), gate=bf16(n(shape)) if shape else None,
             dr=torch.from_numpy(size_d / max(size_r, 1) * n((T, H))).to(res), dx=bf16(size_d * n((T, H))))
    d = {k: None if t is None else t.cuda() for k, t in a.items()}
    kw = dict(w_post=d["w_post"], w_pre=d["w_pre"], gate=d["gate"], scale=0.7, eps=eps)
    args = [f64(a[k]) for k in ("y", "r")]
    tail = [f64(a[k]) for k in ("w_post", "w_pre", "gate")] + [0.7, eps]
    r, x = m.residual_norm(d["y"], d["r"], **kw)
    ref, rx = ob.residual_norm(*args, *tail)
    mag = np.abs(ref) + 2 * np.abs(args[1])
    close(r, ref, mag, REL, "r'")
    s2 = 1 / np.sqrt((ref ** 2).mean(1, keepdims=True) + eps)
    close(x, rx, mag * s2 * np.abs(tail[1]), REL, "x'")
    g = m.residual_norm_backward(d["y"], d["r"], d["dr"], d["dx"], **kw)
    ref, mag = ob.residual_norm_backward(*args, f64(a["dr"]), f64(a["dx"]), *tail)
    if gate != "none":
        axis = dict(axis=0) if gate == "channel" else dict(axis=1, keepdims=True)
        ref["dgate"], mag["dgate"] = ref["dgate"].sum(**axis), mag["dgate"].sum(**axis)
    for name in ("dresidual", "dy", "dw_post", "dw_pre", "dgate"):
        if name != "dgate" or gate != "none":
            close(getattr(g, name), ref[name], mag[name], 2 * REL if name.startswith(("dw", "dg")) else REL, name)


@pytest.mark.parametrize("H", [64, 200, 520, 1032, 4096, 8200])
@pytest.mark.parametrize("size,eps", [(1e-17, 0.0), (1e-14, 0.0), (1e-9, 0.0), (1e-4, 1e-6), (1e4, 1e-6), (1e9, 1e-6),
                                      (1e12, 1e-6), (1e14, 1e-6), (1e15, 1e-6), (1e16, 1e-6), (1e17, 1e-6)])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
def test_large_and_small_rows_after_a_block(H, size, eps, gate):
    """y of any size: its norm is of magnitude one, the gradient of y the smaller the larger y."""
    check(H, size, 1.0, 1.0, eps, gate, H)
    check(H, size, 1.0, 1e-4, eps, gate, H + 1)


@pytest.mark.parametrize("H", [64, 520, 4096])
@pytest.mark.parametrize("size,eps", [(1e4, 1e-6), (1e9, 1e-6), (1e14, 1e-6), (1e16, 1e-6), (1e17, 1e-6)])
def test_a_large_residual_stream(H, size, eps):
    """The norm before the next block divides by the stream's size."""
    check(H, 1.0, size, 1.0, eps, "none", H)
    check(H, size, size, 1e-3, eps, "token", H + 1)
