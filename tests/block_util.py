"""Helpers of the decode-block tests: tensors from a seed, and the comparison with float64.

`close(got, ref, mag, rel)`: every element of `got` within one rounding to its stored type
(2^-8 of the value for bf16, 2^-24 for float32, a little slack for a value that float32 arithmetic
moved over a tie) plus `rel` times `mag`, the sum of magnitudes behind it.
"""
import numpy as np
import torch

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def close(got, ref, mag, rel, what=""):
    g = got.detach().double().cpu().numpy()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    bound = 1.02 * ROUND[got.dtype] * np.abs(ref) + rel * mag + 1e-37
    off = np.abs(g - ref)
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(off / bound):.3g} "
                           f"times the bound, first at {np.argwhere(bad)[0]}")


def bf16(a):
    """float array -> bf16 CPU tensor."""
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16()


def f64(t):
    return None if t is None else t.double().cpu().numpy()
