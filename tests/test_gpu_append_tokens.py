"""The cache append of one token, and of many tokens with several rotary axes, bit-exact against float32 arithmetic."""
import numpy as np
import pytest
import torch

from tests.block_util import bf16
from tests.layer_util import ftmoe
from tests.test_gpu_block_attention import rotate32
from tests.test_gpu_nvfp4_append import Case, i32, rotate_axes32

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "e4m3", "nvfp4"]


def axes_of(m, R):
    """Three axes in turn, the last pairs all on the first."""
    return m.RopeAxes(tuple(i % 3 if i < R // 2 - 3 else 0 for i in range(R // 2)))


def single(D, R, Hq, Hkv, order, kind, at):
    """A case of one token, at place `at` of its sequence."""
    c = Case(D, R, Hq, Hkv, 16, order, kind, T=30, seed=Hq)
    c.T, c.seq, c.pos = 1, c.seq[:1], np.array([at])
    c.wide = bf16(3 * c.rng.standard_normal((1, Hq + 2 * Hkv, D)))
    c.q, c.k, c.v = c.wide[:, :Hq], c.wide[:, Hq:Hq + Hkv], c.wide[:, Hq + Hkv:]
    return c


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,R,Hq,Hkv", [(64, 64, 1, 1), (64, 32, 0, 1), (128, 128, 3, 1), (128, 64, 0, 2), (256, 256, 8, 1),
                                        (256, 0, 2, 2), (128, 128, 40, 8)])
def test_one_token(kind, D, R, Hq, Hkv):
    m = ftmoe()
    for order, at in (("slot", 0), ("head", 17)):
        c = single(D, R, Hq, Hkv, order, kind, at)
        c.run(m, rotate32(c.k, c.rope, c.pos), rotate32(c.q, c.rope, c.pos))
        if R == 0:
            continue
        c = single(D, R, Hq, Hkv, order, kind, at)
        axes, pos = axes_of(m, R), c.rng.integers(0, 64, (3, 1)).astype(np.int32)
        c.run(m, rotate_axes32(c.k, c.rope, pos, axes.axes), rotate_axes32(c.q, c.rope, pos, axes.axes),
              rope_positions=i32(pos), rope_axes=axes)


# tokens of a block on 152 SMs: 3, 3, 8 times 2, 3 (two heads a thread), 21 times 6
MANY = [(1003, 128, 128, 32, 8), (1201, 128, 96, 32, 8), (6001, 64, 64, 4, 2), (2003, 128, 128, 40, 8), (64001, 64, 32, 1, 1)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,D,R,Hq,Hkv", MANY[:4])
def test_axes_of_many_tokens_a_block(kind, T, D, R, Hq, Hkv):
    m = ftmoe()
    c = Case(D, R, Hq, Hkv, 24, "head" if T % 2003 == 0 else "slot", kind, T=T)
    axes = axes_of(m, R)
    pos = c.rng.integers(0, len(c.rope), (3, T)).astype(np.int32)
    pos[:, c.pos < 0] = 1 << 30                          # not looked at for padding
    at = np.where(c.pos < 0, 0, pos)
    c.run(m, rotate_axes32(c.k, c.rope, at, axes.axes), rotate_axes32(c.q, c.rope, at, axes.axes),
          rope_positions=i32(pos), rope_axes=axes)
