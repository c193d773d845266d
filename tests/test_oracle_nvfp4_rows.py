"""The oracle of NVFP4 cache rows and of rotary axes, on the CPU: against torch's E4M3, hand-made blocks and
the one-axis rotation."""
import numpy as np
import pytest
import torch

from oracle import block as ob
from oracle.nvfp4 import E2M1_VALUES, E4M3_VALUES


def test_nearest_e4m3_is_torchs():
    rng = np.random.default_rng(0)
    v = np.abs(rng.standard_normal(5000).astype(np.float32)) * 2.0 ** rng.integers(-12, 9, 5000).astype(np.float32)
    mid = ((E4M3_VALUES[:126].astype(np.float64) + E4M3_VALUES[1:127]) / 2).astype(np.float32)
    v = np.minimum(np.concatenate([v, mid, E4M3_VALUES[:127]]), 448)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ob._nearest(v, E4M3_VALUES[:127]), want)
    assert np.array_equal(ob._nearest(np.array([1e9, np.inf]), E4M3_VALUES[:127]), [126, 126])


def test_ties_of_e2m1_go_to_the_even_code():
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 0.26, 4.99])
    assert ob._nearest(v, E2M1_VALUES[:8]).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 1, 6]


def test_a_block_by_hand():
    x = np.zeros((1, 32), np.float32)
    x[0, :4] = [6.0, -3.0, 0.4, -0.1]                   # s = 1: codes 7, -5, 1 (0.4 -> 0.5), -0
    codes, s = ob.nvfp4_rows(x, 1.0)
    assert s.tolist() == [[0x38, 0]] and codes[0, :2].tolist() == [7 | (13 << 4), 1 | (8 << 4)]
    assert not codes[0, 2:].any()
    assert ob.nvfp4_values(codes, s, 1.0)[0, :4].tolist() == [6.0, -3.0, 0.5, 0.0]
    x[0, 20] = np.nan
    x[0, 3] = -np.inf
    codes, s = ob.nvfp4_rows(x, 1.0)
    assert s.tolist() == [[126, 0x7F]] and ob.nvfp4_values(codes, s, 1.0)[0, 3] == -6 * 448
    assert np.isnan(ob.nvfp4_values(codes, s, 1.0)[0, 16:]).all()


@pytest.mark.parametrize("g", [1.0, 0.0021, 3.0e-5])
def test_rows_are_near_what_they_stand_for(g):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 128)) * 448 * g).astype(np.float32)
    back = ob.nvfp4_values(*ob.nvfp4_rows(x, g), g).astype(np.float64)
    b, y = x.reshape(40, 8, 16).astype(np.float64), back.reshape(40, 8, 16)
    # the scale is within 2^-4 of max / 6, and a code within half its step, at most a sixth of six steps
    top = np.abs(b).max(-1, keepdims=True)
    assert (np.abs(b - y) <= top * (1 / 6 + 1 / 16) * 1.001).all()


def test_equal_axes_turn_as_one():
    rng = np.random.default_rng(2)
    rope = rng.standard_normal((20, 16)).astype(np.float32)
    v, pos = rng.standard_normal((5, 2, 32)), rng.integers(0, 20, 5)
    want = ob.rotate(v, rope, pos)
    assert np.array_equal(ob.rotate_axes(v, rope, [pos] * 3, [0, 1, 2, 2, 1, 0, 0, 1]), want)
    got = ob.rotate_axes(v, rope, [pos, (pos + 1) % 20], [0, 0, 0, 0, 1, 1, 1, 1])
    assert np.array_equal(got[..., :4], want[..., :4])
    other = ob.rotate(v, rope, (pos + 1) % 20)
    assert np.array_equal(got[..., [4, 15]], other[..., [4, 15]])
