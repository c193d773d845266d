"""RopeAxes takes whole numbers of any kind, and nothing else."""
import numpy as np
import pytest
import torch

from tests.test_block_refusals_cpu import m  # noqa: F401


def test_whole_numbers_of_any_kind(m):  # noqa: F811
    for axes in ([0, 1, 2], (0.0, 1.0, 2.0), np.array([0, 1, 2]), torch.tensor([0, 1, 2])):
        got = m.RopeAxes(axes)
        assert got.axes == (0, 1, 2) and got.count == 3
        assert m.RopeAxes.of_sections(axes).axes == (1, 2, 2)


@pytest.mark.parametrize("bad", [(0, 0.5), (1.5, 1.5), np.array([0.0, 1.9]), torch.tensor([0.25, 1.0])])
def test_fractions_are_refused(m, bad):  # noqa: F811
    for axes in (bad, iter(bad)):
        with pytest.raises(ValueError):
            m.RopeAxes(axes)
    with pytest.raises(ValueError):
        m.RopeAxes.of_sections(bad)
    with pytest.raises(ValueError):
        m.RopeAxes.of_sections(bad, interleaved=True)
