"""The norm and its gradient together, as examples/fit_norms.py runs them: the weights that made the recorded
outputs are found again."""
import pytest
import torch

from examples import fit_norms as ex

pytestmark = pytest.mark.gpu


def test_recorded_weights_are_found():
    torch.manual_seed(3)
    fit, recorded = ex.random_block(300, torch.device("cuda"), H=512, E=8, k=2, I=256)
    losses = [fit.step() for _ in range(400)]
    assert losses[-1] < 1e-3 * losses[0], (losses[0], losses[-1])
    for got, want in zip(fit.weights(), recorded):
        # bf16 weights, and Adam's last steps of up to 2 % of one around the optimum
        assert (got.float() - want.float()).abs().max() < 0.05
