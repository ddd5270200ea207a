"""The example's training loop: the loss falls with states in 32 and in 8 bits, and single tokens score as a batch."""
from __future__ import annotations

import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_loss_falls(bits):
    import torch
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_lm.py")
    spec = importlib.util.spec_from_file_location("train_lm", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, (batch, single) = m.main(["--steps", "60", "--bits", str(bits)])
    assert all(math.isfinite(x) for x in losses)
    assert abs(losses[0] - math.log(m.V)) < 2.0                   # random weights: near the uniform guess
    assert losses[-1] < 0.6 * losses[0]
    assert torch.equal(batch, single)                              # integer products, and one order of every sum
