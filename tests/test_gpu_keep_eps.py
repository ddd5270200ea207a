"""Rows whose u is zero: with eps their norm's output and gradients are 0; with eps = 0 there is none, and the other
rows do not see it."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from gpu_util import dev
from test_gpu_rmsnorm import rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [520, 16392])
def test_rows_of_zeros(K):
    import torch
    a, dy, g = dev(rnd(1, 4, K)), dev(rnd(2, 4, K)), dev(1 + 0.2 * rnd(3, K))
    a[1] = -a[1].abs()                               # relu^2 gives nothing
    rest = [0, 2, 3]
    for eps in (1e-6, 0.0):
        Xq, s_x, ka, _ = sbn.sbn_activation_quant(a, act=sbn.SBN_RELU2, gain=g, eps=eps)
        dA, _, dg = sbn.sbn_activation_backward(dy, ka, act=sbn.SBN_RELU2, gain=g, eps=eps)
        assert (Xq[1] == 0).all() and torch.isfinite(s_x[rest]).all() and torch.isfinite(dA[rest]).all()
        if eps:
            assert torch.isfinite(s_x).all() and (dA[1] == 0).all() and torch.isfinite(dg).all()
        else:
            assert s_x[1].isinf() and dA[1].isnan().all()
        one = sbn.sbn_activation_quant(a[2:3], act=sbn.SBN_RELU2, gain=g, eps=eps)
        assert torch.equal(one[0], Xq[2:3]) and torch.equal(one[1], s_x[2:3])
