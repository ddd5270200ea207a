"""Gradients of the hidden states whose product goes over the vocabulary in 2 to 16 parts (the number in
brackets is what the sizes lead to), against 64 bits with test_gpu_cross_entropy.py's bounds."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_cross_entropy import B, close, make, reference
from test_gpu_head_tiles import launches

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,K", [(1021, 20000, 2048), (2100, 9001, 640), (1500, 9001, 640), (700, 20000, 1024), (1021, 9001, 640),
                                   (2100, 20000, 256), (700, 9001, 640), (200, 9001, 640), (700, 20000, 2048), (700, 20000, 256),
                                   (17, 32001, 2560), (200, 20000, 1024)])
def test_parts(T, V, K):
    X, W, y, d = make(T, V, K, T + V + K)
    r = reference(X, W, y, d)
    _, lse = sbn.sbn_cross_entropy(X, W, y)
    (dX, _), ran = launches(lambda: sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=sbn.SBN_F32, need_dW=False))
    assert ran["ce_sum"] == 1
    close(dX, r["dX"], r["bX"], "dX")
    half, _ = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, need_dW=False)
    close(half, r["dX"], r["bX"] + B * r["dX"].abs(), "dX bf16")
