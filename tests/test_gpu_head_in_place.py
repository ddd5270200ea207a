"""Gradients of the head in the place of an input, where the header allows it."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_cross_entropy import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,K", [(70, 300, 64), (300, 2500, 256), (65400, 9500, 64)])
def test_in_place(T, V, K):
    import torch
    X, W, y, d = make(T, V, K, 3, ldx=K + 8, ldw=K + 16)
    _, lse = sbn.sbn_cross_entropy(X, W, y)
    dX, dW = sbn.sbn_cross_entropy_backward(X, W, y, lse, d)
    W2 = torch.empty((V, K + 16), dtype=torch.bfloat16, device="cuda")[:, :K]
    W2.copy_(W)
    a, b = sbn.sbn_cross_entropy_backward(X, W2, y, lse, d, dW=W2)
    assert b is W2 and torch.equal(a, dX) and torch.equal(W2, dW)
    a, _ = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dX=X, need_dW=False)
    assert a is X and torch.equal(X, dX)
