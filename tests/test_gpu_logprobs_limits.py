"""Log probabilities at the ends of their ranges: the longest rows, and more tokens than a grid has blocks."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_cross_entropy import B, close
from test_gpu_logprobs import check_forward, problem, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [2, 270])
def test_the_longest_rows(T):
    import torch
    V, K = 300, 2 ** 18
    X, W, y, dl, dh = problem(T, V, K, 5, scale=0.005)
    r = reference(X, W, y, 1.0, dl, dh, fine=T <= 128)
    got = sbn.sbn_token_logprobs(X, W, y, top=20)
    check_forward(got, r, y, 20)
    dX, dW = sbn.sbn_token_logprobs_backward(X, W, y, got[2], got[1], dl, dh)
    close(dX, r["dX"], r["bX"] + B * r["dX"].abs(), "dX")
    close(dW, r["dW"], r["bW"] + B * r["dW"].abs(), "dW")
    with pytest.raises(sbn.SbnError):
        z = torch.zeros((1, K + 64), dtype=torch.bfloat16, device="cuda")
        sbn.sbn_token_logprobs(z, z)


@pytest.mark.parametrize("top", [0, 1])
def test_more_tokens_than_blocks(top):
    T, V, K = 2 ** 20 + 300, 1100, 64
    X, W, y, _, _ = problem(T, V, K, 6)
    got = sbn.sbn_token_logprobs(X, W, y, top=top)
    for rows in (slice(0, 40), slice(2 ** 20 - 20, 2 ** 20 + 20), slice(T - 40, T)):
        check_forward([None if t is None else t[rows] for t in got], reference(X[rows], W, y[rows]), y[rows], top)
