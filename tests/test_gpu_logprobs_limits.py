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


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("power", [-60, -66, -70, -74])
def test_sums_that_float32_hardly_holds(T, power):
    """Products and sums below 2^-126: whatever the matrix instructions make of them, the order is that of the 64-bit
    sums of products that are rounded as float32 rounds below its range."""
    import torch
    V, K = 3000, 128
    X, W, y, _, _ = problem(T, V, K, 7, scale=1.0)
    X, W = X * 2.0 ** power, W * 2.0 ** power
    assert (X != 0).any(1).all() and (W != 0).any()
    for top in (1, 30):
        got = sbn.sbn_token_logprobs(X, W, y, top=top)
        sums = torch.stack([(x.float() * W.float()).double().sum(1) for x in X])
        assert torch.equal(got[3], torch.sort(sums, dim=1, descending=True, stable=True).indices[:, :top])
        check_forward([*got[:3], None, None], reference(X, W, y), y, 0)
