"""SBN_CHECK_FINITE=1 and the gradient of each token's loss: every element with a
target is looked at, whatever the number of tokens and wherever the vector starts;
what a token without a target holds does not matter; a call that passes the check
computes what it computes without it."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_cross_entropy import make

pytestmark = pytest.mark.gpu
V, K = 100, 64


def case(T, first=0):
    """Inputs with every token a target, dloss starting at element `first` of its memory."""
    import torch
    X, W, y, d = make(T, V, K, 100 + T, ignored=0.0)
    room = torch.ones(T + first, device="cuda")
    room[first:] = d
    _, lse = sbn.sbn_cross_entropy(X, W, y)
    return X, W, y, lse, room[first:]


def refused(*a):
    with pytest.raises(sbn.SbnError) as e:
        sbn.sbn_cross_entropy_backward(*a)
    assert e.value.status == sbn.SBN_ERR_VALUE and "dloss" in str(e.value)


@pytest.mark.parametrize("T,first", [(1, 0), (2, 0), (3, 1), (4, 3), (5, 0), (7, 1), (8, 2), (1021, 1), (70001, 3)])
def test_every_element(T, first, monkeypatch):
    import torch
    X, W, y, lse, d = case(T, first)
    ref = sbn.sbn_cross_entropy_backward(X, W, y, lse, d)
    monkeypatch.setenv("SBN_CHECK_FINITE", "1")
    for labels in (y, y.int()):
        got = sbn.sbn_cross_entropy_backward(X, W, labels, lse, d)
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
        for at in sorted({0, T // 2, T - 1}):
            for bad in ("nan", "inf", "-inf"):
                keep = float(d[at])
                d[at] = float(bad)
                refused(X, W, labels, lse, d)
                d[at] = keep


@pytest.mark.parametrize("label", [-100, -1, V, 2 ** 31 - 1])
def test_tokens_without_a_target(label, monkeypatch):
    import torch
    X, W, y, lse, d = case(9)
    y[3], y[8] = label, label
    ref = sbn.sbn_cross_entropy_backward(X, W, y, lse, d)
    monkeypatch.setenv("SBN_CHECK_FINITE", "1")
    d[3], d[8] = float("nan"), float("inf")
    for labels in (y, y.int()):
        got = sbn.sbn_cross_entropy_backward(X, W, labels, lse, d)
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    d[4] = float("nan")
    refused(X, W, y, lse, d)


def test_what_surrounds_the_vector_is_not_looked_at(monkeypatch):
    import torch
    X, W, y, lse, d = case(6)
    room = torch.full((16,), float("nan"), device="cuda")
    room[5:11] = d
    monkeypatch.setenv("SBN_CHECK_FINITE", "1")
    sbn.sbn_cross_entropy_backward(X, W, y, lse, room[5:11])
