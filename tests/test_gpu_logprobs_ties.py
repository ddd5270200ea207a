"""Top alternatives where more sets of logits qualify than the queues hold, for few tokens (1024 threads
each) and for many (256 threads each)."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_logprobs import check_forward, problem, reference

pytestmark = pytest.mark.gpu
K = 64


@pytest.mark.parametrize("T", [4, 300])
@pytest.mark.parametrize("top", [1, 20, 64])
def test_all_rows_equal(T, top):
    import torch
    V = 20000
    X, W, y, _, _ = problem(T, V, K, 1)
    W = W.contiguous()
    W[:] = W[:1].clone()
    logp, H, _, ids, tlp = sbn.sbn_token_logprobs(X, W, y, top=top)
    assert torch.equal(ids, torch.arange(top, device="cuda").expand(T, top))
    ln = torch.tensor(float(V), device="cuda").log()
    assert (H - ln).abs().max() < 1e-5 and (tlp + ln).abs().max() < 1e-5 and (logp[y >= 0] + ln).abs().max() < 1e-5


@pytest.mark.parametrize("T", [4, 300])
@pytest.mark.parametrize("top", [1, 20, 64])
@pytest.mark.parametrize("at", [[5], [5, 6], [0, 9, 17, 30]])
def test_many_equal_at_the_bound(T, top, at):
    """3200 sets with one, two or four entries of the same logit, a few above it."""
    import torch
    V = 102400
    X = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    X[:, 3] = 1.0
    W = torch.zeros((V, K), dtype=torch.bfloat16, device="cuda")
    v = torch.arange(V, device="cuda")
    for a in at:
        W[v % 32 == a, 3] = 1.0
    best = torch.tensor([7, 50000, 50001, 99999, 102399], device="cuda")
    W[best, 3] = torch.tensor([2.0, 3.0, 3.0, 2.5, 2.0], device="cuda").bfloat16()
    ids, tlp = sbn.sbn_token_logprobs(X, W, top=top)[3:]
    want = torch.sort(W[:, 3].double(), descending=True, stable=True).indices[:top]
    assert torch.equal(ids, want.expand(T, top))
    lp = torch.log_softmax(W[:, 3].double(), 0)[want]
    assert (tlp.double() - lp).abs().max() <= 1e-5


@pytest.mark.parametrize("T,top", [(4, 20), (300, 1), (300, 64)])
def test_a_margin_that_takes_everything(T, top):
    """Rows whose size lies where x is 0: no float32 sum can be told from another by the norms, and all are summed."""
    X, W, y, _, _ = problem(T, 20000, K, 2)
    X, W = X.contiguous(), W.contiguous()
    X[:, 11] = 0.0
    W[:, 11] = 2.0 ** 20
    check_forward(sbn.sbn_token_logprobs(X, W, y, top=top), reference(X, W, y), y, top)
