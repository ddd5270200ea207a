"""Cross entropy of 2^26 and more tokens: the launch that joins the statistics would
need 2^32 threads if it gave every token its own.  Checked at both ends and in the
middle against 64 bits, within the bounds of test_gpu_cross_entropy.py."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_cross_entropy import close, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [(1 << 26) - 17, (1 << 26) + 77])
def test_loss(T):
    import torch
    V, K = 100, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.empty((T, K), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    W = (torch.randn(V, K, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    y = torch.randint(-1, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    loss, lse = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    sbn.sbn_cross_entropy(X, W, y, loss=loss, lse=lse)
    assert torch.isfinite(loss).all() and torch.isfinite(lse).all()
    for at in (slice(0, 300), slice(T // 2, T // 2 + 300), slice(T - 300, T)):
        r = reference(X[at], W, y[at].long(), torch.ones(300, device="cuda"))
        close(lse[at], r["lse"], r["blse"], "lse")
        close(loss[at], r["loss"], 2 * r["blse"], "loss")
