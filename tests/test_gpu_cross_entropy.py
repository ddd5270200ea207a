"""Cross entropy of the output head and its gradients against 64-bit torch.

Bounds, with u = 2^-24 and b = 2^-8, each a worst case:
  l      products of bf16 are exact in float32, K of them are summed: K u A,
         A[t,v] = sum_k |x w|
  lse    the largest error of a logit, and the roundings of its exponentials
         (relative 4 u (1 + |l| + |lse|) with the scaled argument's), their sum
         (V u) and its logarithm: K u max A + 4 u (1 + max|l| + |lse|) + (sqrt(V) + 64) u
         (the sum goes over 64 entries in a row and then in a tree of the same depth)
  loss   that and the target's logit: twice it
  D      |g| p (the logit's and lse's errors + 4 u (1 + |l| + |lse|)) + b |D| + u |g|
  dX     sum_v (D's error |w|) + (V + 16) u sum_v |D w|, plus b |dX| for bf16; dW the same over t
"""
from __future__ import annotations

import numpy as np
import pytest

import sparse_linear_layers_02_amd as sbn

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8


def make(T, V, K, seed, scale=0.05, ldx=None, ldw=None, ignored=0.2):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def mat(n, ld, s):
        t = torch.full((n, ld or K), float("nan"), dtype=torch.bfloat16, device="cuda")
        t[:, :K] = (torch.randn(n, K, generator=g, device="cuda") * s).to(torch.bfloat16)
        return t[:, :K]

    X, W = mat(T, ldx, 1.0), mat(V, ldw, scale)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    drop = torch.rand(T, generator=g, device="cuda") < ignored
    y = torch.where(drop, torch.tensor(-100, device="cuda"), y)
    d = torch.rand(T, generator=g, device="cuda") + 0.5
    return X, W, y, d


def reference(X, W, y, d):
    import torch
    Xd, Wd = X.double(), W.double()
    V, K = Wd.shape
    z = Xd @ Wd.t().contiguous()
    A = Xd.abs() @ Wd.abs().t().contiguous()
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    lse = (top + torch.log(e.sum(1, keepdim=True)))[:, 0]
    kept = (y >= 0) & (y < V)
    at = torch.where(kept, y, 0)[:, None]
    loss = torch.where(kept, lse - z.gather(1, at)[:, 0], 0.0)
    p = torch.exp(z - lse[:, None])
    D = p.clone().scatter_add_(1, at, -torch.ones_like(at, dtype=torch.float64))
    g = torch.where(kept, d.double(), 0.0)[:, None]
    D = D * g
    el = K * U * A
    rl = 4 * U * (1 + z.abs() + lse.abs()[:, None])
    blse = el.amax(1) + rl.amax(1) + (V ** 0.5 + 64) * U
    bD = g.abs() * p * (el + blse[:, None] + rl) + B * D.abs() + U * g.abs()
    bX = bD @ Wd.abs() + (V + 16) * U * (D.abs() @ Wd.abs())
    T = X.shape[0]
    bW = bD.t().contiguous() @ Xd.abs() + (T + 16) * U * (D.abs().t().contiguous() @ Xd.abs())
    return dict(loss=loss, lse=lse, blse=blse, dX=D @ Wd, bX=bX, dW=D.t().contiguous() @ Xd, bW=bW, D=D)


def close(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound.clamp(min=1e-300)).max()):.3g} bounds"


SHAPES = [(1, 1, 64), (1, 1000, 64), (2, 63, 128), (17, 64, 64), (64, 65, 192), (65, 129, 64), (130, 257, 320),
          (1, 513, 2560), (33, 1999, 128), (257, 300, 64), (300, 2500, 256), (1021, 777, 192), (64, 9001, 64),
          (2100, 4700, 64), (4100, 4097, 128)]


@pytest.mark.parametrize("T,V,K", SHAPES)
def test_loss_and_gradients(T, V, K):
    import torch
    X, W, y, d = make(T, V, K, 1000 * T + V, ignored=0.2 if T > 1 else 0.0)
    r = reference(X, W, y, d)
    loss, lse = sbn.sbn_cross_entropy(X, W, y)
    close(lse, r["lse"], r["blse"], "lse")
    close(loss, r["loss"], 2 * r["blse"], "loss")
    assert (loss[(y < 0)] == 0).all()
    loss4, lse4 = sbn.sbn_cross_entropy(X, W, y.int())
    assert torch.equal(loss4, loss) and torch.equal(lse4, lse)
    dX, dW = sbn.sbn_cross_entropy_backward(X, W, y, lse, d)
    close(dX, r["dX"], r["bX"] + B * r["dX"].abs(), "dX bf16")
    close(dW, r["dW"], r["bW"] + B * r["dW"].abs(), "dW bf16")
    assert (dX[y < 0] == 0).all()
    f = sbn.SBN_F32
    dX4, dW4 = sbn.sbn_cross_entropy_backward(X, W, y.int(), lse, d, dxdt=f, dwdt=f)
    close(dX4, r["dX"], r["bX"], "dX f32")
    close(dW4, r["dW"], r["bW"], "dW f32")
    assert torch.equal(dX4.to(torch.bfloat16), dX) and torch.equal(dW4.to(torch.bfloat16), dW)
    x2, w0 = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, need_dW=False)
    x0, w2 = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, need_dX=False)
    assert w0 is None and x0 is None and torch.equal(x2, dX) and torch.equal(w2, dW)


def test_several_pieces_of_the_vocabulary():
    """T V above the workspace's bound on D: dX is summed over pieces."""
    import torch
    T, V, K = 4096, 70001, 64
    X, W, y, d = make(T, V, K, 7)
    assert sbn.sbn_cross_entropy_workspace_bytes(T, V, K, True) < T * V * 2 * 2
    r = reference(X, W, y, d)
    loss, lse = sbn.sbn_cross_entropy(X, W, y)
    close(loss, r["loss"], 2 * r["blse"], "loss")
    dX, dW = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=sbn.SBN_F32)
    close(dX, r["dX"], r["bX"], "dX")
    close(dW, r["dW"], r["bW"] + B * r["dW"].abs(), "dW")
    again = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=sbn.SBN_F32)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dW)


@pytest.mark.parametrize("T,V,K", [(50, 333, 128), (300, 1111, 64)])
def test_strides(T, V, K):
    import torch
    X, W, y, d = make(T, V, K, 5, ldx=K + 24, ldw=K + 8)
    r = reference(X, W, y, d)
    loss, lse = sbn.sbn_cross_entropy(X, W, y)
    close(loss, r["loss"], 2 * r["blse"], "loss")
    bx = torch.full((T, K + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    bw = torch.full((V, K + 40), 5.0, dtype=torch.float32, device="cuda")
    sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dwdt=sbn.SBN_F32, dX=bx[:, :K], dW=bw[:, :K])
    close(bx[:, :K], r["dX"], r["bX"] + B * r["dX"].abs(), "dX")
    close(bw[:, :K], r["dW"], r["bW"], "dW")
    assert (bx[:, K:] == 3.0).all() and (bw[:, K:] == 5.0).all(), "columns past the rows"


def test_no_target_anywhere_and_labels_out_of_range():
    import torch
    T, V, K = 70, 200, 64
    X, W, _, d = make(T, V, K, 9)
    for bad in (-100, -1, V, V + 7, 2 ** 40, -2 ** 40):
        y = torch.full((T,), bad, device="cuda")
        loss, lse = sbn.sbn_cross_entropy(X, W, y)
        assert (loss == 0).all() and torch.isfinite(lse).all()
        dX, dW = sbn.sbn_cross_entropy_backward(X, W, y, lse, d)
        assert (dX == 0).all() and (dW == 0).all()


def test_large_logits_and_a_vocabulary_of_one():
    """Logits of several hundred, one far above the rest: exponentials neither overflow nor vanish wrongly."""
    import torch
    T, V, K = 40, 1000, 64
    X, W, y, d = make(T, V, K, 11, scale=8.0, ignored=0.0)
    r = reference(X, W, y, d)
    assert float(r["lse"].abs().max()) > 100
    loss, lse = sbn.sbn_cross_entropy(X, W, y)
    close(lse, r["lse"], r["blse"], "lse")
    close(loss, r["loss"], 2 * r["blse"], "loss")
    dX, dW = sbn.sbn_cross_entropy_backward(X, W, y, lse, d)
    close(dX, r["dX"], r["bX"] + B * r["dX"].abs(), "dX")
    X, W, y, d = make(5, 1, 64, 12, ignored=0.0)
    loss, lse = sbn.sbn_cross_entropy(X, W, y)
    assert (loss == 0).all()                              # exp(l - l) alone: the logarithm of 1
    z = X.double() @ W.double().t()
    close(lse, z[:, 0], 64 * 2 * U * (X.double().abs() @ W.double().abs().t())[:, 0] + 4 * U, "lse")


def test_no_tokens():
    import torch
    X = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    W = torch.ones((100, 64), dtype=torch.bfloat16, device="cuda")
    y = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = sbn.sbn_cross_entropy(X, W, y)
    assert loss.shape == (0,) and lse.shape == (0,)
    for dt in (sbn.SBN_BF16, sbn.SBN_F32):
        dX, dW = sbn.sbn_cross_entropy_backward(X, W, y, lse, torch.empty(0, device="cuda"), dwdt=dt)
        assert dX.shape == (0, 64) and dW.shape == (100, 64) and (dW == 0).all()


def test_gradient_against_differences():
    """Along random directions, dX and dW (float32) against central differences of
    sum_t d_t loss_t in 64 bits (step 1e-4: the third-order term is under 1e-7 of
    the direction's size)."""
    import torch
    T, V, K, h = 20, 150, 64, 1e-4
    X, W, y, d = make(T, V, K, 13)
    r = reference(X, W, y, d)
    _, lse = sbn.sbn_cross_entropy(X, W, y)
    dX, dW = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=sbn.SBN_F32, dwdt=sbn.SBN_F32)
    kept = (y >= 0).double() * d.double()
    at = torch.where(y >= 0, y, 0)[:, None]

    def L(x, w):
        z = x @ w.t().contiguous()
        return ((torch.logsumexp(z, 1) - z.gather(1, at)[:, 0]) * kept).sum()

    g = torch.Generator(device="cuda").manual_seed(3)
    for mine, bound, which in ((dX, r["bX"], 0), (dW, r["bW"], 1)):
        e = torch.randn(mine.shape, generator=g, device="cuda", dtype=torch.float64)
        x, w = X.double(), W.double()
        up, dn = (L(x + h * e, w), L(x - h * e, w)) if which == 0 else (L(x, w + h * e), L(x, w - h * e))
        num = (up - dn) / (2 * h)
        size = float((e.abs() * (bound + 1e-7)).sum())
        assert abs(float((mine.double() * e).sum() - num)) <= size + 1e-5


def test_finite_check(monkeypatch):
    monkeypatch.setenv("SBN_CHECK_FINITE", "1")
    X, W, y, d = make(8, 100, 64, 17)
    _, lse = sbn.sbn_cross_entropy(X, W, y)
    W[50, 3] = float("nan")
    for f in (lambda: sbn.sbn_cross_entropy(X, W, y), lambda: sbn.sbn_cross_entropy_backward(X, W, y, lse, d)):
        with pytest.raises(sbn.SbnError) as e:
            f()
        assert e.value.status == sbn.SBN_ERR_VALUE


@pytest.mark.parametrize("T,V,K", [(65400, 4500, 192), (65400, 4500, 64)])
def test_several_pieces_with_a_tile_for_every_unit(T, V, K):
    """dX's sums of one piece are where the next one starts (no parts are joined), at ragged edges of its tiles."""
    import torch
    X, W, y, d = make(T, V, K, 11)
    r = reference(X, W, y, d)
    _, lse = sbn.sbn_cross_entropy(X, W, y)
    dX, _ = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=sbn.SBN_F32, need_dW=False)
    close(dX, r["dX"], r["bX"], "dX f32")
    dx16, dW = sbn.sbn_cross_entropy_backward(X, W, y, lse, d)
    assert torch.equal(dx16, dX.to(torch.bfloat16))
    close(dW, r["dW"], r["bW"] + B * r["dW"].abs(), "dW")
