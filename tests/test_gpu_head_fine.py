"""Gradients of the head of type SBN_F32_FINE, from logit gradients D of two bf16
numbers, against 64-bit torch.

Bounds (u = 2^-24), with those of the logits as in test_gpu_cross_entropy.py:
  D   |g| p (the logit's and lse's errors) + (2^-17 + 8 u) |D| + u |g|: the second
      number is rounded to 8 bits of at most 2^-9 |D|
  dX  sum_v (D's error |w|) + (2 V + 32) u sum_v |D w| (1 + 2^-8); dW the same over t
And in the norm over all of dX or dW: one bf16 D is off by a relative 2^-9 / sqrt 3
and more, two by under 2^-17, so with logits of K = 64 to 256 terms the whole error
is under 2^-13 of the gradient; that of one number is not.
"""
from __future__ import annotations

import ctypes

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_cross_entropy import U, close, make, reference

pytestmark = pytest.mark.gpu


def bounds(X, W, y, d):
    import torch
    r = reference(X, W, y, d)
    Xd, Wd, D = X.double(), W.double(), r["D"]
    T, V, K = X.shape[0], W.shape[0], X.shape[1]
    z = Xd @ Wd.t().contiguous()
    A = Xd.abs() @ Wd.abs().t().contiguous()
    rl = 4 * U * (1 + z.abs() + r["lse"].abs()[:, None])
    p = torch.exp(z - r["lse"][:, None])
    g = torch.where((y >= 0) & (y < V), d.double().abs(), 0.0)[:, None]
    bD = g * p * (K * U * A + r["blse"][:, None] + rl) + (2.0 ** -17 + 8 * U) * D.abs() + U * g
    more = U * (1 + 2.0 ** -8)
    r["bX"] = bD @ Wd.abs() + (2 * V + 32) * more * (D.abs() @ Wd.abs())
    r["bW"] = bD.t().contiguous() @ Xd.abs() + (2 * T + 32) * more * (D.abs().t().contiguous() @ Xd.abs())
    return r


@pytest.mark.parametrize("T,V,K", [(1, 1, 64), (2, 63, 128), (65, 129, 64), (257, 300, 64), (300, 2500, 256),
                                   (1021, 777, 192), (64, 9001, 64), (2100, 4700, 64), (4100, 4097, 128),
                                   (4096, 70001, 64)])
def test_fine_gradients(T, V, K):
    import torch
    X, W, y, d = make(T, V, K, 31 * T + V, ignored=0.2 if T > 1 else 0.0)
    r = bounds(X, W, y, d)
    _, lse = sbn.sbn_cross_entropy(X, W, y)
    one, two = sbn.SBN_F32, sbn.SBN_F32_FINE
    dX, dW = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=two, dwdt=two)
    close(dX, r["dX"], r["bX"], "dX")
    close(dW, r["dW"], r["bW"], "dW")
    assert (dX[y < 0] == 0).all()
    if V > 1:
        x1, w1 = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=one, dwdt=one)
        for got, coarse, ref in ((dX, x1, r["dX"]), (dW, w1, r["dW"])):
            off = lambda t: float((t.double() - ref).norm() / ref.norm())  # noqa: E731
            assert off(got) < 2.0 ** -13 and off(coarse) > off(got), (off(got), off(coarse))
            print(f"T={T} V={V} K={K}: {off(coarse):.2e} -> {off(got):.2e}")
    again = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=two, dwdt=two)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dW)


def test_each_gradient_has_its_own_type():
    """One gradient fine, the other in one bf16 number, in either order; strides; a gradient not asked for."""
    import torch
    T, V, K = 300, 1111, 64
    X, W, y, d = make(T, V, K, 5, ldx=K + 24, ldw=K + 8)
    _, lse = sbn.sbn_cross_entropy(X, W, y)
    f, b, two = sbn.SBN_F32, sbn.SBN_BF16, sbn.SBN_F32_FINE
    fine = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=two, dwdt=two)
    plain = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=f, dwdt=b)
    dX, dW = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=two, dwdt=b)
    assert torch.equal(dX, fine[0]) and torch.equal(dW, plain[1])
    bw = torch.full((V, K + 40), 5.0, device="cuda")
    dX, _ = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=f, dwdt=two, dW=bw[:, :K])
    assert torch.equal(dX, plain[0]) and torch.equal(bw[:, :K], fine[1]) and (bw[:, K:] == 5.0).all()
    dX, none = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=two, dwdt=two, need_dW=False)
    assert none is None and torch.equal(dX, fine[0])
    none, dW = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=two, dwdt=two, need_dX=False)
    assert none is None and torch.equal(dW, fine[1])
    e = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    _, dW = sbn.sbn_cross_entropy_backward(e, W, y[:0], lse[:0], d[:0], dxdt=two, dwdt=two)
    assert dW.dtype == torch.float32 and (dW == 0).all()


def test_other_calls_refuse_the_type():
    P = ctypes.c_void_p(0x100000)
    L = sbn.lib()
    st = L.sbn_rmsnorm(P, 64, None, 0, sbn.SBN_F32_FINE, P, sbn.SBN_F32, 4, 64, 1e-6, None, 0, P, 64, None, None)
    assert st == 6
    assert L.sbn_sparse_ternary_gemm(P, P, 16, 256, P, P, P, 256, 2, 4, P, sbn.SBN_F32_FINE, 256, P, 1 << 30, None) == 6
