"""Tensors of more than 2^31 elements (offsets past 32 bits), and views that start at any element.

Checked at their ends against the same calls on short copies, which the other
files hold to the formulas: rows and elements do not depend on their neighbours.
"""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn

pytestmark = pytest.mark.gpu


def test_norm_rows_past_32_bits():
    import torch
    T, K = (1 << 20) + 77, 2048
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    X.normal_(generator=g)
    gain = torch.rand(K, device="cuda") + 0.5
    ends = torch.cat([torch.arange(40, device="cuda"), torch.arange(T - 40, T, device="cuda")])
    short = X[ends]
    Xq, s_x, H, rstd = sbn.sbn_rmsnorm_quant(X, gain, residual=X)
    a = sbn.sbn_rmsnorm_quant(short, gain, residual=short)
    for p, q in zip((Xq, s_x, H, rstd), a):
        assert torch.equal(p[ends], q)
    del Xq
    dX, dg = sbn.sbn_rmsnorm_backward(X, H, gain, rstd, dH=X)
    b, _ = sbn.sbn_rmsnorm_backward(short, a[2], gain, a[3], dH=short)
    assert torch.equal(dX[ends], b) and torch.isfinite(dg).all()


def test_vocabulary_past_32_bits():
    import torch
    T, V, K = 3, (1 << 20) + 1001, 2048
    g = torch.Generator(device="cuda").manual_seed(2)
    W = torch.empty((V, K), dtype=torch.bfloat16, device="cuda")
    W.normal_(std=0.02, generator=g)
    X = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    y = torch.tensor([V - 1, 5, V - 600], device="cuda")
    loss, lse = sbn.sbn_cross_entropy(X, W, y)
    z = torch.cat([X.double() @ w.double().t().contiguous() for w in W.split(1 << 17)], 1)
    want = torch.logsumexp(z, 1)
    assert torch.allclose(lse.double(), want, rtol=0, atol=1e-4)
    assert torch.allclose(loss.double(), want - z.gather(1, y[:, None])[:, 0], rtol=0, atol=1e-4)
    dX, dW = sbn.sbn_cross_entropy_backward(X, W, y, lse, torch.ones(T, device="cuda"))
    D = torch.exp(z - want[:, None])
    D[torch.arange(T), y] -= 1
    for at in (slice(0, 64), slice(V - 700, V)):
        ref = D[:, at].t().contiguous() @ X.double()
        assert (dW[at].double() - ref).norm() <= 2 ** -7 * ref.norm()
    ref = sum(d @ w.double() for d, w in zip(D.split(1 << 17, 1), W.split(1 << 17)))
    assert (dX.double() - ref).norm() <= 2 ** -7 * ref.norm()


def test_adamw_elements_past_32_bits():
    import torch
    n = (1 << 31) + 3001
    p = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    g = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    g.normal_(std=0.01)
    m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    sm, sv = (torch.zeros(-(-n // 256), device="cuda") for _ in range(2))
    tail = n - 3001 - 5 * 256                                      # a multiple of the block
    short = [t[tail:].clone() for t in (p, g, m, v)] + [t[tail // 256:].clone() for t in (sm, sv)]
    sbn.sbn_adamw_step(sbn.AdamWTable([p], [g], [m], [v], m_scales=[sm], v_scales=[sv]), lr=0.01, step=1)
    q = short
    sbn.sbn_adamw_step(sbn.AdamWTable([q[0]], [q[1]], [q[2]], [q[3]], m_scales=[q[4]], v_scales=[q[5]]), lr=0.01, step=1)
    for a, b in zip((p[tail:], m[tail:], v[tail:], sm[tail // 256:], sv[tail // 256:]), (q[0], q[2], q[3], q[4], q[5])):
        assert torch.equal(a, b)
    assert (p[:4096] != 0.5).any()


def test_vectors_that_start_at_any_element():
    import torch
    T, V, K = 33, 500, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn(V, K, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    y = torch.randint(0, V, (T + 1,), generator=g, device="cuda")
    d = torch.rand(T + 3, device="cuda")
    f = lambda: torch.empty(T + 1, device="cuda")[1:]  # noqa: E731
    loss, lse = sbn.sbn_cross_entropy(X, W, y[1:], loss=f(), lse=f())
    got = sbn.sbn_cross_entropy_backward(X, W, y[1:], lse, d[3:])
    loss2, lse2 = sbn.sbn_cross_entropy(X, W, y[1:].clone())
    ref = sbn.sbn_cross_entropy_backward(X, W, y[1:].clone(), lse2, d[3:].clone())
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    gain = torch.ones(K, device="cuda")
    a = sbn.sbn_rmsnorm_quant(X, gain, s_x=f(), rstd=f())
    b = sbn.sbn_rmsnorm_quant(X, gain)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    with pytest.raises(sbn.SbnError):                              # 16-byte loads: refused
        sbn.sbn_rmsnorm(X, torch.ones(K + 1, device="cuda")[1:])


def test_what_tokens_without_a_target_hold_does_not_matter():
    import torch
    T, V, K = 70, 300, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    X = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn(V, K, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[10:30] = -100
    _, lse = sbn.sbn_cross_entropy(X, W, y)
    d = torch.rand(T, device="cuda") + 0.5
    ref = sbn.sbn_cross_entropy_backward(X, W, y, lse, d)
    d[10:20], d[20:30] = float("nan"), float("inf")
    lse[10:20], lse[20:30] = float("nan"), float("-inf")
    got = sbn.sbn_cross_entropy_backward(X, W, y, lse, d)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert (got[0][10:30] == 0).all()


def test_gradients_with_tiny_zero_and_mixed_dloss():
    """D is held relative to the largest |dloss|: gradients scale with it exactly by powers of two, and vanish with it."""
    import torch
    T, V, K = 65, 300, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn(V, K, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    _, lse = sbn.sbn_cross_entropy(X, W, y)
    d = torch.rand(T, generator=g, device="cuda") - 0.5
    kw = dict(dxdt=sbn.SBN_F32, dwdt=sbn.SBN_F32)
    ref = sbn.sbn_cross_entropy_backward(X, W, y, lse, d, **kw)
    for s in (2.0 ** -20, 2.0 ** -80, 2.0 ** 30):
        got = sbn.sbn_cross_entropy_backward(X, W, y, lse, d * s, **kw)
        assert all(torch.equal(a * s, b) for a, b in zip(ref, got))
    got = sbn.sbn_cross_entropy_backward(X, W, y, lse, d * 0, **kw)
    assert all((t == 0).all() for t in got)
