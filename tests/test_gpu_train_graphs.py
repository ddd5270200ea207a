"""The norm, the cross entropy and AdamW under HIP graph capture: replays, with
eager work and synchronisation between them, give the eager results bit for bit;
and calls on two streams at once do not share scratch."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_graphs import replay_matches

pytestmark = pytest.mark.gpu


def _randn(seed, *shape, scale=1.0, bf16=True):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda") * scale
    return x.to(torch.bfloat16) if bf16 else x


def test_norm_forward_and_backward():
    import torch
    T, K = 70, 520
    x, r, dy, dh = (_randn(i, T, K) for i in range(4))
    g = _randn(5, K, bf16=False)
    H, Y, dX = (torch.empty_like(x) for _ in range(3))
    Xq = torch.empty((T, K), dtype=torch.int8, device="cuda")
    s_x, rs, rs2, dg = (torch.empty(n, device="cuda") for n in (T, T, T, K))
    H2 = torch.empty_like(x)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def step():
        sbn.sbn_rmsnorm_quant(x, g, residual=r, H=H, Xq=Xq, s_x=s_x, rstd=rs)
        sbn.sbn_rmsnorm(x, g, residual=r, H=H2, Y=Y, rstd=rs2)
        sbn.sbn_rmsnorm_backward(dy, H, g, rs, dH=dh, dX=dX, dgain=dg, ws=ws)

    replay_matches(step, [H, H2, Y, Xq, s_x, rs, rs2, dX, dg])


@pytest.mark.parametrize("T,V,K", [(300, 5000, 128), (20, 3001, 192)])
def test_cross_entropy(T, V, K):
    import torch
    X, W = _randn(1, T, K), _randn(2, V, K, scale=0.05)
    y = torch.arange(T, device="cuda") % V
    d = torch.full((T,), 1.0 / T, device="cuda")
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dX, dW = torch.empty_like(X), torch.empty((V, K), device="cuda")
    w1 = torch.empty(sbn.sbn_cross_entropy_workspace_bytes(T, V, K), dtype=torch.uint8, device="cuda")
    w2 = torch.empty(sbn.sbn_cross_entropy_workspace_bytes(T, V, K, True), dtype=torch.uint8, device="cuda")

    def step():
        sbn.sbn_cross_entropy(X, W, y, loss=loss, lse=lse, ws=w1)
        sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dwdt=sbn.SBN_F32, dX=dX, dW=dW, ws=w2)

    replay_matches(step, [loss, lse, dX, dW])


def test_adamw():
    import torch
    p0, g = _randn(1, 5000, bf16=False), _randn(2, 5000, bf16=False)
    p, m, v, sh = p0.clone(), torch.zeros_like(p0), torch.zeros_like(p0), torch.empty(5000, dtype=torch.bfloat16,
                                                                                     device="cuda")
    t = sbn.AdamWTable([p], [g], [m], [v], shadows=[sh], weight_decay=0.1)

    def before():
        p.copy_(p0), m.zero_(), v.zero_()

    replay_matches(lambda: sbn.sbn_adamw_step(t, lr=1e-2, step=1), [p, m, v, sh], before=before)


def test_two_streams_at_once():
    """Scratch that the binding allocates belongs to one stream."""
    import torch
    T, V, K = 256, 3000, 256
    ins = [(_randn(10 + i, T, K), _randn(20 + i, V, K, scale=0.05)) for i in range(2)]
    y = torch.arange(T, device="cuda")
    d = torch.ones(T, device="cuda")
    g = torch.ones(K, device="cuda")

    def work(X, W):
        loss, lse = sbn.sbn_cross_entropy(X, W, y)
        Y, H, rs = sbn.sbn_rmsnorm(X, g)
        return (loss, *sbn.sbn_cross_entropy_backward(X, W, y, lse, d), *sbn.sbn_rmsnorm_backward(Y, H, g, rs))

    ref = [work(*a) for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s, a in zip(streams, ins):
            with torch.cuda.stream(s):
                got.append(work(*a))
        torch.cuda.synchronize()
        for a, b in zip(ref, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
