"""The kernels of the norm and the activation with 8-bit checkpoints at every width that has one of its
own: with a residual and a gradient along the residual stream and without, and with several rows to
each block that sums gradients of gains.  Against 64 bits with test_gpu_keep.py's bounds.

Some inputs here go below -87, where a sigmoid is under 2^-126 and has no full mantissa, or is 0: off by
2^-126 at most, so f = a g by |a| 2^-126 and f' = g (1 + a (1 - g)) by (1 + |a|) 2^-126, times |du| and
|du b|; and a result that is itself under 2^-126 by 2^-126."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_keep import ACTS, EPS, rows, same_kept
from test_gpu_rmsnorm import B, U, get, put, rnd

pytestmark = pytest.mark.gpu
# chunks of 8 a thread: 1 of up to 512 and of up to 1024 threads, 2 of 768, 4 of 512, rows read twice
WIDTHS = [2560, 8000, 9000, 14344, 16392, 32768]


def near(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound.clamp(min=1e-300)).max()):.3g} bounds"


def inputs(seed, T, K, f32):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, K, generator=g, device="cuda") * (1 + 19 * (torch.arange(K, device="cuda") % 97 == 0))
    return x if f32 else x.bfloat16()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("K", WIDTHS)
def test_norm_forward(K, res, f32):
    import torch
    T = 2
    x, _ = put(rows(1, T, K), f32)
    r = put(rnd([2, T, K], T, K) * 2, f32)[0] if res else None
    g, _ = put(1 + 0.2 * rnd([3, K], K), True)
    Xq, s_x, H, _ = sbn.sbn_rmsnorm_quant(x, g, residual=r, eps=EPS)
    Xk, s_k, Hk, kept = sbn.sbn_rmsnorm_quant_keep(x, g, residual=r, eps=EPS)
    assert torch.equal(Xk, Xq) and torch.equal(s_k, s_x) and torch.equal(Hk, H)
    want = (x.float() + r.float()).to(x.dtype) if res else x
    assert torch.equal(H, want)
    same_kept(kept, get(H, f32), "H")


def norm_gradient(h, dy, gain, T, F=1):
    """du, its bound, dgain and its bound, as test_gpu_keep.py's."""
    r = 1 / (h.pow(2).mean(1, keepdim=True) + EPS).sqrt()
    w = dy * gain
    back, mean = r ** 2 * (w * h).mean(1, keepdim=True), r ** 2 * (w * h).abs().mean(1, keepdim=True)
    du = r * (w - h * back)
    bound = U * r * ((40 + F) * w.abs() + (44 + 2 * F) * (h * back).abs() + (120 + 4 * F) * h.abs() * mean)
    term = dy * h * r
    return du, bound, term.sum(0), (-(-T // 256) + 100 + 2 * F) * U * term.abs().sum(0)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("along", [False, True])
@pytest.mark.parametrize("T", [2, 600])
@pytest.mark.parametrize("K", WIDTHS)
def test_norm_gradient(T, K, along, f32):
    import torch
    kept = sbn.sbn_keep8_encode(inputs(4, T, K, f32))
    h = sbn.sbn_keep8_decode(kept).double()
    dy = inputs(5, T, K, f32) * 0.01
    dh = inputs(6, T, K, f32) * 0.01 if along else None
    g = 1 + 0.2 * torch.randn(K, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")
    dx, bound, dg, bg = norm_gradient(h, dy.double(), g.double(), T)
    if along:
        dx = dx + dh.double()
    dX, dgain = sbn.sbn_rmsnorm_backward_kept(dy, kept, g, eps=EPS, dH=dh)
    near(dX, dx, bound + (2 * U + (0 if f32 else B)) * dx.abs(), "dX")
    near(dgain, dg, bg, "dgain")


def act64(a, act):
    import torch
    if act == sbn.SBN_RELU2:
        r = a.clamp(min=0)
        return r * r, 2 * r, torch.zeros_like(a)
    g = torch.sigmoid(a)
    return a * g, g * (1 + a * (1 - g)), 12 * (g + a.abs() * g)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("gated,norm", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("K", WIDTHS)
def test_activation_gradient(K, act, gated, norm, f32):
    import torch
    T, F = 600, 3 if act == sbn.SBN_RELU2 else 8
    ka = sbn.sbn_keep8_encode(inputs(1, T, K, f32))
    kb = sbn.sbn_keep8_encode(inputs(2, T, K, f32)) if gated else None
    g = 1 + 0.2 * torch.randn(K, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") if norm else None
    dy = inputs(5, T, K, f32) * 0.01
    a = sbn.sbn_keep8_decode(ka).double()
    b = sbn.sbn_keep8_decode(kb).double() if gated else torch.ones_like(a)
    f, slope, bs = act64(a, act)
    dA, dB, dgain = sbn.sbn_activation_backward(dy, ka, kb, act=act, gain=g, eps=EPS)
    du, bd = dy.double(), torch.zeros_like(a)
    if norm:
        du, bd, dg, bg = norm_gradient(f * b, du, g.double(), T, F)
        near(dgain, dg, bg, "dgain")
    more = (4 if act == sbn.SBN_RELU2 else 20) * U + (0 if f32 else B)
    tiny = 2.0 ** -126 if act == sbn.SBN_SILU else 0.0
    ref = du * b * slope
    near(dA, ref, bd * (b * slope).abs() + U * (du * b).abs() * bs + more * ref.abs() + tiny * (1 + (du * b).abs() * (1 + a.abs())), "dA")
    if gated:
        ref = du * f
        near(dB, ref, bd * f.abs() + more * ref.abs() + tiny * (1 + du.abs() * a.abs()), "dB")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("K", [9000, 12296, 20480])
def test_rows_do_not_depend_on_the_batch(K, f32):
    """Forward and gradients of the first rows as in a call of their own, bit for bit."""
    import torch
    T, few = 600, 3
    a, b, dy = inputs(1, T, K, f32), inputs(2, T, K, f32), inputs(3, T, K, f32)
    g = torch.linspace(0.5, 1.5, K, device="cuda")

    def work(a, b, dy):
        Xq, s_x, ka, kb = sbn.sbn_activation_quant(a, b, act=sbn.SBN_SILU, gain=g)
        dA, dB, _ = sbn.sbn_activation_backward(dy, ka, kb, act=sbn.SBN_SILU, gain=g)
        Xn, s_n, H, kh = sbn.sbn_rmsnorm_quant_keep(a, g, residual=b)
        return [Xq, s_x, *ka, *kb, dA, dB, Xn, s_n, H, *kh, sbn.sbn_rmsnorm_backward_kept(dy, kh, g, dH=a)[0]]

    for x, y in zip(work(a, b, dy), work(*(t[:few].contiguous() for t in (a, b, dy)))):
        assert torch.equal(x[:few], y)
