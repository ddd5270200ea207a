"""8-bit checkpoints, the norm and the feed-forward activation that write them, and
their gradients, against the formulas: codes bit for bit (float32, numpy's order of
operations), the rest in 64 bits.

Bounds, with u = 2^-24 (float32) and b = 2^-8 (bf16), each a worst case:
  silu     exp within 2 u relative of the argument's own rounding (the argument is exact),
           1 + e, the quotient and a g: f within 6 u |f|; f' = g (1 + a (1 - g)) within
           12 u (g + |a| g)
  u        f b: relu^2 2 roundings, silu 7: F u |u| with F = 3 or 8
  codes    relu^2: equal.  silu: v = u gain is off by (F + 1) u |v|, so a code times its
           step m / 127 is off v by half a step + 3 (F + 1) u m
  s_x      m's (F + 1) u, the root's 32 u (a sum of squares of relative error (48 + 2 F) u,
           halved, and 4 u), two more: (2 F + 40) u
  gradient r within (28 + F + 4) u; back = r^2 mean(w u) within (2 (32 + F) + 48 + F + 6) u
           r^2 mean|w u|; du within u r ((40 + F) |w| + (44 + 2 F) |u back| + (120 + 4 F) |u|
           r^2 mean|w u|); dA, dB that times |b f'|, |f|, and F' u more with F' = 4 or 20
  dgain    a term within (36 + 2 F) u, at most ceil(T/256) + 64 in a row:
           (ceil(T/256) + 100 + 2 F) u sum|dy u r|
"""
from __future__ import annotations

import numpy as np
import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_graphs import replay_matches
from test_gpu_head_tiles import launches
from test_gpu_rmsnorm import B, U, close, get, put, reference, rnd, codes_of
from gpu_util import dev, host

pytestmark = pytest.mark.gpu
EPS = 1e-6
TINY = np.float32(2.0 ** -100)
BLOCK = sbn.SBN_KEEP_BLOCK


def keep8(x):
    """(codes, scales) of float32 rows, as the header says."""
    T, K = x.shape
    nb = -(-K // BLOCK)
    p = np.zeros((T, nb * BLOCK), np.float32)
    p[:, :K] = x
    p = p.reshape(T, nb, BLOCK)
    a = np.abs(p).max(2)
    live = a >= TINY
    # near the largest float 127 x would overflow, so both sides are taken down by a power of two, which changes no bit
    down = np.where(a > 1e30, np.float32(2.0 ** -8), np.float32(1.0))
    with np.errstate(all="ignore"):
        q = np.where(live[..., None], np.rint((np.float32(127.0) * (p * down[..., None])) / (a * down)[..., None]), 0).astype(np.int8)
    s = np.where(live, a / np.float32(127.0), np.float32(0.0)).astype(np.float32)
    return q.reshape(T, -1)[:, :K], s


def values8(q, s):
    return q.astype(np.float32) * np.repeat(s, BLOCK, 1)[:, : q.shape[1]]


def same_kept(kept, x, what):
    q, s = keep8(x)
    assert np.array_equal(host(kept.codes), q), what + " codes"
    assert np.array_equal(host(kept.scales), s), what + " scales"


SHAPES = [(1, 8), (1, 2560), (2, 64), (3, 136), (5, 1000), (17, 2048), (63, 4104), (257, 512), (7, 8192), (4, 8200),
          (3, 16384), (2, 16392), (2, 32768), (1025, 328), (600, 2560)]


def rows(seed, T, K):
    x = rnd([seed, T, K], T, K)
    x[:, ::97] *= 20.0
    if T > 2:
        x[2] = 0.0                                   # a padded token
    return x


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,K", SHAPES)
def test_encode_and_decode(T, K, f32):
    import torch
    x, xv = put(rows(1, T, K), f32, K + 24)
    kept = sbn.sbn_keep8_encode(x)
    same_kept(kept, xv, "X")
    v = values8(*keep8(xv))
    assert np.array_equal(host(sbn.sbn_keep8_decode(kept)), v)
    y = torch.full((T, K + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    assert sbn.sbn_keep8_decode(kept, Y=y[:, :K]).data_ptr() == y.data_ptr()
    assert torch.equal(y[:, :K], dev(v).bfloat16()) and (y[:, K:] == 3.0).all()
    step = np.repeat(keep8(xv)[1], BLOCK, 1)[:, :K].astype(np.float64)
    assert (np.abs(v - xv.astype(np.float64)) <= step * (0.5 + 2.0 ** -16)).all()


def test_blocks_of_extremes():
    """Zeros, values too small for a scale, the largest floats, and what NaN and Inf become."""
    import torch
    K = 6 * BLOCK + 8
    x = rnd(5, 2, K)
    x[0, :BLOCK] = 0.0
    x[0, BLOCK:2 * BLOCK] *= 2.0 ** -110
    x[0, 2 * BLOCK:3 * BLOCK] = np.float32(3.4e38) * np.sign(x[0, 2 * BLOCK:3 * BLOCK])
    x[0, 3 * BLOCK] = 2.0 ** 120                     # one far above the rest
    x[0, 4 * BLOCK:5 * BLOCK] *= 2.0 ** -96
    kept = sbn.sbn_keep8_encode(dev(x))
    same_kept(kept, x, "extremes")
    assert (host(kept.scales)[0, :2] == 0).all() and np.isfinite(host(sbn.sbn_keep8_decode(kept))).all()
    for bad in (float("nan"), float("inf"), -float("inf")):
        for f32 in (False, True):
            t = dev(rnd(6, 2, K)).to(torch.float32 if f32 else torch.bfloat16)
            t[1, BLOCK + 17] = bad
            v = sbn.sbn_keep8_decode(sbn.sbn_keep8_encode(t))
            assert torch.isnan(v[1, BLOCK:2 * BLOCK]).all()
            assert torch.isfinite(v[0]).all() and torch.isfinite(v[1, :BLOCK]).all() and torch.isfinite(v[1, 2 * BLOCK:]).all()


def test_every_bf16_quotient():
    """All mantissas against all mantissas of the block's maximum, down to 2^-9 of it: half-integers and
    the quotients next to them."""
    m = (128 + np.arange(128)).astype(np.float32) / 128
    x = np.concatenate([m * np.float32(2.0 ** -e) for e in range(10)])
    rows = []
    for a in m:
        v = np.where(x <= a, x, x / 2)
        v = np.concatenate([v, np.zeros(-v.size % (BLOCK - 1), np.float32)]).reshape(-1, BLOCK - 1)
        rows.append(np.concatenate([np.full((v.shape[0], 1), a, np.float32), v * np.where(np.arange(BLOCK - 1) % 2, 1, -1)], 1).ravel())
    x = np.stack(rows).astype(np.float32)
    for scale in (1.0, 2.0 ** 100, 2.0 ** -80):
        t, v = put(x * np.float32(scale), False)
        same_kept(sbn.sbn_keep8_encode(t), v, "quotients")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,K", SHAPES)
def test_norm_forward(T, K, f32):
    """Every output as sbn_rmsnorm_quant's, bit for bit, and the checkpoint of the stored h."""
    import torch
    res = T % 2 == 1
    x, _ = put(rows(1, T, K), f32)
    r, _ = put(rnd([2, T, K], T, K) * 2, f32) if res else (None, None)
    g, _ = put(1 + 0.2 * rnd([3, K], K), (T + K) % 3 != 0)
    Xq, s_x, H, _ = sbn.sbn_rmsnorm_quant(x, g, residual=r, eps=EPS)
    Xk, s_k, Hk, kept = sbn.sbn_rmsnorm_quant_keep(x, g, residual=r, eps=EPS)
    assert torch.equal(Xk, Xq) and torch.equal(s_k, s_x) and torch.equal(Hk, H)
    same_kept(kept, get(H, f32), "H")


def norm_gradient(h, dy, gain, T, F=1):
    """du, its bound, dgain and its bound at rows h (64 bits)."""
    K = h.shape[1]
    r = 1 / np.sqrt((h ** 2).mean(1, keepdims=True) + EPS)
    w = dy * gain
    back, mean = r ** 2 * (w * h).mean(1, keepdims=True), r ** 2 * np.abs(w * h).mean(1, keepdims=True)
    du = r * (w - h * back)
    bound = U * r * ((40 + F) * np.abs(w) + (44 + 2 * F) * np.abs(h * back) + (120 + 4 * F) * np.abs(h) * mean)
    term = dy * h * r
    return du, bound, term.sum(0), (-(-T // 256) + 100 + 2 * F) * U * np.abs(term).sum(0)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,K", SHAPES)
def test_norm_gradient(T, K, f32):
    kept = sbn.sbn_keep8_encode(dev(rows(4, T, K)))
    h = host(sbn.sbn_keep8_decode(kept)).astype(np.float64)
    dy, dyv = put(rnd([5, T, K], T, K) * 1e-2, f32)
    dh, dhv = put(rnd([6, T, K], T, K) * 1e-2, f32) if T % 2 else (None, 0.0)
    g, gv = put(1 + 0.2 * rnd([7, K], K), T % 3 != 0)
    dx, bound, dg, bg = norm_gradient(h, dyv.astype(np.float64), gv.astype(np.float64), T)
    dx = dx + dhv
    dX, dgain = sbn.sbn_rmsnorm_backward_kept(dy, kept, g, eps=EPS, dH=dh)
    close(get(dX, f32), dx, bound + 2 * U * np.abs(dx) + (0 if f32 else B) * np.abs(dx), "dX")
    close(host(dgain), dg, bg, "dgain")


def act64(a, act):
    """f, f' and the bound's parts in units of u."""
    if act == sbn.SBN_RELU2:
        r = np.maximum(a, 0)
        return r * r, 2 * r, np.zeros_like(a)
    with np.errstate(over="ignore"):
        g = 1 / (1 + np.exp(-a))
    return a * g, g * (1 + a * (1 - g)), 12 * (g + np.abs(a) * g)


ACTS = [sbn.SBN_RELU2, sbn.SBN_SILU]


@pytest.mark.parametrize("gated,norm", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,K", SHAPES)
def test_activation(T, K, f32, act, gated, norm):
    F = 3 if act == sbn.SBN_RELU2 else 8
    a, av = put(rows(1, T, K), f32)
    b, bv = put(rnd([2, T, K], T, K), f32) if gated else (None, None)
    g, gv = put(1 + 0.2 * rnd([3, K], K), T % 3 != 0) if norm else (None, None)
    Xq, s_x, ka, kb = sbn.sbn_activation_quant(a, b, act=act, gain=g, eps=EPS)
    same_kept(ka, av, "A")
    if gated:
        same_kept(kb, bv, "B")
    else:
        assert kb is None
    u = act64(av.astype(np.float64), act)[0]
    if gated:
        u = u * bv.astype(np.float64)
    r = 1 / np.sqrt((u ** 2).mean(1) + EPS) if norm else np.ones(T)
    v = u * gv.astype(np.float64) if norm else u
    m = np.maximum(np.abs(v).max(1), float(TINY))
    if act == sbn.SBN_RELU2:
        p = np.maximum(av, np.float32(0))
        p = (p * p).astype(np.float32)
        p = (p * bv).astype(np.float32) if gated else p
        q, mf = codes_of(p, gv if norm else np.float32(1.0))
        assert np.array_equal(host(Xq), q), "codes"
    err = np.abs(host(Xq).astype(np.float64) * (m / 127)[:, None] - v)
    assert (err <= (m * (0.5 / 127 + 3 * (F + 1) * U))[:, None]).all(), "codes against 64 bits"
    close(host(s_x), m * r / 127, ((2 * F + 40) * U) * m * r / 127, "s_x")
    # nothing kept: the same activations
    Xn, s_n, na, nbb = sbn.sbn_activation_quant(a, b, act=act, gain=g, eps=EPS, keep=False)
    assert na is None and nbb is None and np.array_equal(host(Xn), host(Xq)) and np.array_equal(host(s_n), host(s_x))

    # the gradient, from what was kept
    dy, dyv = put(rnd([5, T, K], T, K) * 1e-2, f32)
    A64 = host(sbn.sbn_keep8_decode(ka)).astype(np.float64)
    B64 = host(sbn.sbn_keep8_decode(kb)).astype(np.float64) if gated else 1.0
    f, slope, bs = act64(A64, act)
    du, bd = dyv.astype(np.float64), np.zeros((T, K))
    dA, dB, dgain = sbn.sbn_activation_backward(dy, ka, kb, act=act, gain=g, eps=EPS)
    if norm:
        du, bd, dg, bg = norm_gradient(f * B64, du, gv.astype(np.float64), T, F)
        close(host(dgain), dg, bg, "dgain")
    else:
        assert dgain is None
    more = (4 if act == sbn.SBN_RELU2 else 20) * U
    dAr = du * B64 * slope
    close(get(dA, f32), dAr, bd * np.abs(B64 * slope) + U * np.abs(du * B64) * bs + more * np.abs(dAr) + (0 if f32 else B) * np.abs(dAr), "dA")
    if gated:
        dBr = du * f
        close(get(dB, f32), dBr, bd * np.abs(f) + more * np.abs(dBr) + (0 if f32 else B) * np.abs(dBr), "dB")
    else:
        assert dB is None


@pytest.mark.parametrize("f32", [False, True])
def test_sigmoid_of_extremes(f32):
    """Rows of one value each, up to the largest, where u stays finite.  A sigmoid g below 2^-126
    has no full mantissa (or is 0), an error of at most 2^-126: of f = a g |a| 2^-126, of f' = g (1 + a (1 - g)),
    with 0 <= 1 - g <= 1, (1 + |a|) 2^-126.  From a = -128 on g < 2^-184, so both are 0 in float32."""
    vals = np.array([0.0, 1e-30, -1e-30, 1.0, -1.0, 17.0, -17.0, 60.0, -60.0, 88.5, -88.5, 89.0, -89.0, 127.0, -127.0, 200.5, -200.5, 1e4,
                     -1e4, 1e30, -1e30, 2.3e38, -2.3e38, 3e38, -3e38], dtype=np.float32)
    a, av = put(np.repeat(vals[:, None], 40, 1), f32)
    Xq, s_x, ka, _ = sbn.sbn_activation_quant(a, act=sbn.SBN_SILU)
    u = act64(av.astype(np.float64), sbn.SBN_SILU)[0]
    m = np.maximum(np.abs(u).max(1), float(TINY))
    tiny = 2.0 ** -126 * (1 + np.minimum(np.abs(av.astype(np.float64)), 128))
    close(host(s_x), m / 127, 60 * U * m / 127 + tiny[:, 0] / 127 + 2.0 ** -149, "s_x")
    assert (np.abs(host(Xq) * host(s_x)[:, None].astype(np.float64) - u) <= (m * (0.5 / 127 + 60 * U))[:, None] + tiny).all()
    f, slope, bs = act64(host(sbn.sbn_keep8_decode(ka)).astype(np.float64), sbn.SBN_SILU)
    dy, dyv = put(np.full(av.shape, 0.5, dtype=np.float32), f32)
    dA, _, _ = sbn.sbn_activation_backward(dy, ka, act=sbn.SBN_SILU)
    close(get(dA, f32), 0.5 * slope, U * 0.5 * bs + 20 * U * np.abs(slope) + (0 if f32 else B) * np.abs(slope) + tiny, "dA")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,K", [(37, 520), (1100, 520), (300, 9000), (300, 14344), (37, 16400)])
def test_halves_of_one_matrix_in_place(T, K, f32):
    """A and B as halves of one product's output, dA in dY's place, outputs given, columns beside them untouched."""
    import torch
    both, _ = put(np.concatenate([rows(1, T, K), rnd(2, T, K)], 1), f32)
    A, Bm = both[:, :K], both[:, K:]
    g = dev(1 + 0.2 * rnd(3, K))
    ref = sbn.sbn_activation_quant(A.contiguous(), Bm.contiguous(), act=sbn.SBN_RELU2, gain=g)
    kept = [sbn.Kept8(torch.empty_like(k.codes), torch.empty_like(k.scales)) for k in ref[2:]]
    got = sbn.sbn_activation_quant(A, Bm, act=sbn.SBN_RELU2, gain=g, kept_A=kept[0], kept_B=kept[1])
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    for k, q in zip(kept, ref[2:]):
        assert torch.equal(k.codes, q.codes) and torch.equal(k.scales, q.scales)
    wide = torch.full((T, 3 * K + 8), 7.0, dtype=both.dtype, device="cuda")
    dy = wide[:, :K]
    dy.copy_(put(rnd(4, T, K) * 1e-2, f32)[0])
    rA, rB, rg = sbn.sbn_activation_backward(dy.contiguous(), *kept, act=sbn.SBN_RELU2, gain=g)
    dA, dB, dg = sbn.sbn_activation_backward(dy, *kept, act=sbn.SBN_RELU2, gain=g, dA=dy, dB=wide[:, K:2 * K])
    assert dA.data_ptr() == dy.data_ptr() and torch.equal(dA, rA) and torch.equal(dB, rB) and torch.equal(dg, rg)
    assert (wide[:, 2 * K:] == 7.0).all()
    dy.copy_(rA)
    rB2 = sbn.sbn_activation_backward(dy.contiguous(), *kept, act=sbn.SBN_SILU)
    dB2 = sbn.sbn_activation_backward(dy, *kept, act=sbn.SBN_SILU, dB=dy)
    assert torch.equal(dB2[0], rB2[0]) and torch.equal(dy, rB2[1])
    # the norm's: the residual stream in place, dX in dH's and in dY's place
    x, r = A.contiguous(), Bm.contiguous()
    Xq, s_x, H, k8 = sbn.sbn_rmsnorm_quant_keep(x, g, residual=r.clone())
    r2 = r.clone()
    Xq2, _, H2, k2 = sbn.sbn_rmsnorm_quant_keep(x, g, residual=r2, H=r2)
    assert H2 is r2 and torch.equal(r2, H) and torch.equal(Xq, Xq2) and torch.equal(k8.codes, k2.codes)
    dX, dg = sbn.sbn_rmsnorm_backward_kept(rA, k8, g, dH=rB)
    for at in ("dY", "dH"):
        y, h = rA.clone(), rB.clone()
        d2, g2 = sbn.sbn_rmsnorm_backward_kept(y, k8, g, dH=h, dX=y if at == "dY" else h)
        assert torch.equal(d2, dX) and torch.equal(g2, dg)


def test_nothing_to_do():
    import torch
    for dt in (torch.bfloat16, torch.float32):
        x = torch.empty((0, 256), dtype=dt, device="cuda")
        g = torch.ones(256, device="cuda")
        Xq, s_x, H, kept = sbn.sbn_rmsnorm_quant_keep(x, g, residual=x)
        assert Xq.shape == (0, 256) and s_x.shape == (0,) and kept.scales.shape == (0, 2)
        dX, dg = sbn.sbn_rmsnorm_backward_kept(x, kept, g)
        assert dX.shape == (0, 256) and (dg == 0).all()
        Xq, s_x, ka, kb = sbn.sbn_activation_quant(x, x, act=sbn.SBN_SILU, gain=g)
        dA, dB, dg = sbn.sbn_activation_backward(x, ka, kb, act=sbn.SBN_SILU, gain=g)
        assert dA.shape == dB.shape == (0, 256) and (dg == 0).all()
        assert sbn.sbn_keep8_decode(sbn.sbn_keep8_encode(x)).shape == (0, 256)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [True, False])
def test_gradient_against_differences(act, gated):
    """Along random directions, dA, dB and dgain (float32) against central differences, in 64
    bits, of sum(dY * norm(f(a) b) gain) at the kept values.  Step 1e-5: the third-order term is
    under 1e-8 of the direction's size, the differences' own rounding under 1e-9 of it; the
    gradients' is under 1e-5 of |gradient| summed over the direction (some 200 u)."""
    import torch
    T, K, h = 9, 264, 1e-5
    a, b, dy = dev(rnd(1, T, K)), dev(rnd(2, T, K)), dev(rnd(3, T, K))
    g = dev(1 + 0.2 * rnd(4, K))
    ka = sbn.sbn_keep8_encode(a)
    kb = sbn.sbn_keep8_encode(b) if gated else None
    dA, dB, dg = sbn.sbn_activation_backward(dy, ka, kb, act=act, gain=g, eps=EPS)

    def L(a, b, g):
        f = torch.relu(a) ** 2 if act == sbn.SBN_RELU2 else a * torch.sigmoid(a)
        u = f * b if gated else f
        return (dy.double() * u * torch.rsqrt((u * u).mean(1, keepdim=True) + EPS) * g).sum()

    at = [sbn.sbn_keep8_decode(ka).double(), sbn.sbn_keep8_decode(kb).double() if gated else None, g.double()]
    gen = torch.Generator(device="cuda").manual_seed(7)
    for i, grad in enumerate((dA, dB, dg)):
        if grad is None:
            continue
        e = torch.randn(grad.shape, generator=gen, device="cuda", dtype=torch.float64)
        up, dn = list(at), list(at)
        up[i], dn[i] = at[i] + h * e, at[i] - h * e
        num = (L(*up) - L(*dn)) / (2 * h)
        size = float((e.abs() * grad.double().abs()).sum())
        assert abs(float((grad.double() * e).sum() - num)) <= 1e-5 * size + 1e-6


def test_gradient_of_the_norm_is_orthogonal_to_the_kept_row():
    """Scaling a row does not change its norm: dX (without dH, eps next to nothing) has no part along h."""
    T, K = 20, 1024
    kept = sbn.sbn_keep8_encode(dev(rnd(1, T, K)))
    dX, _ = sbn.sbn_rmsnorm_backward_kept(dev(rnd(2, T, K)), kept, dev(1 + 0.2 * rnd(3, K)), eps=0.0)
    h, d = host(sbn.sbn_keep8_decode(kept)).astype(np.float64), host(dX).astype(np.float64)
    assert (np.abs((h * d).sum(1)) <= 300 * U * (np.abs(h) * np.abs(d)).sum(1)).all()


def test_captured():
    import torch
    T, K = 70, 520
    a, b, dy = (dev(rnd(i, T, K)).bfloat16() for i in range(3))
    g = dev(1 + 0.2 * rnd(3, K))
    new = lambda: sbn.Kept8(torch.empty((T, K), dtype=torch.int8, device="cuda"), torch.empty((T, 5), device="cuda"))  # noqa: E731
    ka, kb, kh = new(), new(), new()
    Xq, Xn = (torch.empty((T, K), dtype=torch.int8, device="cuda") for _ in range(2))
    s_x, s_n = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dA, dB, dX, H = (torch.empty_like(a) for _ in range(4))
    dg, dn = torch.empty(K, device="cuda"), torch.empty(K, device="cuda")

    def step():
        sbn.sbn_activation_quant(a, b, act=sbn.SBN_SILU, gain=g, Xq=Xq, s_x=s_x, kept_A=ka, kept_B=kb)
        sbn.sbn_activation_backward(dy, ka, kb, act=sbn.SBN_SILU, gain=g, dA=dA, dB=dB, dgain=dg)
        sbn.sbn_rmsnorm_quant_keep(a, g, residual=b, H=H, Xq=Xn, s_x=s_n, kept=kh)
        sbn.sbn_rmsnorm_backward_kept(dA, kh, g, dH=dB, dX=dX, dgain=dn)

    replay_matches(step, [Xq, s_x, *ka, *kb, *kh, Xn, s_n, dA, dB, dX, H, dg, dn])


def test_streams_at_once():
    """Two streams at once, and calls given a stream, do not share scratch."""
    import torch
    T, K = 700, 1024
    g = dev(1 + 0.2 * rnd(3, K))
    sets = [(dev(rnd(i, T, K)), dev(rnd(10 + i, T, K)), dev(rnd(20 + i, T, K))) for i in range(2)]

    def work(a, b, dy, **kw):
        Xq, s_x, ka, kb = sbn.sbn_activation_quant(a, b, act=sbn.SBN_RELU2, gain=g, **kw)
        dA, dB, dg = sbn.sbn_activation_backward(dy, ka, kb, act=sbn.SBN_RELU2, gain=g, **kw)
        dX, dn = sbn.sbn_rmsnorm_backward_kept(dA, ka, g, dH=dB, **kw)
        return Xq, s_x, dA, dB, dg, dX, dn, sbn.sbn_keep8_decode(sbn.sbn_keep8_encode(dX, **kw), **kw)

    ref = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for given in (False, True):
        got = []
        for s, x in zip(streams, sets):
            if given:
                got.append(work(*x, stream=s))
            else:
                with torch.cuda.stream(s):
                    got.append(work(*x))
        torch.cuda.synchronize()
        for a, b in zip(ref, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_many_elements():
    """Offsets past 2^31 elements: the last rows as in a call of their own."""
    import torch
    T, K, last = 67000, 32768, 40                    # 2.2e9 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    for t in range(0, T, 8000):
        a[t: t + 8000] = torch.randn(min(8000, T - t), K, generator=g, device="cuda", dtype=torch.bfloat16)
    gain = torch.linspace(0.5, 1.5, K, device="cuda")
    Xq, s_x, ka, _ = sbn.sbn_activation_quant(a, act=sbn.SBN_RELU2, gain=gain)
    dA, _, _ = sbn.sbn_activation_backward(a, ka, act=sbn.SBN_RELU2, gain=gain)
    e = sbn.sbn_keep8_encode(a)
    y = sbn.sbn_keep8_decode(e, dt=sbn.SBN_BF16)
    tail = a[-last:].contiguous()
    Xt, st, kt, _ = sbn.sbn_activation_quant(tail, act=sbn.SBN_RELU2, gain=gain)
    dt, _, _ = sbn.sbn_activation_backward(tail, kt, act=sbn.SBN_RELU2, gain=gain)
    assert torch.equal(Xq[-last:], Xt) and torch.equal(s_x[-last:], st) and torch.equal(dA[-last:], dt)
    for k in (ka, e):
        assert torch.equal(k.codes[-last:], kt.codes) and torch.equal(k.scales[-last:], kt.scales)
    assert torch.equal(y[-last:], sbn.sbn_keep8_decode(kt, dt=sbn.SBN_BF16))


@pytest.mark.parametrize("gain", [True, False])
def test_many_short_rows(gain):
    """More rows than a grid has blocks (2^20): the last ones as in a call of their own."""
    import torch
    T, K, last = 2 ** 20 + 77, 40, 100
    g = torch.Generator(device="cuda").manual_seed(2)
    a, b = (torch.randn(T, K, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = torch.linspace(0.5, 1.5, K, device="cuda") if gain else None

    def work(a, b):
        Xq, s_x, ka, kb = sbn.sbn_activation_quant(a, b, act=sbn.SBN_SILU, gain=w)
        dA, dB, _ = sbn.sbn_activation_backward(b, ka, kb, act=sbn.SBN_SILU, gain=w)
        out = [Xq, s_x, *ka, *kb, dA, dB]
        if gain:
            Xn, s_n, H, kh = sbn.sbn_rmsnorm_quant_keep(a, w, residual=b)
            out += [Xn, s_n, H, *kh, sbn.sbn_rmsnorm_backward_kept(b, kh, w, dH=a)[0]]
        return out

    for x, y in zip(work(a, b), work(a[-last:].contiguous(), b[-last:].contiguous())):
        assert torch.equal(x[-last:], y)


def test_more_threads_than_a_launch_takes():
    """Checkpoints of so many short rows that they are taken in two launches."""
    import torch
    T, K, last = 2 ** 27 + 9, 8, 3 * 2 ** 20                        # 16 threads a row
    x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    for t in range(0, T, 2 ** 25):
        n = min(2 ** 25, T - t)
        x[t: t + n] = (torch.arange(t, t + n, device="cuda") % 8191 - 4000)[:, None] * torch.arange(1, K + 1, device="cuda")
    kept, launched = launches(lambda: sbn.sbn_keep8_encode(x))
    assert launched["keep8_encode"] == 2
    tail = sbn.sbn_keep8_encode(x[-last:].contiguous())
    assert torch.equal(kept.codes[-last:], tail.codes) and torch.equal(kept.scales[-last:], tail.scales)
    assert torch.equal(sbn.sbn_keep8_decode(kept, dt=sbn.SBN_BF16)[-last:], sbn.sbn_keep8_decode(tail, dt=sbn.SBN_BF16))


def test_finite_check(monkeypatch):
    monkeypatch.setenv("SBN_CHECK_FINITE", "1")
    a, g = dev(rnd(1, 4, 64)), dev(rnd(2, 64))
    bad = a.clone()
    bad[2, 3] = float("inf")
    Xq, s_x, ka, kb = sbn.sbn_activation_quant(a, a, act=sbn.SBN_SILU, gain=g)
    for f in (lambda: sbn.sbn_activation_quant(bad, a, act=sbn.SBN_SILU), lambda: sbn.sbn_activation_quant(a, bad, act=sbn.SBN_SILU),
              lambda: sbn.sbn_activation_backward(bad, ka, kb, act=sbn.SBN_SILU), lambda: sbn.sbn_keep8_encode(bad),
              lambda: sbn.sbn_rmsnorm_quant_keep(a, g, residual=bad), lambda: sbn.sbn_rmsnorm_backward_kept(a, ka, g, dH=bad)):
        with pytest.raises(sbn.SbnError) as e:
            f()
        assert e.value.status == sbn.SBN_ERR_VALUE
