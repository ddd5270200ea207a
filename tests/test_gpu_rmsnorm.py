"""RMS norm with the residual's addition, its 8-bit output and its gradient,
against the formulas in 64 bits (numpy).

Bounds, with u = 2^-24 (float32) and b = 2^-8 (bf16), each a worst case:
  rstd   a sum of squares of K terms is summed 32 or fewer in a row and then in
         a tree, so its relative error is under 48 u; the root halves it, and
         mean, root and quotient add 4 u: 28 u, taken as 32 u
  y      rstd's, and three more roundings: 36 u |y|, plus b |y| for bf16
  codes  equal: u = h gain, max, 127 u / a have one float32 rounding each, in
         any order of the sums
  s_x    rstd's, and two roundings: 34 u
  dX     with w = gain dy, n = h rstd, c = mean(w n): c's error is under
         (48 + 6) u mean|w n|; dX's under u (rstd (6|w| + 8|n c| + 54 |n| mean|w n|) + |dX|),
         plus b |dX| for bf16
  dgain  at most ceil(T/512) + 48 terms in a row: (ceil(T/512) + 52) u sum|dy n|
"""
from __future__ import annotations

import numpy as np
import pytest

import sparse_linear_layers_02_amd as sbn
from gpu_util import dev, dev_bf16, host
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
EPS = 1e-6


def rnd(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape, dtype=np.float32)


def put(a, f32, ld=None):
    """`a` on the device as float32 or bf16, rows at stride ld; and its value as stored, float32."""
    import torch
    if f32:
        t, v = dev(a), a.astype(np.float32)
    else:
        bits = f32_to_bf16_bits(a)
        t, v = dev_bf16(bits), bf16_bits_to_f32(bits)
    if ld is not None and a.ndim == 2:
        wide = torch.full((a.shape[0], ld), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, : a.shape[1]] = t
        t = wide[:, : a.shape[1]]
    return t, v


def get(t, f32):
    return host(t) if f32 else bf16_bits_to_f32(host(t.contiguous()))


def reference(x, r, g, f32):
    h = x if r is None else (x + r).astype(np.float32)
    if r is not None and not f32:
        h = bf16_bits_to_f32(f32_to_bf16_bits(h))
    hd = h.astype(np.float64)
    rstd = 1.0 / np.sqrt((hd ** 2).mean(1) + EPS)
    return h, rstd, hd * rstd[:, None] * g.astype(np.float64)


def codes_of(h, g):
    u = (h * g).astype(np.float32)
    a = np.maximum(np.abs(u).max(1), np.float32(2.0 ** -100))
    return np.rint((np.float32(127.0) * u) / a[:, None]).astype(np.int8), a


def close(got, ref, bound, what):
    err = np.abs(got.astype(np.float64) - ref)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(err / np.maximum(bound, 1e-300)):.3g} bounds"


SHAPES = [(1, 8), (1, 2560), (2, 64), (3, 72), (5, 1000), (17, 2048), (63, 4104), (257, 512), (7, 8192), (4, 8200),
          (3, 16384), (2, 16392), (2, 32768), (1025, 328), (2050, 2560), (1030, 4096)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,K", SHAPES)
def test_forward(T, K, f32):
    gain_f32 = (T + K) % 3 != 0
    res = T % 2 == 1
    x, xv = put(rnd([1, T, K], T, K) * 3, f32)
    r, rv = put(rnd([2, T, K], T, K) * 2, f32) if res else (None, None)
    g, gv = put(1 + 0.2 * rnd([3, K], K), gain_f32)
    h, rstd, y = reference(xv, rv, gv, f32)
    Y, H, RS = sbn.sbn_rmsnorm(x, g, residual=r, eps=EPS)
    Xq, s_x, H2, RS2 = sbn.sbn_rmsnorm_quant(x, g, residual=r, eps=EPS)
    for t in (H, H2):
        assert np.array_equal(get(t, f32), h), "H"
    for t in (RS, RS2):
        close(host(t), rstd, 32 * U * rstd, "rstd")
    close(get(Y, f32), y, (36 * U + (0 if f32 else B)) * np.abs(y), "Y")
    q, a = codes_of(h, gv)
    assert np.array_equal(host(Xq), q), "codes"
    s = a.astype(np.float64) * rstd / 127
    close(host(s_x), s, 34 * U * s, "s_x")


@pytest.mark.parametrize("f32", [False, True])
def test_strides_in_place_and_given_outputs(f32):
    import torch
    T, K = 37, 520
    x, xv = put(rnd(11, T, K), f32, 536)
    r, rv = put(rnd(12, T, K), f32, 1040)
    g, gv = put(1 + 0.2 * rnd(13, K), True)
    h, rstd, y = reference(xv, rv, gv, f32)
    Y = torch.full((T, 544), 7.0, dtype=x.dtype, device="cuda")
    out, H, _ = sbn.sbn_rmsnorm(x, g, residual=r, eps=EPS, H=r, Y=Y[:, :K])     # the residual stream in place
    assert H is r and out.data_ptr() == Y.data_ptr()
    assert np.array_equal(get(r, f32), h) and torch.isnan(r.as_strided((T - 1,), (1040,), K)).all()
    close(get(out, f32), y, (36 * U + (0 if f32 else B)) * np.abs(y), "Y")
    assert (Y[:, K:] == 7.0).all(), "columns past the row"
    assert np.array_equal(get(x, f32), xv), "the input"


def test_rows_of_zeros_and_extremes():
    """A zero row has codes 0 and a finite scale; tiny, huge and one-hot rows keep their codes."""
    K = 256
    x = np.zeros((6, K), np.float32)
    x[1, 5] = 1e-30
    x[2] = 1e15 * rnd(21, K)
    x[3, 200] = -4.0
    x[4] = 1e-18 * rnd(22, K)
    x[5] = -0.0
    t, v = put(x, True)
    g, gv = put(np.ones(K, np.float32), True)
    Xq, s_x, H, rstd = sbn.sbn_rmsnorm_quant(t, g, eps=EPS)
    q, a = codes_of(v, gv)
    assert H is t
    assert np.array_equal(host(Xq), q)
    assert not host(Xq)[0].any() and not host(Xq)[5].any() and host(Xq)[3, 200] == -127 and host(Xq)[1, 5] == 127
    ref = a.astype(np.float64) / np.sqrt((v.astype(np.float64) ** 2).mean(1) + EPS) / 127
    close(host(s_x), ref, 34 * U * ref + 2.0 ** -149, "s_x")
    assert np.isfinite(host(rstd)).all()
    y, _, _ = sbn.sbn_rmsnorm(t, g, eps=EPS)
    assert np.isfinite(host(y)).all() and not host(y)[0].any()


def test_feeds_the_sparse_product():
    """The codes and scales go into the layer's calls as sbn_act_quant's do."""
    T, K, R = 24, 256, 64
    x, xv = put(rnd(31, T, K), False)
    g, gv = put(1 + 0.1 * rnd(32, K), False)
    codes, meta, s_w = sbn.sbn_mask_ternarize_pack(dev_bf16(f32_to_bf16_bits(0.02 * rnd(33, R, K))), 2, 4)
    Xq, s_x, _, _ = sbn.sbn_rmsnorm_quant(x, g)
    acc = sbn.sbn_sparse_ternary_gemm(Xq, s_x, codes, meta, s_w, R, 2, 4, ydt=sbn.SBN_I32_ACC)
    y = sbn.sbn_sparse_ternary_gemm(Xq, s_x, codes, meta, s_w, R, 2, 4, ydt=sbn.SBN_F32)
    ref = host(acc).astype(np.float64) * host(s_x)[:, None] * host(s_w)[0]
    close(host(y), ref, 4 * U * np.abs(ref), "Y")
    one = sbn.sbn_sparse_ternary_gemv(Xq[:3], s_x[:3], codes, meta, s_w, R, 2, 4, ydt=sbn.SBN_I32_ACC)
    assert np.array_equal(host(one), host(acc)[:3])


def grads(dy, h, g, rstd, dh):
    dy, h, g, rs = (a.astype(np.float64) for a in (dy, h, g, rstd))
    K = h.shape[1]
    n, w = h * rs[:, None], g * dy
    c = (w * n).mean(1, keepdims=True)
    dx = rs[:, None] * (w - n * c)
    cabs = np.abs(w * n).mean(1, keepdims=True)
    bound = U * rs[:, None] * (6 * np.abs(w) + 8 * np.abs(n * c) + 54 * np.abs(n) * cabs)
    if dh is not None:
        dx = dx + dh
    T = h.shape[0]
    return dx, bound + U * np.abs(dx), (dy * n).sum(0), (-(-T // 512) + 52) * U * np.abs(dy * n).sum(0)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,K", [s for s in SHAPES] + [(1500, 64)])
def test_backward(T, K, f32):
    gain_f32 = (T + K) % 3 == 0
    res = T % 2 == 0
    h, hv = put(rnd([4, T, K], T, K) * 3, f32)
    dy, dyv = put(rnd([5, T, K], T, K) * 1e-2, f32)
    dh, dhv = put(rnd([6, T, K], T, K) * 1e-2, f32) if res else (None, None)
    g, gv = put(1 + 0.2 * rnd([7, K], K), gain_f32)
    rstd = (1.0 / np.sqrt((hv.astype(np.float64) ** 2).mean(1) + EPS)).astype(np.float32)
    dX, dg = sbn.sbn_rmsnorm_backward(dy, h, g, dev(rstd), dH=dh)
    dx, bx, dgr, bg = grads(dyv, hv, gv, rstd, dhv)
    close(get(dX, f32), dx, bx + (0 if f32 else B * np.abs(dx)), "dX")
    close(host(dg), dgr, bg, "dgain")
    again = sbn.sbn_rmsnorm_backward(dy, h, g, dev(rstd), dH=dh)
    assert np.array_equal(get(again[0], f32), get(dX, f32)) and np.array_equal(host(again[1]), host(dg))


def test_backward_strides_and_in_place():
    T, K = 130, 264
    h, hv = put(rnd(41, T, K), False, 280)
    dy, dyv = put(rnd(42, T, K), False, 272)
    dh, dhv = put(rnd(43, T, K), False, 320)
    g, gv = put(1 + 0.2 * rnd(44, K), True)
    rstd = (1.0 / np.sqrt((hv.astype(np.float64) ** 2).mean(1) + EPS)).astype(np.float32)
    dx, bx, dgr, bg = grads(dyv, hv, gv, rstd, dhv)
    out, dg = sbn.sbn_rmsnorm_backward(dy, h, g, dev(rstd), dH=dh, dX=dh)         # the residual stream's gradient in place
    assert out is dh
    close(get(dh, False), dx, bx + B * np.abs(dx), "dX")
    close(host(dg), dgr, bg, "dgain")
    out, _ = sbn.sbn_rmsnorm_backward(dy, h, g, dev(rstd), dX=dy)
    dx, bx, _, _ = grads(dyv, hv, gv, rstd, None)
    close(get(out, False), dx, bx + B * np.abs(dx), "dX in dY's place")


def test_no_rows():
    import torch
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, device="cuda")
    Y, H, rstd = sbn.sbn_rmsnorm(x, g, residual=x)
    Xq, s_x, _, _ = sbn.sbn_rmsnorm_quant(x, g)
    assert Y.shape == (0, 64) and H.shape == (0, 64) and rstd.shape == (0,) and Xq.shape == (0, 64)
    dX, dg = sbn.sbn_rmsnorm_backward(x, x, g, rstd)
    assert dX.shape == (0, 64) and (dg == 0).all() and dg.shape == (64,)


@pytest.mark.parametrize("res", [False, True])
def test_gradient_against_differences(res):
    """L = sum(y o) + sum(h p): the kernel's dX and dgain along random directions
    against central differences of L in 64 bits.  The difference's own error is
    under 1e-8 |L's terms| at a step of 1e-5; the kernel's is its bound, summed
    over the direction."""
    T, K, d = 9, 328, 1e-5
    x = rnd(51, T, K)
    r = rnd(52, T, K) if res else None
    g = 1 + 0.2 * rnd(53, K)
    o, p = rnd(54, T, K), rnd(55, T, K)

    def L(h, gain):
        return (h / np.sqrt((h ** 2).mean(1, keepdims=True) + EPS) * gain * o).sum() + (h * p).sum()

    _, H, rstd = sbn.sbn_rmsnorm(dev(x), dev(g), residual=None if r is None else dev(r), eps=EPS)
    dX, dg = sbn.sbn_rmsnorm_backward(dev(o), H, dev(g), rstd, dH=dev(p))
    hv = host(H).astype(np.float64)
    ex, eg = rnd(56, T, K).astype(np.float64), rnd(57, K).astype(np.float64)
    _, bx, _, bg = grads(o, host(H), g, host(rstd), p)
    g64 = g.astype(np.float64)
    num = (L(hv + d * ex, g64) - L(hv - d * ex, g64)) / (2 * d)
    scale = np.abs(o).sum() + np.abs(p * hv).sum()
    # rstd itself is rounded (32 u), which moves every term of the gradient
    slack = 128 * U * (np.abs(ex) * (np.abs(host(dX)) + np.abs(o * g))).sum()
    assert abs((host(dX) * ex).sum() - num) <= (np.abs(ex) * bx).sum() + slack + 1e-8 * scale / d * 1e-3
    num = (L(hv, g64 + d * eg) - L(hv, g64 - d * eg)) / (2 * d)
    slack = 64 * U * (np.abs(eg) * np.abs(host(dg))).sum() + 64 * U * np.abs(o * hv).sum()
    assert abs((host(dg) * eg).sum() - num) <= (np.abs(eg) * bg).sum() + slack + 1e-8 * scale / d * 1e-3


def test_another_stream():
    import torch
    s = torch.cuda.Stream()
    x, xv = put(rnd(61, 40, 512), False)
    g, gv = put(np.ones(512, np.float32), True)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = sbn.sbn_rmsnorm_quant(x, g)
    s.synchronize()
    b = sbn.sbn_rmsnorm_quant(x, g)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_finite_check(monkeypatch):
    monkeypatch.setenv("SBN_CHECK_FINITE", "1")
    x, _ = put(rnd(71, 4, 64), True)
    g, _ = put(np.ones(64, np.float32), True)
    sbn.sbn_rmsnorm(x, g)
    x[2, 3] = float("inf")
    for f in (lambda: sbn.sbn_rmsnorm(x, g), lambda: sbn.sbn_rmsnorm_quant(x, g), lambda: sbn.sbn_rmsnorm(x * 0 + 1, x[2])):
        with pytest.raises(sbn.SbnError) as e:
            f()
        assert e.value.status == sbn.SBN_ERR_VALUE


@pytest.mark.parametrize("K", [8, 2560, 4104])
def test_rows_near_the_largest_float(K):
    """h gain up to 3e38: neither 127 times a value nor the reciprocal of a row's maximum is a normal float."""
    T = 40
    x, xv = put((rnd([8, K], T, K) * 2e17).astype(np.float32), True)
    gain = np.full(K, 1e20, np.float32)
    g, gv = put(gain, True)
    u = (xv * gv).astype(np.float32)
    a = np.abs(u).max(1)
    assert np.isfinite(a).all() and a.max() > 2.0 ** 125
    q = np.rint((np.float32(127.0) * (u * np.float32(2.0 ** -8))) / (a * np.float32(2.0 ** -8))[:, None]).astype(np.int8)
    Xq, s_x, _, rs = sbn.sbn_rmsnorm_quant(x, g, eps=EPS)
    assert np.array_equal(host(Xq), q)
    ref = a.astype(np.float64) / 127.0 / np.sqrt((xv.astype(np.float64) ** 2).mean(1) + EPS)
    close(host(s_x), ref, 40 * U * ref, "s_x")
