"""The C ABI of include/sbn_keep.h and its binding without a GPU: exported symbols and
refusals, which come before any launch (fake device addresses that nothing dereferences)."""
from __future__ import annotations

import ctypes

import pytest

import sparse_linear_layers_02_amd as sbn
from test_train_abi import ALIGN, BF16, DTYPE, F32, MIS, NULL, ODD, OK, P, P2, P3, SHAPE, VALUE, WS

Q = [ctypes.c_void_p(0x400000 + 0x100000 * i) for i in range(8)]


@pytest.fixture(scope="module")
def L():
    return sbn.lib()


def test_exports_every_header_symbol(L):
    names = sbn.keep_header_symbols()
    assert len(names) == 8 and all(hasattr(L, n) for n in names)
    assert not set(names) & set(sbn.header_symbols()) and not set(names) & set(sbn.train_header_symbols())
    ours = {n for n in dir(sbn.keeping) if n.startswith("sbn_") or n in ("Kept8", "SBN_KEEP_BLOCK", "SBN_RELU2", "SBN_SILU")}
    assert ours <= set(sbn.__all__) and all(getattr(sbn, n) is getattr(sbn.keeping, n) for n in ours)


def refusals(call, cases):
    for kw, status in cases:
        assert call(**kw) == status, kw
        assert sbn.lib().sbn_last_error() != b""


def test_checkpoints(L):
    base = dict(X=P, ld=64, dt=BF16, T=4, K=64, q=P2, s=P3)

    def enc(**kw):
        a = {**base, **kw}
        return L.sbn_keep8_encode(a["X"], a["ld"], a["dt"], a["T"], a["K"], a["q"], a["s"], None)

    def dec(**kw):
        a = {**base, **kw}
        return L.sbn_keep8_decode(a["q"], a["s"], a["T"], a["K"], a["X"], a["ld"], a["dt"], None)

    for call in (enc, dec):
        assert call(T=0, X=None, q=None, s=None) == OK
        refusals(call, [(dict(X=None), NULL), (dict(q=None), NULL), (dict(s=None), NULL), (dict(T=-1), SHAPE),
                        (dict(K=60), SHAPE), (dict(K=0), SHAPE), (dict(K=32776), SHAPE), (dict(T=1 << 36), SHAPE),
                        (dict(ld=56), SHAPE), (dict(ld=68), ALIGN), (dict(dt=2), DTYPE), (dict(X=MIS), ALIGN),
                        (dict(q=MIS), ALIGN), (dict(s=ODD), ALIGN), (dict(q=P), SHAPE), (dict(s=P), SHAPE)])


def test_norm(L):
    base = dict(X=P, ldx=64, res=P2, ldr=64, dt=BF16, gain=P3, gdt=F32, T=4, K=64, eps=1e-6, H=P2, ldh=64, Xq=Q[0], s=Q[1],
                q=Q[2], qs=Q[3])

    def call(**kw):
        a = {**base, **kw}
        return L.sbn_rmsnorm_quant_keep(*(a[k] for k in base), None)

    assert call(T=0, X=None, gain=None, Xq=None, q=None) == OK
    refusals(call, [(dict(X=None), NULL), (dict(gain=None), NULL), (dict(H=None), NULL), (dict(Xq=None), NULL),
                    (dict(s=None), NULL), (dict(q=None), NULL), (dict(qs=None), NULL), (dict(K=60), SHAPE), (dict(T=-1), SHAPE),
                    (dict(ldx=56), SHAPE), (dict(ldr=68), ALIGN), (dict(dt=3), DTYPE), (dict(gdt=2), DTYPE),
                    (dict(eps=-1.0), VALUE), (dict(eps=float("inf")), VALUE), (dict(q=MIS), ALIGN), (dict(qs=ODD), ALIGN),
                    (dict(Xq=P), SHAPE), (dict(q=P), SHAPE), (dict(q=Q[0]), SHAPE), (dict(qs=Q[1]), SHAPE), (dict(q=P2), SHAPE),
                    (dict(H=P2, ldh=72), SHAPE)])

    back = dict(dY=P, lddy=64, dH=P2, lddh=64, dt=F32, q=Q[0], qs=Q[1], gain=P3, gdt=BF16, T=4, K=64, eps=1e-6, dX=Q[2],
                lddx=64, dg=Q[3], ws=Q[4], wsb=1 << 20)

    def grad(**kw):
        a = {**back, **kw}
        return L.sbn_rmsnorm_backward_kept(*(a[k] for k in back), None)

    refusals(grad, [(dict(dY=None), NULL), (dict(q=None), NULL), (dict(qs=None), NULL), (dict(gain=None), NULL),
                    (dict(dX=None), NULL), (dict(dg=None), NULL), (dict(ws=None), NULL), (dict(wsb=256), WS), (dict(K=12), SHAPE),
                    (dict(lddy=32), SHAPE), (dict(lddh=66), ALIGN), (dict(dt=3), DTYPE), (dict(gdt=3), DTYPE),
                    (dict(eps=float("nan")), VALUE), (dict(dH=MIS), ALIGN), (dict(dX=P, lddx=128), SHAPE),
                    (dict(dX=P2, lddx=128), SHAPE), (dict(dX=Q[0]), SHAPE), (dict(dg=MIS), ALIGN)])
    b = ctypes.c_size_t()
    for f in (L.sbn_rmsnorm_backward_kept_workspace_bytes, L.sbn_activation_backward_workspace_bytes):
        assert f(4, 64, ctypes.byref(b)) == OK and b.value == 1024
        assert f(4, 64, None) == NULL and f(4, 63, ctypes.byref(b)) == SHAPE


def test_activation(L):
    base = dict(A=P, lda=64, B=P2, ldb=64, dt=BF16, act=0, gain=P3, gdt=F32, T=4, K=64, eps=1e-6, Xq=Q[0], s=Q[1], qa=Q[2],
                sa=Q[3], qb=Q[4], sb=Q[5])

    def call(**kw):
        a = {**base, **kw}
        return L.sbn_activation_quant(*(a[k] for k in base), None)

    assert call(T=0, A=None, Xq=None, qa=None) == OK
    refusals(call, [(dict(A=None), NULL), (dict(Xq=None), NULL), (dict(s=None), NULL), (dict(qa=None), NULL),
                    (dict(sa=None), NULL), (dict(qb=None), NULL), (dict(sb=None), NULL), (dict(B=None), NULL),
                    (dict(qa=None, sa=None), NULL), (dict(act=2), VALUE), (dict(act=-1), VALUE), (dict(K=60), SHAPE),
                    (dict(lda=56), SHAPE), (dict(ldb=68), ALIGN), (dict(dt=2), DTYPE), (dict(gdt=2), DTYPE),
                    (dict(eps=-1.0), VALUE), (dict(B=MIS), ALIGN), (dict(gain=MIS), ALIGN), (dict(qb=MIS), ALIGN),
                    (dict(sb=ODD), ALIGN), (dict(Xq=P), SHAPE), (dict(qa=P2), SHAPE), (dict(qb=Q[2]), SHAPE),
                    (dict(sb=Q[3]), SHAPE)])

    back = dict(dY=P, lddy=64, dt=F32, qa=Q[0], sa=Q[1], qb=Q[2], sb=Q[3], act=1, gain=P3, gdt=F32, T=4, K=64, eps=1e-6,
                dA=Q[4], ldda=64, dB=Q[5], lddb=64, dg=Q[6], ws=Q[7], wsb=1 << 20)

    def grad(**kw):
        a = {**back, **kw}
        return L.sbn_activation_backward(*(a[k] for k in back), None)

    assert grad(T=0, gain=None, dg=None) == OK
    refusals(grad, [(dict(dY=None), NULL), (dict(qa=None), NULL), (dict(sa=None), NULL), (dict(qb=None), NULL),
                    (dict(sb=None), NULL), (dict(dB=None), NULL), (dict(dA=None), NULL), (dict(dg=None), NULL),
                    (dict(gain=None), NULL), (dict(ws=None), NULL), (dict(wsb=256), WS), (dict(act=2), VALUE),
                    (dict(eps=float("nan")), VALUE), (dict(lddy=32), SHAPE), (dict(lddb=66), ALIGN), (dict(dt=3), DTYPE),
                    (dict(gdt=3), DTYPE), (dict(dB=Q[4]), SHAPE), (dict(dA=P, ldda=128), SHAPE), (dict(dB=P, lddb=128), SHAPE),
                    (dict(dA=Q[0]), SHAPE), (dict(dB=Q[1]), SHAPE), (dict(dA=MIS), ALIGN)])


def test_binding_refuses():
    import torch
    bf, f32, i8 = torch.bfloat16, torch.float32, torch.int8
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt)  # noqa: E731
    k = lambda T, K: sbn.Kept8(z(T, K, dt=i8), z(T, -(-K // 128), dt=f32))  # noqa: E731
    wide = sbn.Kept8(z(4, 128, dt=i8)[:, :64], z(4, 1, dt=f32))
    bad = [
        lambda: sbn.sbn_keep8_encode(z(4, 64, dt=torch.float16)),
        lambda: sbn.sbn_keep8_encode(z(64, 4).t()),
        lambda: sbn.sbn_keep8_encode(z(64)),
        lambda: sbn.sbn_keep8_encode(z(4, 64), kept=k(4, 128)),
        lambda: sbn.sbn_keep8_encode(z(4, 64), kept=wide),
        lambda: sbn.sbn_keep8_decode(z(4, 64, dt=i8)),
        lambda: sbn.sbn_keep8_decode((z(4, 64, dt=i8), z(4, 2, dt=f32))),
        lambda: sbn.sbn_keep8_decode((z(4, 64, dt=torch.uint8), z(4, 1, dt=f32))),
        lambda: sbn.sbn_keep8_decode(k(4, 64), dt=2),
        lambda: sbn.sbn_keep8_decode(k(4, 64), Y=z(4, 72)),
        lambda: sbn.sbn_rmsnorm_quant_keep(z(4, 64), z(32)),
        lambda: sbn.sbn_rmsnorm_quant_keep(z(4, 64), z(64), H=z(4, 64)),
        lambda: sbn.sbn_rmsnorm_quant_keep(z(4, 64), z(64), residual=z(4, 64, dt=f32)),
        lambda: sbn.sbn_rmsnorm_quant_keep(z(4, 64), z(64), Xq=z(4, 64)),
        lambda: sbn.sbn_rmsnorm_backward_kept(z(4, 64), k(5, 64), z(64)),
        lambda: sbn.sbn_rmsnorm_backward_kept(z(4, 64), k(4, 64), z(64), dX=z(4, 64, dt=f32)),
        lambda: sbn.sbn_rmsnorm_backward_kept(z(4, 64), k(4, 64), z(64), ws=z(1 << 16, dt=torch.uint8)[::2]),
        lambda: sbn.sbn_activation_quant(z(4, 64), z(4, 72), act=0),
        lambda: sbn.sbn_activation_quant(z(4, 64), z(4, 64, dt=f32), act=0),
        lambda: sbn.sbn_activation_quant(z(4, 64), act=0, kept_B=k(4, 64)),
        lambda: sbn.sbn_activation_quant(z(4, 64), act=0, keep=False, kept_A=k(4, 64)),
        lambda: sbn.sbn_activation_quant(z(4, 64), act=0, s_x=z(5, dt=f32)),
        lambda: sbn.sbn_activation_backward(z(4, 64), k(4, 64), act=0, dB=z(4, 64)),
        lambda: sbn.sbn_activation_backward(z(4, 64), k(4, 64), act=0, dgain=z(64, dt=f32)),
        lambda: sbn.sbn_activation_backward(z(4, 64), k(4, 64), k(4, 128), act=0),
        lambda: sbn.sbn_activation_backward(z(4, 64), k(4, 64), act=0, gain=z(64), ws=torch.zeros(64, device="meta")),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(sbn.SbnError):
            f()
            raise AssertionError(f"case {i} was accepted")
    # layouts that are right, in host memory
    for f in (lambda: sbn.sbn_keep8_encode(z(4, 64)), lambda: sbn.sbn_keep8_decode(k(4, 64)),
              lambda: sbn.sbn_rmsnorm_quant_keep(z(4, 64), z(64)), lambda: sbn.sbn_rmsnorm_backward_kept(z(4, 64), k(4, 64), z(64)),
              lambda: sbn.sbn_activation_quant(z(4, 64), act=0), lambda: sbn.sbn_activation_backward(z(4, 64), k(4, 64), act=0)):
        with pytest.raises(sbn.SbnError) as e:
            f()
        assert e.value.status == SHAPE and "GPU" in str(e.value)
