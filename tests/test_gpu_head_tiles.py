"""Every tile shape of the cross entropy's products, whole contractions and split ones,
over the lengths that training has, and vocabularies in three pieces.  Which tiles ran is
read from the names of the launches, so that a change of the rule that chooses them
cannot leave one untested.

Elementwise bounds are those of test_gpu_cross_entropy.py, worst cases that grow with K.
In the norm over all elements the roundings are independent: of D and the result, 2^-9
each, so a gradient is off by under 2^-7 of its own, and lse, which is off by the sums of
K products in float32, by under 2^-16 (some sqrt(K) 2^-24 times the size of a logit)."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_cross_entropy import B, close, make, reference

pytestmark = pytest.mark.gpu


def launches(f):
    """f() and the number of its launches by name."""
    import torch
    torch.cuda.synchronize()
    sbn.sbn_profile_enable(True)
    try:
        sbn.sbn_profile_reset()
        out = f()
        torch.cuda.synchronize()
        return out, {name: n for name, (n, _) in sbn.sbn_profile_dump().items()}
    finally:
        sbn.sbn_profile_enable(False)
        sbn.sbn_profile_reset()


def check(T, V, K, dxdt=None, dwdt=None):
    """The names and numbers of the launches of a loss and its gradients, both held to the reference."""
    f = sbn.SBN_F32
    dxdt, dwdt = f if dxdt is None else dxdt, f if dwdt is None else dwdt
    X, W, y, d = make(T, V, K, T + V + K)
    r = reference(X, W, y, d)
    (loss, lse), ran = launches(lambda: sbn.sbn_cross_entropy(X, W, y))
    close(lse, r["lse"], r["blse"], "lse")
    close(loss, r["loss"], 2 * r["blse"], "loss")
    assert (lse.double() - r["lse"]).norm() <= 2.0 ** -16 * r["lse"].norm()
    (dX, dW), more = launches(lambda: sbn.sbn_cross_entropy_backward(X, W, y, lse, d, dxdt=dxdt, dwdt=dwdt))
    for got, ref, bound, what in ((dX, r["dX"], r["bX"], "dX"), (dW, r["dW"], r["bW"], "dW")):
        close(got, ref, bound + (0 if got.dtype.itemsize == 4 else B * ref.abs()), what)
        assert (got.double() - ref).norm() <= 2.0 ** -7 * ref.norm(), what
    ran.update(more)
    for name in ("ce_join", "ce_gmax"):
        ran.pop(name, None)
    return ran


# tokens, entries, K: tiles of the logits and of D, of dX, of dW, and sums of parts
TILES = [
    ((8100, 7000, 4096), "wide", "wide", "wide", 0),               # 64 stages, 110 and 127
    ((6077, 1288, 2112), "wide", "wide", "square", 0),
    ((3835, 1384, 2752), "square", "wide", "wide", 1),             # dW in parts
    ((1285, 3664, 3136), "square", "wide", "wide", 1),             # dX in parts
    ((65, 17007, 2112), "square", "square", "wide", 1),            # dX in parts
    ((7304, 756, 2112), "square", "square", "square", 1),          # dW in parts
    ((16, 1796, 2112), "flat", "flat", "square", 1),               # dX in parts
    ((17, 734, 2112), "flat", "flat", "flat", 0),
    ((5000, 300, 320), "flat", "flat", "flat", 1),                 # dW in parts
]


@pytest.mark.parametrize("types", ["f32", "bf16"])
@pytest.mark.parametrize("shape,logits,x,w,sums", TILES)
def test_tiles(shape, logits, x, w, sums, types):
    dt = sbn.SBN_F32 if types == "f32" else sbn.SBN_BF16
    want = {f"ce_logits_{logits}": 1, f"ce_dlogits_{logits}": 1, f"ce_dx_{x}": 1, f"ce_dw_{w}": 1}
    if sums:
        want["ce_sum"] = sums
    assert check(*shape, dxdt=dt, dwdt=dt) == want


def test_all_tile_shapes_are_here():
    tiles = ("wide", "square", "flat")
    for i in (1, 2, 3):
        assert {t[i] for t in TILES} == set(tiles)


@pytest.mark.parametrize("T,V,K,x,x_sums,w,w_sums", [
    (65400, 9500, 64, "square", 0, "square", 3),                   # dX's sums go through float32 tile by tile
    (65400, 9500, 192, "wide", 0, "wide", 3),
    (4100, 140001, 64, "square", 3, "square", 0),                  # and by the sum of its parts
])
def test_three_pieces(T, V, K, x, x_sums, w, w_sums):
    """The middle piece of dX adds to the sums of the first where they lie."""
    assert sbn.sbn_cross_entropy_workspace_bytes(T, V, K, True) < T * V * 2 * 2
    ran = check(T, V, K)
    assert sum(n for k, n in ran.items() if k.startswith("ce_dlogits")) == 3
    assert ran[f"ce_dx_{x}"] == 3 and ran[f"ce_dw_{w}"] == 3 and ran.get("ce_sum", 0) == x_sums + w_sums


def test_fine_gradients_in_three_pieces():
    """SBN_F32_FINE: two products a piece, added."""
    two = sbn.SBN_F32_FINE
    ran = check(65400, 4700, 64, dxdt=two, dwdt=two)
    assert sum(n for k, n in ran.items() if k.startswith("ce_dlogits")) == 3
    assert sum(n for k, n in ran.items() if k.startswith("ce_dx")) == 6
    assert sum(n for k, n in ran.items() if k.startswith("ce_dw")) == 6
