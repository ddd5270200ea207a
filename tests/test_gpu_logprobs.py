"""Log probabilities, entropies, top alternatives and their gradients against 64-bit torch.

Bounds, with u = 2^-24 and b = 2^-8, each a worst case (l: scaled logits):
  l        products of bf16 are exact in float32, K of them are summed, one factor: scale K u A,
           A[t,v] = sum_k |x w|
  lse      as test_gpu_cross_entropy.py, with two more roundings of an exponent for the scale:
           its largest logit error + 6 u (1 + max|l| + |lse|) + (sqrt(V) + 64) u
  logp     that and the token's logit: twice it
  entropy  sum_v p (|log p| + |H| + 1) (a logit's error + 6 u (1 + |l| + |lse|)), from the
           derivative -p (log p + H) and the products of p and exponents, and the sums'
           (sqrt(V) + 128) u (1 + sum p |log p|)
  top      ids: those of 64-bit sums; values: lse's and 2 u of their own
  D        with s = sum of the errors of l, of lse and 6 u (1 + |l| + |lse|):
           p s (|dlogp| + |dH| (|log p| + |H| + 1)) + p |dH| (entropy's) + 8 u p (|dlogp| + |dH|
           (|log p| + |H|)) + b |D| + 2 u |dlogp|; in two bf16 numbers, as up to 128 tokens, 2^-16 for b
  dX       scale (sum_v D's |w| + (V + 16) u sum_v |D w|), + b |dX| for bf16; dW the same over t
"""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_cross_entropy import B, U, close, make
from test_gpu_graphs import replay_matches
from test_gpu_head_tiles import launches

pytestmark = pytest.mark.gpu


def problem(T, V, K, seed, **kw):
    """X, W, tokens, dlogp, dentropy; some rows without a token, some without any gradient."""
    import torch
    X, W, y, d = make(T, V, K, seed, **kw)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    dl = torch.randn(T, generator=g, device="cuda")
    dh = 0.3 * torch.randn(T, generator=g, device="cuda")
    if T > 4:
        dl[3] = dh[3] = 0.0
        dh[1] = 0.0
    return X, W, y, dl, dh


def logits(X, W, scale):
    Xd, Wd = X.double(), W.double()
    return Xd @ Wd.t().contiguous() * scale, Xd.abs() @ Wd.abs().t().contiguous() * scale


def reference(X, W, y, scale=1.0, dl=None, dh=None, fine=False):
    import torch
    z, A = logits(X, W, scale)
    T, V, K = X.shape[0], W.shape[0], X.shape[1]
    lse = torch.logsumexp(z, 1)
    el = K * U * A
    rl = 6 * U * (1 + z.abs() + lse.abs()[:, None])
    blse = el.amax(1) + rl.amax(1) + (V ** 0.5 + 64) * U
    kept = (y >= 0) & (y < V)
    at = torch.where(kept, y, 0)[:, None]
    logp = torch.where(kept, z.gather(1, at)[:, 0] - lse, 0.0)
    lp = z - lse[:, None]
    p = lp.exp()
    plp = p * lp
    H = -plp.sum(1)
    bH = (p * (lp.abs() + H.abs()[:, None] + 1) * (el + rl)).sum(1) + (V ** 0.5 + 128) * U * (1 + plp.abs().sum(1))
    r = dict(z=z, lse=lse, blse=blse, logp=logp, H=H, bH=bH)
    if dl is None:
        return r
    gl = torch.where(kept, dl.double(), 0.0)[:, None]
    gh = dh.double()[:, None]
    one = torch.zeros_like(p).scatter_(1, at, kept.double()[:, None])
    D = gl * (one - p) - gh * p * (lp + H[:, None])
    s = el + blse[:, None] + rl
    sizes = lp.abs() + H.abs()[:, None]
    bD = (p * s * (gl.abs() + gh.abs() * (sizes + 1)) + p * gh.abs() * bH[:, None] + 8 * U * p * (gl.abs() + gh.abs() * sizes)
          + (2.0 ** -16 if fine else B) * D.abs() + 2 * U * gl.abs())
    Xd, Wd = X.double(), W.double()
    r.update(D=D, dX=scale * (D @ Wd), dW=scale * (D.t().contiguous() @ Xd),
             bX=scale * (bD @ Wd.abs() + (V + 16) * U * (D.abs() @ Wd.abs())),
             bW=scale * (bD.t().contiguous() @ Xd.abs() + (T + 16) * U * (D.abs().t().contiguous() @ Xd.abs())))
    return r


def check_forward(got, r, y, top):
    import torch
    logp, H, lse, ids, tlp = got
    close(lse, r["lse"], r["blse"], "lse")
    if y is not None:
        close(logp, r["logp"], 2 * r["blse"], "logp")
        assert (logp[(y < 0)] == 0).all()
    else:
        assert logp is None
    close(H, r["H"], r["bH"], "entropy")
    if top:
        v, order = torch.sort(r["z"], dim=1, descending=True, stable=True)
        assert ids.dtype == torch.int64 and torch.equal(ids, order[:, :top]), "ids"
        ref = v[:, :top] - r["lse"][:, None]
        close(tlp, ref, r["blse"][:, None] + 2 * U * ref.abs(), "top_logp")
    else:
        assert ids is None and tlp is None


SHAPES = [(1, 1, 64), (1, 1000, 64), (2, 63, 128), (17, 64, 64), (64, 65, 192), (65, 129, 64), (130, 257, 320),
          (1, 513, 2560), (33, 1999, 128), (257, 300, 64), (300, 2500, 256), (1021, 777, 192), (64, 9001, 64),
          (2100, 4700, 64), (4100, 4097, 128), (3, 30011, 64), (128, 1500, 192), (129, 1500, 192)]


@pytest.mark.parametrize("T,V,K", SHAPES)
def test_forward_and_gradients(T, V, K):
    import torch
    scale = (1.0, 0.75, 1.3)[(T + V) % 3]
    X, W, y, dl, dh = problem(T, V, K, 1000 * T + V, ignored=0.2 if T > 1 else 0.0)
    r = reference(X, W, y, scale, dl, dh, fine=T <= 128)
    for top in sorted({0, 1, min(V, 7), min(V, 64)}):
        check_forward(sbn.sbn_token_logprobs(X, W, y, scale=scale, top=top), r, y, top)
    logp, H, lse, _, _ = a = sbn.sbn_token_logprobs(X, W, y, scale=scale)
    b = sbn.sbn_token_logprobs(X, W, y.int(), scale=scale)
    assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3]))
    check_forward(sbn.sbn_token_logprobs(X, W, scale=scale, top=min(V, 5)), r, None, min(V, 5))
    f = sbn.SBN_F32
    dX, dW = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, scale=scale)
    close(dX, r["dX"], r["bX"] + B * r["dX"].abs(), "dX bf16")
    close(dW, r["dW"], r["bW"] + B * r["dW"].abs(), "dW bf16")
    dX4, dW4 = sbn.sbn_token_logprobs_backward(X, W, y.int(), lse, H, dl, dh, scale=scale, dxdt=f, dwdt=f)
    close(dX4, r["dX"], r["bX"], "dX f32")
    close(dW4, r["dW"], r["bW"], "dW f32")
    assert torch.equal(dX4.bfloat16(), dX) and torch.equal(dW4.bfloat16(), dW)
    if T > 4:
        assert (dX[3] == 0).all()
    x2, w0 = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, scale=scale, need_dW=False)
    x0, w2 = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, scale=scale, need_dX=False)
    assert w0 is None and x0 is None and torch.equal(x2, dX) and torch.equal(w2, dW)


@pytest.mark.parametrize("T,V,K", [(300, 2500, 256), (1100, 900, 64)])
def test_fine_gradients(T, V, K):
    two = sbn.SBN_F32_FINE
    X, W, y, dl, dh = problem(T, V, K, 5)
    r = reference(X, W, y, 1.3, dl, dh, fine=True)
    _, H, lse, _, _ = sbn.sbn_token_logprobs(X, W, y, scale=1.3)
    dX, dW = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, scale=1.3, dxdt=two, dwdt=two)
    close(dX, r["dX"], r["bX"], "dX")
    close(dW, r["dW"], r["bW"], "dW")
    x2, w2 = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, scale=1.3, dxdt=two)      # one of them alone
    x3, w3 = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, scale=1.3, dwdt=two)
    assert (x2 == dX).all() and (w3 == dW).all()
    one = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, scale=1.3)
    assert (x3 == one[0]).all() and (w2 == one[1]).all()


def test_one_gradient_alone():
    """dlogp or dentropy None is zeros; a loss's gradient is that of the log probability, turned round."""
    import torch
    T, V, K = 70, 900, 128
    X, W, y, dl, dh = problem(T, V, K, 6)
    _, H, lse, _, _ = sbn.sbn_token_logprobs(X, W, y)
    f, zero = sbn.SBN_F32, torch.zeros_like(dl)
    kw = dict(dxdt=f, dwdt=f)
    both = lambda *a: sbn.sbn_token_logprobs_backward(X, W, *a, **kw)  # noqa: E731
    for p, q in ((both(y, lse, None, dl), both(y, lse, H, dl, zero)), (both(y, lse, H, None, dh), both(y, lse, H, zero, dh)),
                 (both(None, lse, H, None, dh), both(y, lse, H, None, dh))):
        assert all(torch.equal(s, t) for s, t in zip(p, q))
    dX, dW = both(y, lse, H, None, None)
    assert (dX == 0).all() and (dW == 0).all()
    r = reference(X, W, y, 1.0, -dl, zero)
    ce = sbn.sbn_cross_entropy_backward(X, W, y, lse, dl, dxdt=f, dwdt=f)
    close(ce[0], r["dX"], r["bX"], "dX")
    close(ce[1], r["dW"], r["bW"], "dW")


def test_rows_without_a_gradient_give_nothing():
    """What lse, entropy and (without a token) dlogp hold there does not matter."""
    import torch
    T, V, K = 40, 500, 64
    X, W, y, dl, dh = problem(T, V, K, 7)
    _, H, lse, _, _ = sbn.sbn_token_logprobs(X, W, y)
    ref = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, torch.where(y < 0, 0.0, dh))
    nan = torch.tensor(float("nan"), device="cuda")
    bad = [torch.where(y < 0, nan, t) for t in (lse, H, dl)]
    got = sbn.sbn_token_logprobs_backward(X, W, y, *bad, torch.where(y < 0, 0.0, dh))
    assert all(torch.equal(s, t) for s, t in zip(ref, got)) and (got[0][y < 0] == 0).all()


@pytest.mark.parametrize("T,V,K", [(50, 333, 128), (300, 1111, 64)])
def test_strides_and_given_outputs(T, V, K):
    import torch
    X, W, y, dl, dh = problem(T, V, K, 8, ldx=K + 24, ldw=K + 8)
    r = reference(X, W, y, 1.0, dl, dh)
    out = [torch.empty(T, device="cuda") for _ in range(3)]
    ids, tlp = torch.empty((T, 9), dtype=torch.int64, device="cuda"), torch.empty((T, 9), device="cuda")
    got = sbn.sbn_token_logprobs(X, W, y, top=9, logp=out[0], entropy=out[1], lse=out[2], top_ids=ids, top_logp=tlp)
    assert all(a is b for a, b in zip(got, (*out, ids, tlp)))
    check_forward(got, r, y, 9)
    bx = torch.full((T, K + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    bw = torch.full((V, K + 40), 5.0, dtype=torch.float32, device="cuda")
    sbn.sbn_token_logprobs_backward(X, W, y, out[2], out[1], dl, dh, dwdt=sbn.SBN_F32, dX=bx[:, :K], dW=bw[:, :K])
    close(bx[:, :K], r["dX"], r["bX"] + B * r["dX"].abs(), "dX")
    close(bw[:, :K], r["dW"], r["bW"], "dW")
    assert (bx[:, K:] == 3.0).all() and (bw[:, K:] == 5.0).all(), "columns past the rows"


@pytest.mark.parametrize("T,V,K", [(70, 300, 64), (300, 2500, 256), (65400, 9500, 64)])
def test_gradients_in_place_of_inputs(T, V, K):
    import torch
    X, W, y, dl, dh = problem(T, V, K, 19, ldx=K + 8, ldw=K + 16)
    _, H, lse, _, _ = sbn.sbn_token_logprobs(X, W, y)
    dX, dW = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh)
    W2 = torch.empty((V, K + 16), dtype=torch.bfloat16, device="cuda")[:, :K]
    W2.copy_(W)
    a, b = sbn.sbn_token_logprobs_backward(X, W2, y, lse, H, dl, dh, dW=W2)
    assert b is W2 and torch.equal(a, dX) and torch.equal(W2, dW)
    a, _ = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, dX=X, need_dW=False)
    assert a is X and torch.equal(X, dX)


def test_tokens_out_of_range():
    import torch
    T, V, K = 70, 200, 64
    X, W, _, dl, dh = problem(T, V, K, 9)
    for bad in (-100, -1, V, V + 7, 2 ** 40, -2 ** 40):
        y = torch.full((T,), bad, device="cuda")
        logp, H, lse, _, _ = sbn.sbn_token_logprobs(X, W, y)
        assert (logp == 0).all() and torch.isfinite(lse).all() and (H > 0).all()
        dX, dW = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl)
        assert (dX == 0).all() and (dW == 0).all()


def test_sharp_and_flat_distributions():
    """Logits of several hundred, where all but one probability vanish, and equal ones, at both ends of scale."""
    import torch
    T, V, K = 40, 1000, 64
    X, W, y, dl, dh = problem(T, V, K, 11, scale=8.0, ignored=0.0)
    for scale in (1.0, 2.0 ** 6, 2.0 ** -20):
        r = reference(X, W, y, scale, dl, dh)
        got = sbn.sbn_token_logprobs(X, W, y, scale=scale, top=4)
        check_forward(got, r, y, 4)
        assert (got[1] >= -1e-6).all()
        dX, dW = sbn.sbn_token_logprobs_backward(X, W, y, got[2], got[1], dl, dh, scale=scale)
        close(dX, r["dX"], r["bX"] + B * r["dX"].abs(), "dX")
        close(dW, r["dW"], r["bW"] + B * r["dW"].abs(), "dW")
    X, W, y, _, _ = problem(5, 1, 64, 12, ignored=0.0)
    check_forward(sbn.sbn_token_logprobs(X, W, y, top=1), reference(X, W, y), y, 1)


def test_equal_logits_go_by_index():
    import torch
    T, V, K = 6, 5000, 128
    X, W, y, _, _ = problem(T, V, K, 13)
    W = W.contiguous()
    W[17] = W[4000] = W[4001] = W[4002] = W[18] = W[2222] * 3        # likely near the top or the bottom of each row
    W[4100:4140] = 0.0
    X[2] = 0.0                                                      # a padded row: all equal
    X[3] = -X[1]
    r = reference(X, W, y)
    for top in (1, 3, 20, 64):
        check_forward(sbn.sbn_token_logprobs(X, W, y, top=top), r, y, top)
    for fill in (0.0, 0.5, -0.25):                                  # every logit of a row equal
        Wf = torch.full((V, K), fill, dtype=torch.bfloat16, device="cuda")
        _, H, _, ids, tlp = sbn.sbn_token_logprobs(X.abs(), Wf, y, top=64)
        assert torch.equal(ids, torch.arange(64, device="cuda").expand(T, 64))
        assert (H - torch.tensor(float(V), device="cuda").log()).abs().max() < 1e-4
    X2, W2, y2, _, _ = problem(2, 20000, 64, 14)                    # as many as no queue holds
    W2[:] = W2[:1].clone()
    assert torch.equal(sbn.sbn_token_logprobs(X2, W2, y2, top=30)[3], torch.arange(30, device="cuda").expand(2, 30))


@pytest.mark.parametrize("T,V", [(5, 3000), (400, 3000)])
def test_logits_that_32_bits_cannot_tell_apart(T, V):
    """Large parts that cancel or are equal, and a small one that decides."""
    import torch
    K = 256
    X, W, y, _, _ = problem(T, V, K, 15, ignored=0.0)
    X, W = X.contiguous(), W.contiguous()
    W[:, :128] = W[:1, :128].clone() * 64                           # the same for all entries
    W[:, 128:] *= 2.0 ** -12
    check_forward(sbn.sbn_token_logprobs(X, W, y, top=12), reference(X, W, y), y, 12)
    X[:, 64:128] = X[:, :64]
    W[:, 64:128] = -W[:, :64]                                       # and now their sum is 0
    check_forward(sbn.sbn_token_logprobs(X, W, y, top=12), reference(X, W, y), y, 12)


def test_ascending_and_descending_rows():
    """Entries in order of their logits, and the largest all in one lane's places."""
    import torch
    T, V, K = 3, 4096, 64
    X = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    X[:, 0], X[:, 1] = 1.0, 2.0 ** -7
    W = torch.zeros((V, K), dtype=torch.bfloat16, device="cuda")
    v = torch.arange(V, device="cuda")
    W[:, 0], W[:, 1] = (v // 128).bfloat16(), (v % 128).bfloat16()  # logits v / 128, exactly
    y = torch.zeros(T, dtype=torch.int64, device="cuda")
    assert torch.equal(sbn.sbn_token_logprobs(X, W, y, top=64)[3], (V - 1 - torch.arange(64, device="cuda")).expand(T, 64))
    assert torch.equal(sbn.sbn_token_logprobs(-X, W, y, top=64)[3], torch.arange(64, device="cuda").expand(T, 64))
    W.zero_()
    best = [o + 16 * i + e for o in (128, 2048) for i in range(8) for e in range(4)]
    W[best, 0] = torch.arange(1, len(best) + 1, device="cuda").bfloat16()
    want = torch.tensor(best[::-1], device="cuda")
    assert torch.equal(sbn.sbn_token_logprobs(X, W, y, top=64)[3], want.expand(T, 64))


def rows(T, top):
    """The launches after the logits'."""
    return {"logprob_rows": 1} if T <= 256 else {"logprob_join": 1, "logprob_top": 1} if top else {"logprob_join": 1}


# tokens, entries, K: the tiles of the logits and of D
@pytest.mark.parametrize("shape,tile", [((8100, 7000, 4096), "wide"), ((1285, 3664, 3136), "square"), ((65, 17007, 2112), "square"),
                                        ((16, 1796, 2112), "slim"), ((40, 32700, 320), "slim"), ((5000, 300, 320), "slim"),
                                        ((16, 33000, 2112), "flat"), ((5500, 300, 320), "flat")])
def test_tiles(shape, tile):
    T, V, K = shape
    X, W, y, dl, dh = problem(T, V, K, T + V + K)
    r = reference(X, W, y, 1.0, dl, dh)
    got, ran = launches(lambda: sbn.sbn_token_logprobs(X, W, y, top=10))
    check_forward(got, r, y, 10)
    assert ran == {f"logprob_logits_{tile}": 1, **rows(T, True)}
    plain, ran = launches(lambda: sbn.sbn_token_logprobs(X, W, y))
    assert ran == {f"logprob_logits_{tile}": 1, **rows(T, False)}
    assert all(bool((p == q).all()) for p, q in zip(got[:3], plain[:3]))
    (dX, dW), ran = launches(lambda: sbn.sbn_token_logprobs_backward(X, W, y, got[2], got[1], dl, dh))
    assert ran[f"logprob_dlogits_{tile}"] == 1
    for g, ref, bound, what in ((dX, r["dX"], r["bX"], "dX"), (dW, r["dW"], r["bW"], "dW")):
        close(g, ref, bound + B * ref.abs(), what)
        assert (g.double() - ref).norm() <= 2.0 ** -7 * ref.norm(), what


@pytest.mark.parametrize("T,V,dxdt,pieces", [(4096, 70001, sbn.SBN_F32, 2), (4096, 70001, sbn.SBN_F32_FINE, 3),
                                             (100, 1100003, sbn.SBN_F32, 2)])
def test_several_pieces_of_the_vocabulary(T, V, dxdt, pieces):
    import torch
    K = 64
    X, W, y, dl, dh = problem(T, V, K, 7)
    r = reference(X, W, y, 0.75, dl, dh, fine=T <= 128)
    logp, H, lse, _, _ = sbn.sbn_token_logprobs(X, W, y, scale=0.75)
    f = dict(scale=0.75, dxdt=dxdt)
    (dX, dW), ran = launches(lambda: sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, **f))
    assert sum(n for k, n in ran.items() if k.startswith("logprob_dlogits")) == pieces
    close(dX, r["dX"], r["bX"], "dX")
    close(dW, r["dW"], r["bW"] + B * r["dW"].abs(), "dW")
    again = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, **f)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dW)


def test_no_tokens():
    import torch
    X = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    W = torch.ones((100, 64), dtype=torch.bfloat16, device="cuda")
    y = torch.empty(0, dtype=torch.int64, device="cuda")
    logp, H, lse, ids, tlp = sbn.sbn_token_logprobs(X, W, y, top=3)
    assert logp.shape == H.shape == lse.shape == (0,) and ids.shape == tlp.shape == (0, 3)
    e = torch.empty(0, device="cuda")
    dX, dW = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, e, e, dwdt=sbn.SBN_F32)
    assert dX.shape == (0, 64) and (dW == 0).all()


def test_gradient_against_differences():
    """Along random directions, dX and dW (float32) against central differences of
    sum_t dlogp_t logp_t + dentropy_t H_t in 64 bits (step 1e-4: the third-order term is under
    1e-7 of the direction's size)."""
    import torch
    T, V, K, h, scale = 20, 150, 64, 1e-4, 1.3
    X, W, y, dl, dh = problem(T, V, K, 13)
    r = reference(X, W, y, scale, dl, dh)
    _, H, lse, _, _ = sbn.sbn_token_logprobs(X, W, y, scale=scale)
    f = sbn.SBN_F32
    dX, dW = sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, scale=scale, dxdt=f, dwdt=f)
    at = torch.where(y >= 0, y, 0)[:, None]
    gl = torch.where(y >= 0, dl.double(), 0.0)

    def L(x, w):
        lp = torch.log_softmax(scale * (x @ w.t().contiguous()), 1)
        return (lp.gather(1, at)[:, 0] * gl).sum() - ((lp.exp() * lp).sum(1) * dh.double()).sum()

    g = torch.Generator(device="cuda").manual_seed(3)
    for mine, bound, which in ((dX, r["bX"], 0), (dW, r["bW"], 1)):
        e = torch.randn(mine.shape, generator=g, device="cuda", dtype=torch.float64)
        x, w = X.double(), W.double()
        up, dn = (L(x + h * e, w), L(x - h * e, w)) if which == 0 else (L(x, w + h * e), L(x, w - h * e))
        num = (up - dn) / (2 * h)
        assert abs(float((mine.double() * e).sum() - num)) <= float((e.abs() * (bound + 1e-7)).sum()) + 1e-5


@pytest.mark.parametrize("T,V,K", [(300, 5000, 128), (20, 3001, 192), (1100, 2000, 64)])
def test_captured(T, V, K):
    import torch
    X, W, y, dl, dh = problem(T, V, K, 21)
    logp, H, lse, tlp = (torch.empty(n, device="cuda") for n in (T, T, T, (T, 6)))
    ids = torch.empty((T, 6), dtype=torch.int64, device="cuda")
    dX, dW = torch.empty((T, K), dtype=torch.bfloat16, device="cuda"), torch.empty((V, K), device="cuda")

    def step():
        sbn.sbn_token_logprobs(X, W, y, top=6, scale=1.25, logp=logp, entropy=H, lse=lse, top_ids=ids, top_logp=tlp)
        sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, scale=1.25, dwdt=sbn.SBN_F32, dX=dX, dW=dW)

    replay_matches(step, [logp, H, lse, ids, tlp, dX, dW])


def test_streams_at_once():
    import torch
    ins = [problem(256, 3000, 256, 30 + i) for i in range(2)]

    def work(X, W, y, dl, dh, **kw):
        logp, H, lse, ids, tlp = sbn.sbn_token_logprobs(X, W, y, top=4, **kw)
        return (logp, H, lse, ids, tlp, *sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh, **kw))

    ref = [work(*a) for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for given in (False, True, False):
        got = []
        for s, a in zip(streams, ins):
            if given:
                got.append(work(*a, stream=s))
            else:
                with torch.cuda.stream(s):
                    got.append(work(*a))
        torch.cuda.synchronize()
        for a, b in zip(ref, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_threads_at_once():
    """Two threads of calls, on streams of their own and both on one."""
    import threading

    import torch
    ins = [problem(200 + 70 * i, 3000, 128, 50 + i) for i in range(2)]

    def work(X, W, y, dl, dh):
        logp, H, lse, ids, tlp = sbn.sbn_token_logprobs(X, W, y, top=4)
        return (logp, H, lse, ids, tlp, *sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh))

    ref = [work(*a) for a in ins]
    torch.cuda.synchronize()
    one = torch.cuda.Stream()
    for streams in ([torch.cuda.Stream(), torch.cuda.Stream()], [one, one]):
        got = [[], []]

        def run(i):
            with torch.cuda.stream(streams[i]):
                got[i] += [work(*ins[i]) for _ in range(20)]

        threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        for a, r in zip(got, ref):
            assert len(a) == 20 and all(torch.equal(p, q) for out in a for p, q in zip(out, r))


@pytest.mark.parametrize("T,top", [(5, 3), (5, 64), (300, 3), (300, 20)])
def test_rows_that_are_not_finite_stay_alone(T, top):
    """Outside the contract: the call ends, its ids are of the vocabulary, and the other rows have their values."""
    import torch
    V, K = 2100, 64
    X, W, y, _, _ = problem(T, V, K, 60, ignored=0.0)
    ref = sbn.sbn_token_logprobs(X, W, y, top=top)
    bad = X.clone()
    bad[1, 5], bad[3, 7] = float("nan"), float("inf")
    got = sbn.sbn_token_logprobs(bad, W, y, top=top)
    rest = torch.tensor([t not in (1, 3) for t in range(T)], device="cuda")
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(got, ref))
    assert ((got[3] >= 0) & (got[3] < V)).all()
    assert got[0][1].isnan() and got[2][1].isnan()


def test_a_batch_of_a_large_vocabulary():
    """The alternatives' pairs past 2^31 bytes: the last rows as in a call of their own."""
    import torch
    T, V, K = 20000, 500009, 64
    X, W, y, _, _ = problem(T, V, K, 40)
    assert sbn.sbn_token_logprobs_workspace_bytes(T, V, K, 5) > 2 ** 31
    logp, H, lse, ids, tlp = sbn.sbn_token_logprobs(X, W, y, top=5)
    for rows in (slice(0, 30), slice(T - 30, T)):
        check_forward([t[rows] for t in (logp, H, lse, ids, tlp)], reference(X[rows], W, y[rows]), y[rows], 5)


def test_finite_check(monkeypatch):
    monkeypatch.setenv("SBN_CHECK_FINITE", "1")
    X, W, y, dl, dh = problem(8, 100, 64, 17)
    y[2] = -1
    dl[2] = float("nan")                                            # of a row without a token
    _, H, lse, _, _ = sbn.sbn_token_logprobs(X, W, y)
    sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, dh)
    bad = dh.clone()
    bad[2] = float("inf")
    W2 = W.clone()
    W2[50, 3] = float("nan")
    for f in (lambda: sbn.sbn_token_logprobs(X, W2, y), lambda: sbn.sbn_token_logprobs_backward(X, W, y, lse, H, dl, bad)):
        with pytest.raises(sbn.SbnError) as e:
            f()
        assert e.value.status == sbn.SBN_ERR_VALUE
