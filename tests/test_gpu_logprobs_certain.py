"""Distributions that are nearly certain: log probabilities and entropies next to 0 keep their
relative precision, and stay on their side of 0.

The logits here are exact in float32, so with u = 2^-24 a term of r = sum exp(l - m) is off by
its exponent (the difference is exact, log2 e times the scale and the product are rounded: 3 u gap),
the exponential's 2 u, and the sum's (sqrt(V) + 64) u as in test_gpu_logprobs.py; ln(1 + r) adds
4 u.  The entropy's terms x (gap) take 4 u more, and both of its parts are positive, so
  logp      (3 gap + sqrt(V) + 72) u relative,  entropy  (3 gap + sqrt(V) + 80) u relative,
gap the largest that counts: exp(-gap) of what lies further is below 2^-24 of the rest."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_cross_entropy import U

pytestmark = pytest.mark.gpu
K = 64


def head(T, V, kind, seed):
    """X of ones in two places, W whose logits are 256 + w: one of 40, the others 18 to 24 below, or all but one far below."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    X[:, 0] = X[:, 9] = 1.0
    W = torch.zeros((V, K), dtype=torch.bfloat16, device="cuda")
    at = V // 3
    W[:, 0] = 256.0
    if kind == "spread":
        W[:, 9] = 16.0 + torch.randint(0, 49, (V,), generator=g, device="cuda") / 8
    else:
        W[:, 9] = -160.0
        W[at + 1 if kind == "beside" else V - 2, 9] = 21.0
    W[at, 9] = 40.0
    return X, W, at


def near(got, ref, rel, what):
    err = (got.double() - ref).abs()
    assert (err <= rel * ref.abs()).all(), f"{what}: {float((err / ref.abs()).max()):.3g} of {rel:.3g}"


@pytest.mark.parametrize("kind", ["spread", "beside", "elsewhere"])
@pytest.mark.parametrize("T,V", [(3, 1000), (16, 33000), (200, 17007), (300, 9000), (2100, 9000)])
@pytest.mark.parametrize("scale", [1.0, 0.75])
def test_nearly_certain(T, V, kind, scale):
    import torch
    X, W, at = head(T, V, kind, V + T)
    y = torch.full((T,), at, device="cuda")
    y[1::2] = V - 2
    gaps = scale * (296.0 - (256.0 + W[:, 9].double()))
    terms = torch.exp(-gaps)
    terms[at] = 0.0
    ln = torch.log1p(terms.sum())
    want = torch.where(torch.arange(T, device="cuda") % 2 == 0, -ln, -gaps[V - 2] - ln)
    H = ln + (terms * gaps).sum() / (1 + terms.sum())
    rel = (3 * 24 * scale + V ** 0.5 + 72) * U
    for top in (0, 1, 5):
        logp, ent, lse, ids, tlp = sbn.sbn_token_logprobs(X, W, y, scale=scale, top=top)
        near(logp, want, rel, "logp")
        near(ent, H.expand(T), rel + 8 * U, "entropy")
        near(lse, (296.0 * scale + ln).expand(T), 2 * U, "lse")
        assert (logp < 0).all() and (ent > 0).all()
        if top:
            v, order = torch.sort(-gaps, descending=True, stable=True)
            assert torch.equal(ids, order[:top].expand(T, top)) and (tlp < 0).all()
            near(tlp, (v[:top] - ln).expand(T, top), rel, "top_logp")


def test_the_only_entry():
    """Nothing else to be: log probability and entropy are 0."""
    import torch
    for T in (4, 300):
        X = torch.randn(T, K, device="cuda").bfloat16() * 8
        W = torch.randn(1, K, device="cuda").bfloat16() * 8
        logp, H, _, ids, tlp = sbn.sbn_token_logprobs(X, W, torch.zeros(T, dtype=torch.int64, device="cuda"), top=1)
        assert (logp == 0).all() and (H == 0).all() and (ids == 0).all() and (tlp == 0).all()


@pytest.mark.parametrize("T", [40, 400])
def test_never_above_zero(T):
    """Random heads of sharp distributions: no log probability above 0, no entropy below."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    V = 3000
    X = (torch.randn(T, 256, generator=g, device="cuda") * 4).bfloat16()
    W = torch.randn(V, 256, generator=g, device="cuda").bfloat16()
    first = sbn.sbn_token_logprobs(X, W, top=1)[3][:, 0].contiguous()
    for scale in (0.5, 1.0, 64.0):
        logp, H, _, _, tlp = sbn.sbn_token_logprobs(X, W, first, scale=scale, top=9)
        assert (logp <= 0).all() and (H >= 0).all() and (tlp <= 0).all()


@pytest.mark.parametrize("T", [9, 300, 1100])
def test_a_certain_row_changes_no_other(T):
    """How a row's sums are formed goes by that row alone."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    V = 9000
    X = torch.randn(T, 256, generator=g, device="cuda").bfloat16()
    W = (torch.randn(V, 256, generator=g, device="cuda") * 0.05).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    a = sbn.sbn_token_logprobs(X, W, y, top=5)
    X[3::7] *= 64                                    # nearly certain
    b = sbn.sbn_token_logprobs(X, W, y, top=5)
    rest = torch.arange(T, device="cuda") % 7 != 3
    assert all(torch.equal(p[rest], q[rest]) for p, q in zip(a, b))
