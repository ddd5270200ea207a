"""The example's step through log probabilities: without a bonus the loss's gradients, with one those of
the formula in 64 bits.  D is rounded to bf16 in both (2^-9 of each entry on average, which sums
keep: 2^-9 of a gradient's norm, and half as much again for dX's own rounding), what a wrong
sign or factor would be is of the gradient's own size: 2^-6 of the norm is told from either."""
from __future__ import annotations

import pytest

from test_gpu_block import example

pytestmark = pytest.mark.gpu


def step(m, keep, entropy):
    import torch
    model = m.Model(32, 0, keep, entropy)
    tokens = torch.arange(m.T, device="cuda") % m.V
    targets = (tokens * 7 + 3) % m.V
    y = model.forward(tokens)[0]
    loss = model.train_step(tokens, targets, 0.0)
    return y, model.head, targets, loss, [g.clone() for _, gs in model.tables for g in gs]


@pytest.mark.parametrize("keep", [16, 8])
def test_without_a_bonus(keep):
    m = example()
    *_, a, loss = step(m, keep, 0.0)
    *_, b, policy = step(m, keep, 1e-30)
    assert abs(float(a) - float(b)) <= 1e-5 * abs(float(a))
    for p, q in zip(loss, policy):
        assert (p - q).norm() <= 2.0 ** -6 * p.norm()


@pytest.mark.parametrize("C", [0.1, 3.0])
def test_with_a_bonus(C):
    """The head's gradient of mean(-log p - C H)."""
    import torch
    m = example()
    y, head, targets, _, grads = step(m, 8, C)
    T = y.shape[0]
    lp = torch.log_softmax(y.double() @ head.double().t().contiguous(), 1)
    p, H = lp.exp(), -(lp.exp() * lp).sum(1, keepdim=True)
    D = p.scatter_add(1, targets[:, None], torch.full((T, 1), -1.0, dtype=torch.float64, device="cuda")) + C * p * (lp + H)
    want = (D / T).t().contiguous() @ y.double()
    assert (grads[1].double() - want).norm() <= 2.0 ** -6 * want.norm()
    if C > 1:                                        # the bonus has a part in it that the bound would miss
        bonus = (C * p * (lp + H) / T).t().contiguous() @ y.double()
        assert bonus.norm() > 2.0 ** -3 * want.norm()
