"""8-bit AdamW states at the ends of their range: a second moment above 0 keeps a code
in any block that has a scale, and where a block's second moments are too small for a
scale, its first moments cannot be divided by nothing."""
from __future__ import annotations

import numpy as np
import pytest

import sparse_linear_layers_02_amd as sbn
from gpu_util import dev, host

pytestmark = pytest.mark.gpu
F = np.float32


@pytest.mark.parametrize("n", [8, 256, 261, 1000])
def test_small_second_moments_beside_large_ones(n):
    """v down to the smallest float beside 2^10: v / s underflows, the code stays at least 1."""
    v = np.zeros(n, F)
    small = [2.0 ** -149, 2.0 ** -140, 2.0 ** -127, 2.0 ** -126, 2.0 ** -100, 1e-20, 0.0]
    v[: len(small)] = small
    v[-len(small):] = small if n > 8 else v[-len(small):]
    v[7] = 2.0 ** 10
    v[256::256] = 2.0 ** 10                                        # every block's largest
    c, s = sbn.sbn_adamw_encode_v(dev(v))
    c, s = host(c), np.repeat(host(s), 256)[:n]
    live = s > 0
    assert (s[:7] == 2.0 ** 10).all() and c[7] == 255
    assert np.array_equal(c[live] > 0, v[live] > 0)
    assert (c[live & (v > 0) & (v < 1e-7)] == 1).all()
    assert (host(sbn.sbn_adamw_decode_v(dev(c), dev(host(sbn.sbn_adamw_encode_v(dev(v))[1]))))[live & (v > 0)] > 0).all()


def states(n):
    import torch
    z = lambda dt, k: torch.zeros(k, dtype=dt, device="cuda")  # noqa: E731
    b = -(-n // 256)
    return z(torch.int8, n), z(torch.uint8, n), z(torch.float32, b), z(torch.float32, b)


@pytest.mark.parametrize("eps", [1e-8, 1e-20, 1e-37])
@pytest.mark.parametrize("size", [1e-16, 1e-18])                  # (of 1e-22 the square itself is no float32)
def test_tiny_gradients_then_none(size, eps):
    """|m / sqrt(v)| of Adam is at most 1 / sqrt((1-b2)/(1-b1)^2) of its terms, 0.45 here, and bias
    corrections of the first steps give under 2: no step moves a parameter by more than 2 lr."""
    import torch
    n, lr = 700, 0.125
    p = torch.zeros(n, device="cuda")
    g = torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * size
    g[::3] = 0
    m, v, sm, sv = states(n)
    t = sbn.AdamWTable([p], [g], [m], [v], m_scales=[sm], v_scales=[sv])
    for step in range(1, 6):
        before = p.clone()
        sbn.sbn_adamw_step(t, lr=lr, step=step, beta1=0.9, beta2=0.95, eps=eps)
        assert torch.isfinite(p).all() and ((p - before).abs() <= 2 * lr).all(), step
        if step == 2:
            g.zero_()


def test_states_encoded_apart():
    """First moments with a scale beside second moments without one, as encoding them apart can give."""
    import torch
    n = 300
    m, sm = sbn.sbn_adamw_encode_m(torch.full((n,), 1e-20, device="cuda"))
    v, sv = sbn.sbn_adamw_encode_v(torch.full((n,), 1e-40, device="cuda"))
    assert (sm > 0).all() and not sv.any()
    p, g = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    sbn.sbn_adamw_step(sbn.AdamWTable([p], [g], [m], [v], m_scales=[sm], v_scales=[sv]), lr=0.5, step=9, eps=1e-30)
    assert (p == 1).all() and not sm.any() and not m.any()
