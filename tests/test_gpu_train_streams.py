"""Calls that are given a stream: what they allocate belongs to that stream.  Memory
that the current stream has just freed is its allocator's next choice there, and its
earlier work may still be using it when the other stream writes."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn

pytestmark = pytest.mark.gpu
T, V, K = 512, 1000, 1024                                          # outputs of at least 2 KB, so a size has its own blocks


def calls():
    """name -> (a call that takes `stream`, the tensors it returns)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    X, gain, W = r(T, K).bfloat16(), torch.ones(K, device="cuda"), (r(V, K) * 0.05).bfloat16()
    y, d = torch.randint(0, V, (T,), generator=g, device="cuda"), torch.ones(T, device="cuda")
    _, H, rstd = sbn.sbn_rmsnorm(X, gain, residual=X)
    _, lse = sbn.sbn_cross_entropy(X, W, y)
    c, s = sbn.sbn_adamw_encode_m(r(T * K))
    x = r(T * K)
    return {
        "rmsnorm": lambda **kw: sbn.sbn_rmsnorm(X, gain, residual=X, **kw),
        "rmsnorm_quant": lambda **kw: sbn.sbn_rmsnorm_quant(X, gain, residual=X, **kw),
        "rmsnorm_backward": lambda **kw: sbn.sbn_rmsnorm_backward(X, H, gain, rstd, **kw),
        "cross_entropy": lambda **kw: sbn.sbn_cross_entropy(X, W, y, **kw),
        "cross_entropy_backward": lambda **kw: sbn.sbn_cross_entropy_backward(X, W, y, lse, d, **kw),
        "encode": lambda **kw: sbn.sbn_adamw_encode_v(x.abs(), **kw),
        "decode": lambda **kw: (sbn.sbn_adamw_decode_m(c, s, **kw),),
    }


NAMES = ["rmsnorm", "rmsnorm_quant", "rmsnorm_backward", "cross_entropy", "cross_entropy_backward", "encode", "decode"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_belong_to_the_given_stream(name):
    import torch
    f = calls()[name]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ref = f()
    sizes = [t.untyped_storage().nbytes() for t in ref]
    torch.cuda.synchronize()
    freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    own = {t.untyped_storage().data_ptr() for t in freed}
    del freed                                                      # cached for the current stream
    out = f(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    taken = [t.untyped_storage().data_ptr() for t in out if t.untyped_storage().data_ptr() in own]
    assert not taken, "memory of the current stream"


def test_step_on_a_given_stream():
    import torch
    p, g = torch.ones(5000, device="cuda"), torch.ones(5000, device="cuda")
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    t = sbn.AdamWTable([p], [g], [m], [v])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert sbn.sbn_adamw_step(t, lr=0.5, step=1, eps=1e-8, stream=s) is None
    s.synchronize()
    assert torch.allclose(p, torch.full_like(p, 0.5))
