"""Host threads that enqueue on one stream at once: each gets its own results."""
from __future__ import annotations

import threading

import pytest

import sparse_linear_layers_02_amd as sbn

pytestmark = pytest.mark.gpu


def test_two_threads_on_one_stream():
    import torch
    T, V, K = 130, 3000, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gain, d = torch.ones(K, device="cuda"), torch.ones(T, device="cuda")
    ins = [(r(T, K).bfloat16(), (r(V, K) * 0.05).bfloat16(), torch.randint(0, V, (T,), generator=g, device="cuda"))
           for _ in range(2)]

    def work(X, W, y):
        loss, lse = sbn.sbn_cross_entropy(X, W, y)
        Y, H, rs = sbn.sbn_rmsnorm(X, gain)
        return (loss, *sbn.sbn_cross_entropy_backward(X, W, y, lse, d), *sbn.sbn_rmsnorm_backward(Y, H, gain, rs))

    ref = [work(*a) for a in ins]
    torch.cuda.synchronize()
    got = [[], []]

    def run(i):
        for _ in range(100):
            got[i].append(work(*ins[i]))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, many in zip(ref, got):
        assert len(many) == 100
        for b in many:
            assert all(torch.equal(p, q) for p, q in zip(a, b))
