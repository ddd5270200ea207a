"""Log probabilities of so many tokens that their statistics are formed in parts: rows on both sides
of a part's border and the last ones against 64 bits, all ids against calls of fewer tokens."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_head_tiles import launches
from test_gpu_logprobs import check_forward, problem, reference

pytestmark = pytest.mark.gpu


# sets of 8 logits: 512 MiB of pairs; statistics alone: 4 GiB
@pytest.mark.parametrize("T,V,K,top,part", [(9001, 65536, 1024, 64, 4608), (800001, 65536, 64, 0, 400128)])
def test_parts(T, V, K, top, part):
    import torch
    X, W, y, _, _ = problem(T, V, K, 3)
    for tokens in (y, y.int()):
        got, ran = launches(lambda: sbn.sbn_token_logprobs(X, W, tokens, scale=0.75, top=top))
        assert sum(n for k, n in ran.items() if k.startswith("logprob_logits")) == 2 and ran["logprob_join"] == 2
        for rows in (slice(0, 20), slice(part - 20, part + 20), slice(T - 20, T)):
            out = [None if t is None else t[rows] for t in got]
            check_forward(out, reference(X[rows], W, y[rows], 0.75), y[rows], top)
    few = [sbn.sbn_token_logprobs(X[t: t + 3000], W, y[t: t + 3000], scale=0.75, top=top) for t in range(0, min(T, 60000), 3000)]
    n = sum(f[0].shape[0] for f in few)
    for i in (0, 1, 2):                              # other tiles, perhaps: equal to float32's rounding
        a, b = got[i][:n], torch.cat([f[i] for f in few])
        assert (a - b).abs().max() <= 2.0 ** -14
    if top:
        assert torch.equal(got[3][:n], torch.cat([f[3] for f in few]))


def test_parts_captured():
    """In a graph, replayed: no part reads what another left."""
    import torch
    from test_gpu_graphs import replay_matches
    T, V, K, top = 9001, 65536, 1024, 64
    X, W, y, _, _ = problem(T, V, K, 4)
    out = dict(zip(("logp", "entropy", "lse"), (torch.empty(T, device="cuda") for _ in range(3))))
    ids, tlp = torch.empty((T, top), dtype=torch.int64, device="cuda"), torch.empty((T, top), device="cuda")
    replay_matches(lambda: sbn.sbn_token_logprobs(X, W, y, top=top, top_ids=ids, top_logp=tlp, **out), [*out.values(), ids, tlp])
