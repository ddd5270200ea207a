"""Top alternatives among rows of W of very different sizes: one whose large parts cancel has
a float32 sum that is off by far more than the other rows' are, and is found all the same.  The
ids are those of 64-bit sums; the values' bounds are test_gpu_logprobs.py's."""
from __future__ import annotations

import pytest

import sparse_linear_layers_02_amd as sbn
from test_gpu_head_tiles import launches
from test_gpu_logprobs import check_forward, problem, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 5, 300])
@pytest.mark.parametrize("top", [1, 3, 20, 64])
def test_a_row_whose_large_parts_cancel(T, top):
    """Its logit is 1, its float32 sum whatever 2^24 + 1 - 2^24 gives; 125 others have 0.5, the rest -1."""
    import torch
    V, K = 5000, 64
    X = torch.ones((T, K), dtype=torch.bfloat16, device="cuda")
    W = torch.zeros((V, K), dtype=torch.bfloat16, device="cuda")
    W[:, 0] = -1.0
    W[7::40, 0] = 0.5                                # each in a set of its own
    at = 3333
    W[at, 0], W[at, 1], W[at, 63] = 2.0 ** 24, 1.0, -2.0 ** 24
    ids, tlp = sbn.sbn_token_logprobs(X, W, top=top)[3:]
    want = torch.cat([torch.tensor([at], device="cuda"), torch.arange(7, V, 40, device="cuda")])[:top]
    assert torch.equal(ids, want.expand(T, top))
    assert ((tlp[:, :1] - tlp).double() - (torch.arange(top, device="cuda") > 0) * 0.5).abs().max() <= 2.0 ** -20


# tokens, entries, K, alternatives, the logits' tiles; sets of 32, 16 and 8 sums
@pytest.mark.parametrize("T,V,K,top,tile", [(3, 30011, 64, 7, "slim"), (16, 1796, 2112, 30, "slim"), (16, 33000, 2112, 5, "flat"),
                                            (65, 17007, 2112, 12, "square"), (300, 2500, 256, 33, "slim"),
                                            (2100, 9000, 1024, 5, "wide"), (2100, 9000, 1024, 40, "wide")])
def test_rows_of_many_sizes(T, V, K, top, tile):
    """Every fifth row has two large parts that cancel, 2^0 to 2^14 times its others, among rows 2^-6 to 2^2 times as large."""
    import torch
    X, W, y, _, _ = problem(T, V, K, T + V + top)
    X, W = X.contiguous(), W.contiguous()
    g = torch.Generator(device="cuda").manual_seed(V)
    W *= (2.0 ** torch.randint(-6, 3, (V, 1), generator=g, device="cuda")).bfloat16()
    X[:, K // 2] = X[:, 3] = X[:, 3].abs() + 0.5
    n = len(range(0, V, 5))
    big = (2.0 ** torch.randint(0, 15, (n,), generator=g, device="cuda") * (1 + torch.rand(n, generator=g, device="cuda"))).bfloat16()
    W[::5, 3], W[::5, K // 2] = big, -big
    got, ran = launches(lambda: sbn.sbn_token_logprobs(X, W, y, top=top))
    assert ran[f"logprob_logits_{tile}"] == 1
    z = reference(X, W, y)["z"]
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(got[3], order)
    check_forward(got, reference(X, W, y), y, top)


def test_one_row_far_larger_than_all_others():
    """Whether it is among the alternatives or not, the others keep their places."""
    import torch
    for T, V in ((5, 4000), (400, 4000)):
        X, W, y, _, _ = problem(T, V, 128, 9)
        W = W.contiguous()
        W[1234] *= 2.0 ** 12
        check_forward(sbn.sbn_token_logprobs(X, W, y, top=10), reference(X, W, y), y, 10)
        W[:, 5] = 0.0
        W[1234] = 0.0
        W[1234, 5] = 3e38                            # squares past float32
        X = X.contiguous()
        X[:, 5] = 0.0
        X[0, 5] = 2.0 ** -120
        r = reference(X, W, y)
        ids = sbn.sbn_token_logprobs(X, W, y, top=10)[3]
        assert torch.equal(ids, torch.sort(r["z"], dim=1, descending=True, stable=True).indices[:, :10])


@pytest.mark.parametrize("V", [257, 260, 300, 511, 513])
def test_vocabularies_that_leave_most_of_a_tile_empty(V):
    """Whole tiles of 256 entries: sets of which all or a part is past the vocabulary are among the candidates."""
    import torch
    T, K = 70000, 64
    X, W, y, _, _ = problem(T, V, K, V)
    z = reference(X, W, y)["z"]
    got, ran = launches(lambda: sbn.sbn_token_logprobs(X, W, y, top=64))
    assert ran["logprob_logits_wide"] == 1
    assert torch.equal(got[3], torch.sort(z, dim=1, descending=True, stable=True).indices[:, :64])
