"""Trains a small Sparse-BitLinear language model on synthetic text, every step
through the library: embedding -> blocks of [RMS norm with the residual's addition
and 8-bit output -> sparse ternary layer -> squared ReLU -> sparse ternary layer]
-> RMS norm -> cross entropy of the head, the gradients of all of them, and one
AdamW step over all tensors, whose bf16 weights the next step's pack reads.

    python examples/train_lm.py [--steps N] [--bits 32|8] [--seed S]

The text repeats a random successor table, so the loss falls from log(vocabulary)
towards 0 if, and only if, the gradients are right.  Prints the loss and, at the
end, the scores of one token decoded at a time against the same tokens in a batch.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_linear_layers_02_amd as sbn  # noqa: E402

V, K, R, BLOCKS, T, N, M = 1000, 256, 512, 2, 1024, 2, 4


class Model:
    """bf16 weights, float32 gains, and the AdamW state of all of them."""

    def __init__(self, bits: int, seed: int):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g, device="cuda") / math.sqrt(s[-1])).bfloat16()  # noqa: E731
        self.emb, self.head = w(V, K) * 4, w(V, K)
        self.up, self.down = [w(R, K) for _ in range(BLOCKS)], [w(K, R) for _ in range(BLOCKS)]
        self.gains = [torch.ones(n, device="cuda") for n in [K] * (BLOCKS + 1) + [R] * BLOCKS]
        self.weights = [self.emb, self.head, *self.up, *self.down]
        self.tables = [self._table(self.weights, bits, 0.01), self._table(self.gains, 32, 0.0)]
        self.step = 0

    def _table(self, params, bits, decay):
        grads = [torch.zeros(p.shape, device="cuda") for p in params]
        m, v = ([torch.zeros(p.shape, device="cuda") for p in params] for _ in range(2))
        kw = {}
        if bits == 8:
            (m, kw["m_scales"]), (v, kw["v_scales"]) = (zip(*(enc(x) for x in s)) for enc, s in
                                                        ((sbn.sbn_adamw_encode_m, m), (sbn.sbn_adamw_encode_v, v)))
        return sbn.AdamWTable(params, grads, list(m), list(v), weight_decay=decay,
                              **{k: list(x) for k, x in kw.items()}), grads

    def _layer(self, W, Xq, s_x):
        packed = sbn.sbn_mask_ternarize_pack(W, N, M)
        gemm = sbn.sbn_sparse_ternary_gemv if Xq.shape[0] <= 16 else sbn.sbn_sparse_ternary_gemm
        return gemm(Xq, s_x, *packed, W.shape[0], N, M), packed

    def forward(self, tokens):
        """Hidden states before the head, and what the backward needs."""
        h, x, kept = self.emb[tokens], None, []
        for b in range(BLOCKS):
            Xq, s_x, h, rs = sbn.sbn_rmsnorm_quant(h if x is None else x, self.gains[b], residual=None if x is None else h)
            a, pa = self._layer(self.up[b], Xq, s_x)
            act = torch.relu(a).square()
            Aq, s_a, act, ra = sbn.sbn_rmsnorm_quant(act, self.gains[BLOCKS + 1 + b])
            x, pb = self._layer(self.down[b], Aq, s_a)
            kept.append((Xq, s_x, h, rs, a, pa, Aq, s_a, act, ra, pb))
        y, h, rs = sbn.sbn_rmsnorm(x, self.gains[BLOCKS], residual=h)
        return y, (kept, h, rs)

    def train_step(self, tokens, targets, lr):
        y, (kept, h, rs) = self.forward(tokens)
        loss, lse = sbn.sbn_cross_entropy(y, self.head, targets)
        (wt, gw), (gt, gg) = self.tables
        d = torch.full((y.shape[0],), 1.0 / y.shape[0], device="cuda")
        dy, _ = sbn.sbn_cross_entropy_backward(y, self.head, targets, lse, d, dwdt=sbn.SBN_F32, dW=gw[1])
        dh, _ = sbn.sbn_rmsnorm_backward(dy, h, self.gains[BLOCKS], rs, dgain=gg[BLOCKS])
        for b in reversed(range(BLOCKS)):
            Xq, s_x, h, rs, a, pa, Aq, s_a, act, ra, pb = kept[b]
            dact, _ = sbn.sbn_backward(dh, Aq, s_a, *pb, N, M, dxdt=sbn.SBN_BF16, dW=gw[2 + BLOCKS + b])
            dact, _ = sbn.sbn_rmsnorm_backward(dact, act, self.gains[BLOCKS + 1 + b], ra, dgain=gg[BLOCKS + 1 + b])
            da = dact * (2 * torch.relu(a))
            dx, _ = sbn.sbn_backward(da, Xq, s_x, *pa, N, M, dxdt=sbn.SBN_BF16, dW=gw[2 + b])
            # dh goes on along the residual stream beside what comes through the block
            dh, _ = sbn.sbn_rmsnorm_backward(dx, h, self.gains[b], rs, dH=dh, dX=dx, dgain=gg[b])
        gw[0].zero_().index_add_(0, tokens, dh.float())
        self.step += 1
        for t in (wt, gt):
            sbn.sbn_adamw_step(t, lr=lr, step=self.step, beta2=0.95)
        return loss.mean()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--bits", type=int, choices=(32, 8), default=32)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(a.seed)
    after = torch.randperm(V, generator=g, device="cuda")
    model, losses = Model(a.bits, a.seed), []
    for i in range(a.steps):
        tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
        losses.append(model.train_step(tokens, after[tokens], 3e-3))
        if i % 10 == 0 or i + 1 == a.steps:
            print(f"step {i:4d}  loss {losses[-1].item():.4f}", flush=True)
    tokens = torch.arange(8, device="cuda")
    score = lambda t: sbn.sbn_cross_entropy(model.forward(t)[0], model.head, after[t])[0]  # noqa: E731
    batch, single = score(tokens), torch.cat([score(tokens[i: i + 1]) for i in range(8)])
    print(f"scores of 8 tokens, one at a time against together: largest difference "
          f"{(batch - single).abs().max().item():.2e}")
    return [x.item() for x in losses], (batch, single)


if __name__ == "__main__":
    main()
