"""Cases of operators beside the sparse layer: log probabilities of given tokens
with the distribution's entropy and its top alternatives, and their gradients;
the function between a feed-forward block's products with the next layer's int8
activations as its output, and its gradient; and the norm, both kept for the
backward pass as 8-bit checkpoints.  Each in its plain form (elementary torch
operations, 32 bits; 64 where logits are told apart) and through the library's calls.

`own` chooses the side: False computes the plain forms, True calls the library.
"""
from __future__ import annotations

import math

import torch
import torch.nn.functional as F

own = False

EPS = 1e-6                      # added to the mean square of a row
TINY = 2.0 ** -100              # least maximum of a row or block that is told from zero
BLOCK = 128                     # neighbours of a row that share a scale in an 8-bit checkpoint


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the next token of one sequence, with what else it could have been: latency
        {"name": "score_token", "op": "score", "T": 1, "V": 50001, "K": 2560, "top": 8, "scale": 1.0},
        # a drafted continuation checked in one call, at a sampling temperature, many alternatives
        {"name": "score_draft", "op": "score", "T": 37, "V": 32001, "K": 4096, "top": 20, "scale": 1.25},
        # log probabilities and entropies of whole batches under a reference policy
        {"name": "score_batch", "op": "score", "T": 4096, "V": 65536, "K": 2560, "top": 0, "scale": 1.0},
        # the same with alternatives, kept to train another model on
        {"name": "score_batch_top", "op": "score", "T": 4096, "V": 65536, "K": 2560, "top": 8, "scale": 1.0},
        # a policy's training step on a short odd batch and an odd vocabulary, entropy rewarded
        {"name": "policy_odd", "op": "policy", "T": 1021, "V": 32001, "K": 2560, "scale": 1.0},
        # a full training step of a policy
        {"name": "policy_train", "op": "policy", "T": 8192, "V": 65536, "K": 4096, "scale": 1.0},
        # one token between the products of a feed-forward block while text is generated: latency, nothing kept
        {"name": "ffn_token", "op": "ffn", "T": 1, "R": 6912, "dt": "bf16", "act": "relu2", "gated": True, "norm": True,
         "keep": False},
        # the same place in a training step, both factors kept in 8 bits
        {"name": "ffn_train", "op": "ffn", "T": 8192, "R": 11008, "dt": "bf16", "act": "relu2", "gated": True,
         "norm": True, "keep": True},
        # its gradient from what was kept
        {"name": "ffn_grad_train", "op": "ffn_grad", "T": 8192, "R": 11008, "dt": "bf16", "act": "relu2", "gated": True,
         "norm": True},
        # a short odd batch of another block: sigmoid gate, no norm, 32-bit gradients
        {"name": "ffn_grad_odd_f32", "op": "ffn_grad", "T": 333, "R": 6920, "dt": "f32", "act": "silu", "gated": True,
         "norm": False},
        # the norm in front of a layer in a training step: codes for the product, the residual stream kept in 8 bits
        {"name": "norm_keep_train", "op": "norm", "T": 8192, "K": 4096, "dt": "bf16", "residual": True},
        # its gradient from what was kept, the gradient of the residual stream added
        {"name": "norm_kept_grad_train", "op": "norm_grad", "T": 8192, "K": 4096, "dt": "bf16", "residual": True},
    ]


def _between(rng, least, most):
    """A whole number, spread evenly over the logarithm."""
    return min(most, max(least, int(round(math.exp(rng.uniform(math.log(least), math.log(most)))))))


def draw(rng):
    op = rng.choice(["score", "score", "policy", "policy", "ffn", "ffn_grad", "norm", "norm_grad"])
    if op in ("score", "policy"):
        case = {"op": op, "T": _between(rng, 1, 4096), "V": _between(rng, 1000, 65536), "K": 64 * _between(rng, 4, 64),
                "scale": rng.choice([1.0, 0.5, 1.25])}
        if op == "score":
            case["top"] = rng.choice([0, 1, 5, 20, 32])
        return case
    if op in ("ffn", "ffn_grad"):
        case = {"op": op, "T": _between(rng, 1, 8192), "R": 8 * _between(rng, 32, 1376), "dt": rng.choice(["bf16", "f32"]),
                "act": rng.choice(["relu2", "silu"]), "gated": rng.random() < 0.7, "norm": rng.random() < 0.6}
        if op == "ffn":
            case["keep"] = rng.random() < 0.6
        return case
    return {"op": op, "T": _between(rng, 1, 8192), "K": 8 * _between(rng, 32, 512), "dt": rng.choice(["bf16", "f32"]),
            "residual": rng.random() < 0.7}


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


def work(case):
    op = case["op"]
    if op in ("score", "policy"):
        T, V, K = case["T"], case["V"], case["K"]
        read = 2.0 * K * (T + V) + 8 * T
        if op == "score":
            return {"bytes": read + 12 * T + 12.0 * T * case["top"], "flops": 2.0 * T * V * K}
        # logits, then both gradients; the logits are not kept, so their product is needed twice
        return {"bytes": 2 * read + 2.0 * K * (T + V) + 28 * T, "flops": 8.0 * T * V * K}
    T, e = case["T"], _BYTES[case["dt"]]
    kept = 1 + 4.0 / BLOCK                                   # a code, and its part of the scale
    if op in ("ffn", "ffn_grad"):
        n, two = T * case["R"], 2 if case["gated"] else 1
        gain = 4 * case["R"] if case["norm"] else 0
        if op == "ffn":   # inputs -> codes, and the values of the codes; what is kept, and its values
            return {"bytes": n * (e * two + 1 + 2 + (two * (kept + 2) if case["keep"] else 0)) + 4 * T + gain,
                    "flops": 10.0 * n * two}
        return {"bytes": n * (e + two * (kept + e)) + 2 * gain, "flops": 20.0 * n}
    K, r = case["K"], 1 if case["residual"] else 0
    if op == "norm":
        return {"bytes": T * K * (e * (1 + 2 * r) + 1 + 2 + kept + 2) + 4 * T + 4 * K, "flops": 12.0 * T * K}
    return {"bytes": T * K * (e * (2.0 + r) + kept) + 8 * K, "flops": 16.0 * T * K}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(g, T, K):
    """Activations: normal, a hundredth of the channels twenty times larger."""
    x = _randn(g, T, K)
    hot = torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]
    x[:, hot] *= 20.0
    return x


def _inputs(case, seed):
    """What both sides and exact() compute from."""
    g = _gen(seed)
    op = case["op"]
    if op in ("score", "policy"):
        T, V, K = case["T"], case["V"], case["K"]
        W = (_randn(g, V, K) * 0.02).to(torch.bfloat16)
        tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
        sure = 6.0 * torch.rand(T, 1, generator=g, device="cuda") / (0.02 * 0.02 * K)      # the token's logit raised by 0 to 6
        X = (_randn(g, T, K) + sure * W[tokens].float()).to(torch.bfloat16)
        s = {"X": X, "W": W, "tokens": tokens}
        if op == "policy":      # advantages; prompts and padding have no token and no entropy bonus
            keep = torch.rand(T, generator=g, device="cuda") >= 0.1
            s["tokens"] = torch.where(keep, tokens, -100)
            s["dlogp"] = torch.where(keep, _randn(g, T) / T, 0.0)
            s["dentropy"] = torch.where(keep, -0.05 / T, 0.0)
        return s
    T, dt = case["T"], _DT[case["dt"]]
    if op in ("ffn", "ffn_grad"):
        R = case["R"]
        s = {"A": _rows(g, T, R).to(dt), "B": _randn(g, T, R).to(dt) if case["gated"] else None,
             "gain": 1.0 + 0.1 * _randn(g, R) if case["norm"] else None}
        if op == "ffn_grad":    # from the 8-bit values of A and B
            s["dY"] = (_randn(g, T, R) * 1e-2).to(dt)
            s["kA"] = _to8(s.pop("A").float())
            s["kB"] = _to8(s.pop("B").float()) if case["gated"] else None
        return s
    K = case["K"]
    s = {"gain": 1.0 + 0.1 * _randn(g, K)}
    x = _rows(g, T, K)
    if op == "norm_grad":
        s["kH"] = _to8(x)
        s["dY"] = (_randn(g, T, K) * 1e-2).to(dt)
        s["dH"] = (_randn(g, T, K) * 1e-2).to(dt) if case["residual"] else None
    else:
        s["X"] = x.to(dt)
        s["res"] = (_randn(g, T, K) * 2.0).to(dt) if case["residual"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    return s


# ------------------------------------------------------------------ 8-bit checkpoints
# a code q in -127..127 stands for q s, s = a / 127, a the largest magnitude of the row's block of 128
def _blocks(x):
    T, K = x.shape
    return F.pad(x, (0, -K % BLOCK)).view(T, -1, BLOCK)


def _to8(x):
    """(codes [T, K], scales [T, blocks]) of float32 rows."""
    b = _blocks(x)
    a = b.abs().amax(2)
    a = torch.where(a < TINY, 0.0, a)
    q = torch.where(a[..., None] > 0, torch.round((127.0 * b) / a[..., None]), 0.0)
    return q.to(torch.int8).view(x.shape[0], -1)[:, : x.shape[1]].contiguous(), a / 127.0


def _of8(codes, scales):
    return (_blocks(codes.float()) * scales[..., None]).view(codes.shape[0], -1)[:, : codes.shape[1]]


# ------------------------------------------------------------------ plain forms
def _plain_head(s):
    case = s["case"]
    X, W, y = s["X"].float(), s["W"].float(), s["tokens"]
    logits = (X @ W.t()) * case["scale"]
    top = logits.amax(1, keepdim=True)
    kept = (y >= 0) & (y < case["V"])
    at = torch.where(kept, y, 0)[:, None]
    chosen = logits.gather(1, at)
    e = torch.exp(logits - top)
    z = e.sum(1, keepdim=True)
    lse = top + torch.log(z)
    p = e / z
    del e
    entropy = (lse - (p * logits).sum(1, keepdim=True))
    out = {"logp": torch.where(kept, (chosen - lse)[:, 0], 0.0), "entropy": entropy[:, 0]}
    if case["op"] == "score":
        out["lse"] = lse[:, 0]
        if case["top"]:
            # logits too near each other for 32 bits are told apart in 64; ties go to the lowest index
            k = case["top"]
            near = torch.topk(logits, min(k + 8, case["V"]), dim=1).indices.sort(dim=1).values
            exact = (s["W"][near].float() * X[:, None, :]).sum(2, dtype=torch.float64) * case["scale"]
            value, order = torch.sort(exact, dim=1, descending=True, stable=True)
            out["top_ids"] = near.gather(1, order)[:, :k].contiguous()
            out["top_logp"] = (value[:, :k] - lse).float()
        return out
    d = -p * (logits - lse + entropy)
    d = d * s["dentropy"][:, None]
    d -= p * torch.where(kept, s["dlogp"], 0.0)[:, None]
    d.scatter_add_(1, at, torch.where(kept, s["dlogp"], 0.0)[:, None])
    d *= case["scale"]
    out["dX"], out["dW"] = (d @ W).to(torch.bfloat16), (d.t() @ X).to(torch.bfloat16)
    return out


def _act(a, kind):
    """f(a) and f'(a)."""
    if kind == "relu2":
        r = torch.relu(a)
        return r * r, 2.0 * r
    g = 1.0 / (1.0 + torch.exp(-a))
    return a * g, g * (1.0 + a * (1.0 - g))


def _codes(v, rstd):
    """The values of a row's int8 codes times rstd, in 16 bits."""
    a = v.abs().amax(1, keepdim=True).clamp(min=TINY)
    return (torch.round((127.0 * v) / a) * ((a * rstd) / 127.0)).to(torch.bfloat16)


def _plain_ffn(s):
    case = s["case"]
    u = _act(s["A"].float(), case["act"])[0]
    if case["gated"]:
        u = u * s["B"].float()
    if case["norm"]:
        rstd = torch.rsqrt((u * u).mean(1, keepdim=True) + EPS)
        out = {"values": _codes(u * s["gain"], rstd)}
    else:
        out = {"values": _codes(u, 1.0)}
    if case["keep"]:
        out["A"] = _of8(*_to8(s["A"].float())).to(torch.bfloat16)
        if case["gated"]:
            out["B"] = _of8(*_to8(s["B"].float())).to(torch.bfloat16)
    return out


def _plain_norm_back(h, dy, gain):
    """Gradients of h and gain of y = h rstd gain."""
    w = dy * gain
    rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    n = h * rstd
    return (w - n * (w * n).mean(1, keepdim=True)) * rstd, (dy * n).sum(0)


def _plain_ffn_grad(s):
    case = s["case"]
    dy = s["dY"].float()
    f, df = _act(_of8(*s["kA"]), case["act"])
    b = _of8(*s["kB"]) if case["gated"] else None
    out = {}
    if case["norm"]:
        dy, out["dgain"] = _plain_norm_back(f * b if case["gated"] else f, dy, s["gain"])
    if case["gated"]:
        out["dA"], out["dB"] = (dy * b * df).to(s["dY"].dtype), (dy * f).to(s["dY"].dtype)
    else:
        out["dA"] = (dy * df).to(s["dY"].dtype)
    return out


def _plain_norm(s):
    dt = _DT[s["case"]["dt"]]
    H = s["X"] if s["res"] is None else (s["X"].float() + s["res"].float()).to(dt)
    h = H.float()
    rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    return {"H": H, "values": _codes(h * s["gain"], rstd), "kept": _of8(*_to8(h)).to(torch.bfloat16)}


def _plain_norm_grad(s):
    dx, dgain = _plain_norm_back(_of8(*s["kH"]), s["dY"].float(), s["gain"])
    if s["dH"] is not None:
        dx = dx + s["dH"].float()
    return {"dX": dx.to(s["dY"].dtype), "dgain": dgain}


# ------------------------------------------------------------------ the library's calls
def _times(Xq, s_x):
    """The values of int8 codes with a scale per token, in 16 bits."""
    return torch.mul(Xq, s_x[:, None], out=torch.empty(Xq.shape, dtype=torch.bfloat16, device=Xq.device))


def _own(s):
    import sparse_linear_layers_02_amd as sbn
    case = s["case"]
    op = case["op"]
    if op in ("score", "policy"):
        logp, entropy, lse, ids, top = sbn.sbn_token_logprobs(s["X"], s["W"], s["tokens"], scale=case["scale"],
                                                              top=case.get("top", 0))
        out = {"logp": logp, "entropy": entropy}
        if op == "score":
            out["lse"] = lse
            if case["top"]:
                out["top_ids"], out["top_logp"] = ids, top
            return out
        out["dX"], out["dW"] = sbn.sbn_token_logprobs_backward(s["X"], s["W"], s["tokens"], lse, entropy, s["dlogp"],
                                                               s["dentropy"], scale=case["scale"])
        return out
    if op == "norm":
        Xq, s_x, H, kept = sbn.sbn_rmsnorm_quant_keep(s["X"], s["gain"], residual=s["res"], eps=EPS)
        return {"H": H, "values": _times(Xq, s_x), "kept": sbn.sbn_keep8_decode(kept, dt=sbn.SBN_BF16)}
    if op == "norm_grad":
        dX, dgain = sbn.sbn_rmsnorm_backward_kept(s["dY"], sbn.Kept8(*s["kH"]), s["gain"], dH=s["dH"], eps=EPS)
        return {"dX": dX, "dgain": dgain}
    act = sbn.SBN_RELU2 if case["act"] == "relu2" else sbn.SBN_SILU
    if op == "ffn":
        Xq, s_x, kA, kB = sbn.sbn_activation_quant(s["A"], s["B"], act=act, gain=s["gain"], eps=EPS, keep=case["keep"])
        out = {"values": _times(Xq, s_x)}
        if case["keep"]:
            out["A"] = sbn.sbn_keep8_decode(kA, dt=sbn.SBN_BF16)
            if case["gated"]:
                out["B"] = sbn.sbn_keep8_decode(kB, dt=sbn.SBN_BF16)
        return out
    kB = sbn.Kept8(*s["kB"]) if case["gated"] else None
    dA, dB, dgain = sbn.sbn_activation_backward(s["dY"], sbn.Kept8(*s["kA"]), kB, act=act, gain=s["gain"], eps=EPS)
    out = {"dgain": dgain} if case["norm"] else {}
    out["dA"] = dA
    if case["gated"]:
        out["dB"] = dB
    return out


_PLAIN = {"score": _plain_head, "policy": _plain_head, "ffn": _plain_ffn, "ffn_grad": _plain_ffn_grad, "norm": _plain_norm,
          "norm_grad": _plain_norm_grad}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("score", "policy"):
        return _exact_head(case, s)
    gain = s["gain"].double() if s.get("gain") is not None else None
    if op == "norm":
        h = s["X"].double()
        if s["res"] is not None:
            h = (h + s["res"].double()).to(_DT[case["dt"]]).double()          # the stored stream is what is normalised
        rstd = (h.pow(2).sum(1) / case["K"] + EPS).pow(-0.5)
        return {"H": h, "values": _exact_round(h * gain * rstd[:, None]), "kept": _exact_kept(h)}
    if op == "norm_grad":
        dx, dgain = _exact_norm_back(_exact_of(*s["kH"]), s["dY"].double(), gain)
        return {"dX": dx if s["dH"] is None else dx + s["dH"].double(), "dgain": dgain}
    if op == "ffn":
        a, b = s["A"].double(), s["B"].double() if case["gated"] else 1.0
        u = (a.clamp(min=0).pow(2) if case["act"] == "relu2" else a * torch.sigmoid(a)) * b
        if case["norm"]:
            u = u * gain * (u.pow(2).sum(1, keepdim=True) / case["R"] + EPS).pow(-0.5)
        out = {"values": _exact_round(u)}
        if case["keep"]:
            out["A"] = _exact_kept(a)
            if case["gated"]:
                out["B"] = _exact_kept(b)
        return out
    a, b = _exact_of(*s["kA"]), _exact_of(*s["kB"]) if case["gated"] else torch.ones((), dtype=torch.float64, device="cuda")
    if case["act"] == "relu2":
        f, slope = a.clamp(min=0).pow(2), 2 * a.clamp(min=0)
    else:
        g = torch.sigmoid(a)
        f, slope = a * g, g + a * g * torch.sigmoid(-a)
    du, out = s["dY"].double(), {}
    if case["norm"]:
        du, out["dgain"] = _exact_norm_back(f * b, du, gain)
    out["dA"] = du * b * slope
    if case["gated"]:
        out["dB"] = du * f
    return out


def _exact_head(case, s):
    X, W, y = s["X"].double(), s["W"].double(), s["tokens"]
    z = X.matmul(W.t().contiguous())
    z *= case["scale"]
    lse = z.logsumexp(1)
    rows = ((y >= 0) & (y < case["V"])).nonzero()[:, 0]
    logp = torch.zeros_like(lse)
    logp[rows] = z[rows, y[rows]] - lse[rows]
    z -= lse[:, None]
    p = z.exp()
    entropy = -(p * z).sum(1)
    out = {"logp": logp, "entropy": entropy}
    if case["op"] == "score":
        out["lse"] = lse
        if case["top"]:
            best = z.topk(case["top"], dim=1)
            out["top_ids"], out["top_logp"] = best.indices, best.values
        return out
    z += entropy[:, None]
    z *= -s["dentropy"].double()[:, None]
    given = torch.zeros_like(lse)
    given[rows] = s["dlogp"].double()[rows]
    z -= given[:, None]
    z *= p
    z[rows, y[rows]] += given[rows]
    z *= case["scale"]
    out["dX"], out["dW"] = z.matmul(W), z.t().contiguous().matmul(X)
    return out


def _exact_round(y):
    """Rows rounded to 127 steps up to their largest magnitude."""
    step = y.abs().max(1).values[:, None] / 127.0
    return torch.where(step > 0, (y / step).round() * step, 0.0)


def _exact_kept(x):
    T, K = x.shape
    return _exact_round(F.pad(x, (0, -K % BLOCK)).reshape(-1, BLOCK)).reshape(T, -1)[:, :K]


def _exact_of(codes, scales):
    return codes.double() * scales.double().repeat_interleave(BLOCK, dim=1)[:, : codes.shape[1]]


def _exact_norm_back(h, dy, gain):
    # with y = gain h r, r = (mean h^2 + eps)^-1/2: dL/dh = r w - h r^3 <w, h> / K, w = gain dy
    K = h.shape[1]
    r = (h.pow(2).sum(1, keepdim=True) / K + EPS).pow(-0.5)
    w = gain * dy
    return r * w - h * r.pow(3) * ((w * h).sum(1, keepdim=True) / K), torch.einsum("tk,tk->k", dy, h * r)
