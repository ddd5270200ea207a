"""Binding of the calls declared in ``include/sbn_score.h``: log probabilities of
given tokens under the output head, with entropies and top alternatives, and their
gradients.

As in ``training.py``: layouts that the C ABI cannot see are checked here, outputs
and workspaces are allocated with PyTorch where the caller passed none, everything
else happens in the HIP kernels.  A call that is given a `stream` runs as inside
``torch.cuda.stream(stream)``.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

from . import _SIGNATURES, SBN_BF16, PKG_DIR, SbnError, _check, _req
from .training import (_addr, _given, _head_args, _head_grad_out, _ld, _matrix, _on, _raw_stream, _scratch, _so, _sz, _torch,
                       _vector)

SCORE_HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "sbn_score.h")
SBN_LOGPROBS_MAX_TOP = 64

_i64, _int, _vp, _f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float
_SIGNATURES.update({
    "sbn_token_logprobs_workspace_bytes": ([_i64, _i64, _i64, _int, ctypes.POINTER(_sz)], _int),
    "sbn_token_logprobs": ([_vp, _i64, _vp, _i64, _vp, _int, _i64, _i64, _i64, _f32, _vp, _vp, _vp, _int, _vp, _vp, _vp,
                            _sz, _vp], _int),
    "sbn_token_logprobs_backward_workspace_bytes": ([_i64, _i64, _i64, ctypes.POINTER(_sz)], _int),
    "sbn_token_logprobs_backward": ([_vp, _i64, _vp, _i64, _vp, _int, _f32, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp,
                                     _int, _i64, _vp, _int, _i64, _vp, _sz, _vp], _int),
})


def score_header_symbols() -> list[str]:
    """Names of the functions declared in include/sbn_score.h."""
    text = open(SCORE_HEADER_PATH).read()
    return sorted(set(re.findall(r"^\s*sbn_status\s+(sbn_\w+)\s*\(", text, re.M)))


def _scored_args(fn, X, W, tokens):
    """T, V, K and the bytes of a token; tokens may be None."""
    if tokens is not None:
        return _head_args(fn, X, W, tokens)
    for t, name in ((X, "X"), (W, "W")):
        _matrix(t, name, fn)
        _req(t, name, "bf16", False, fn)
    T, K = X.shape
    if W.shape[1] != K or W.device != X.device:
        raise SbnError(fn, 2, f"W {tuple(W.shape)} on {W.device} does not go with X {tuple(X.shape)} on {X.device}")
    return T, W.shape[0], K, 8


@functools.lru_cache(maxsize=1024)
def sbn_token_logprobs_workspace_bytes(T: int, V: int, K: int, top: int = 0, backward: bool = False) -> int:
    b = _sz()
    if backward:
        fn = "sbn_token_logprobs_backward_workspace_bytes"
        _check(fn, _so().sbn_token_logprobs_backward_workspace_bytes(T, V, K, ctypes.byref(b)))
    else:
        fn = "sbn_token_logprobs_workspace_bytes"
        _check(fn, _so().sbn_token_logprobs_workspace_bytes(T, V, K, top, ctypes.byref(b)))
    return b.value


def sbn_token_logprobs(X, W, tokens=None, *, scale: float = 1.0, top: int = 0, logp=None, entropy=None, lse=None,
                       top_ids=None, top_logp=None, ws=None, stream=None):
    """Log probabilities of `tokens` ([T] int64 or int32; outside [0, V): none,
    log probability 0) under the softmax of scale * X W^T, X [T, K] and W [V, K]
    bf16, with the entropy of each row's distribution and its `top` most likely
    entries, largest first, equal ones by index (in the order of 64-bit sums).
    Returns (logp, entropy, lse, top_ids, top_logp): float32 [T] three times,
    int64 and float32 [T, top]; logp is None without tokens, the last two with
    top = 0."""
    if stream is not None:
        return _on(stream, sbn_token_logprobs, locals())
    fn = "sbn_token_logprobs"
    torch = _torch()
    T, V, K, tb = _scored_args(fn, X, W, tokens)
    dev = X.device

    def vector(t, name):
        if t is None:
            return X.new_empty(T, dtype=torch.float32)
        _vector(t, name, T, torch.float32, dev, fn)
        return t

    if tokens is not None:
        logp = vector(logp, "logp")
    elif logp is not None:
        raise SbnError(fn, 2, "logp goes with tokens")
    entropy, lse = vector(entropy, "entropy"), vector(lse, "lse")
    nbytes = sbn_token_logprobs_workspace_bytes(T, V, K, top)          # refuses what top cannot be
    if top:
        for t, name, dt in ((top_ids, "top_ids", torch.int64), (top_logp, "top_logp", torch.float32)):
            if t is not None and (t.dtype is not dt or t.shape != (T, top) or t.device != dev or not t.is_contiguous()):
                raise SbnError(fn, 2, f"{name} must be {dt} {[T, top]} on {dev}, contiguous")
        if top_ids is None:
            top_ids = X.new_empty((T, top), dtype=torch.int64)
        if top_logp is None:
            top_logp = X.new_empty((T, top), dtype=torch.float32)
    elif top_ids is not None or top_logp is not None:
        raise SbnError(fn, 2, "top_ids and top_logp go with top > 0")
    if ws is not None:
        _given(ws, dev, fn)
    raw = _raw_stream(dev)
    if ws is None:
        ws = _scratch("token_logprobs", nbytes, dev, raw)
    _check(fn, _so().sbn_token_logprobs(X.data_ptr(), _ld(X), W.data_ptr(), _ld(W), _addr(tokens), tb, T, V, K, scale,
                                        _addr(logp), entropy.data_ptr(), lse.data_ptr(), top, _addr(top_ids),
                                        _addr(top_logp), ws.data_ptr(), ws.numel(), raw))
    return logp, entropy, lse, top_ids, top_logp


def sbn_token_logprobs_backward(X, W, tokens, lse, entropy, dlogp, dentropy=None, *, scale: float = 1.0,
                                dxdt: int = SBN_BF16, dwdt: int = SBN_BF16, dX=None, dW=None, need_dX: bool = True,
                                need_dW: bool = True, ws=None, stream=None):
    """Gradients of the hidden states and of the head's weights from the
    forward's lse and entropy and the gradients of each row's log probability
    and entropy ([T] float32, None for zeros; entropy may be None with
    dentropy, tokens with dlogp).  Types as for sbn_cross_entropy_backward.
    Returns (dX, dW), each None where it is not needed."""
    if stream is not None:
        return _on(stream, sbn_token_logprobs_backward, locals())
    fn = "sbn_token_logprobs_backward"
    torch = _torch()
    T, V, K, tb = _scored_args(fn, X, W, tokens)
    for t, name in ((lse, "lse"), (entropy, "entropy"), (dlogp, "dlogp"), (dentropy, "dentropy")):
        if t is not None:
            _vector(t, name, T, torch.float32, X.device, fn)
    if lse is None or (dentropy is not None and entropy is None) or (dlogp is not None and tokens is None):
        raise SbnError(fn, 1, "lse is needed, entropy with dentropy, tokens with dlogp")
    dX = _head_grad_out(dX, "dX", need_dX, dxdt, X, fn)
    dW = _head_grad_out(dW, "dW", need_dW, dwdt, W, fn)
    if ws is not None:
        _given(ws, X.device, fn)
    raw = _raw_stream(X.device)
    if ws is None:
        ws = _scratch("cross_entropy_backward", sbn_token_logprobs_workspace_bytes(T, V, K, 0, True), X.device, raw)
    _check(fn, _so().sbn_token_logprobs_backward(
        X.data_ptr(), _ld(X), W.data_ptr(), _ld(W), _addr(tokens), tb, scale, lse.data_ptr(), _addr(entropy),
        _addr(dlogp), _addr(dentropy), T, V, K, _addr(dX), dxdt, 0 if dX is None else _ld(dX), _addr(dW), dwdt,
        0 if dW is None else _ld(dW), ws.data_ptr(), ws.numel(), raw))
    return dX, dW
