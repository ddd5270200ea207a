"""Binding of the calls declared in ``include/sbn_train.h``: the RMS norm with
the layer's 8-bit activations as its output, the cross entropy of the output
head, and AdamW over many tensors.

As in the package's own module: layouts that the C ABI cannot see are checked
here, outputs and workspaces are allocated with PyTorch where the caller passed
none, everything else happens in the HIP kernels.  A call that is given a
`stream` runs as inside ``torch.cuda.stream(stream)``: outputs and workspaces
that it allocates are that stream's.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import sys

from . import _SIGNATURES, _WS, SBN_BF16, SBN_F32, SBN_F32_FINE, PKG_DIR, SbnError, _check, _req, lib

TRAIN_HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "sbn_train.h")
SBN_ADAMW_BLOCK = 256

_i64, _int, _sz, _vp, _f32, _f64 = (ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float,
                                    ctypes.c_double)
_SIGNATURES.update({
    "sbn_rmsnorm": ([_vp, _i64, _vp, _i64, _int, _vp, _int, _i64, _i64, _f32, _vp, _i64, _vp, _i64, _vp, _vp], _int),
    "sbn_rmsnorm_quant": ([_vp, _i64, _vp, _i64, _int, _vp, _int, _i64, _i64, _f32, _vp, _i64, _vp, _vp, _vp, _vp],
                          _int),
    "sbn_rmsnorm_backward_workspace_bytes": ([_i64, _i64, ctypes.POINTER(_sz)], _int),
    "sbn_rmsnorm_backward": ([_vp, _i64, _vp, _i64, _vp, _i64, _int, _vp, _int, _vp, _i64, _i64, _vp, _i64, _vp, _vp,
                              _sz, _vp], _int),
    "sbn_cross_entropy_workspace_bytes": ([_i64, _i64, _i64, ctypes.POINTER(_sz)], _int),
    "sbn_cross_entropy": ([_vp, _i64, _vp, _i64, _vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _sz, _vp], _int),
    "sbn_cross_entropy_backward_workspace_bytes": ([_i64, _i64, _i64, ctypes.POINTER(_sz)], _int),
    "sbn_cross_entropy_backward": ([_vp, _i64, _vp, _i64, _vp, _int, _vp, _vp, _i64, _i64, _i64, _vp, _int, _i64, _vp,
                                    _int, _i64, _vp, _sz, _vp], _int),
    "sbn_adamw_plan": ([_vp, _i64, _int, _int, _int, _vp, ctypes.POINTER(_i64)], _int),
    "sbn_adamw_step": ([_vp, _vp, _i64, _int, _int, _int, _f64, _f64, _f64, _f64, _i64, _vp, _vp], _int),
    "sbn_adamw_decode_state": ([_vp, _vp, _i64, _int, _vp, _vp], _int),
    "sbn_adamw_encode_state": ([_vp, _i64, _int, _vp, _vp, _vp], _int),
})


def train_header_symbols() -> list[str]:
    """Names of the functions declared in include/sbn_train.h."""
    text = open(TRAIN_HEADER_PATH).read()
    return sorted(set(re.findall(r"^\s*sbn_status\s+(sbn_\w+)\s*\(", text, re.M)))


# Small calls are bound by what happens here before the launch, so the checks
# below cost one expression where all is well, and say what is wrong elsewhere;
# torch and the library are looked up without an import statement or a lock.
_package = sys.modules[__package__]
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _so():
    return _package._lib or lib()


_FLOATS = {}


def _dtype(t, name: str, fn: str) -> int:
    dt = _FLOATS.get(t.dtype)
    if dt is None:
        torch = _torch()
        _FLOATS.update({torch.bfloat16: SBN_BF16, torch.float32: SBN_F32})
        dt = _FLOATS.get(t.dtype)
        if dt is None:
            raise SbnError(fn, 6, f"{name} must be bfloat16 or float32, got {t.dtype}")
    return dt


def _rows(t, name: str, like, fn: str):
    """`t` is a row-major tensor of `like`'s shape, type and device."""
    if t.dtype is like.dtype and t.shape == like.shape and t.device == like.device and t.stride(1) == 1:
        return
    if t.dtype != like.dtype:
        raise SbnError(fn, 6, f"{name} must be {like.dtype}, got {t.dtype}")
    if t.shape != like.shape or t.device != like.device:
        raise SbnError(fn, 2, f"{name} must be {tuple(like.shape)} on {like.device}, "
                              f"got {tuple(t.shape)} on {t.device}")
    _matrix(t, name, fn)


def _vector(t, name: str, n: int, dtype, device, fn: str):
    """`t` is a contiguous vector of n `dtype` on `device`."""
    if t.dtype is dtype and t.shape == (n,) and t.stride(0) == 1 and t.device == device:
        return
    if t.dtype != dtype:
        raise SbnError(fn, 6, f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != n or t.device != device:
        raise SbnError(fn, 2, f"{name} must be [{n}] on {device}, got {tuple(t.shape)} on {t.device}")
    if n > 1 and t.stride(0) != 1:
        raise SbnError(fn, 2, f"{name} must be contiguous")


def _ld(t) -> int:
    """Row stride; of a single row, which has none that matters, its length."""
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 7) // 8 * 8


def _matrix(t, name: str, fn: str):
    if t.dim() != 2:
        raise SbnError(fn, 2, f"{name} must have two dimensions, got {t.dim()}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise SbnError(fn, 2, f"{name} must have unit column stride (row-major)")


def _addr(t):
    return None if t is None else t.data_ptr()


def _on(stream, call, args):
    """`call` with `args` (its parameters by name) while `stream` is current: what it
    allocates then belongs to that stream, whose earlier work alone has to be done."""
    args["stream"] = None
    with _torch().cuda.stream(stream):
        return call(**args)


def _raw_stream(device) -> int:
    """The HIP stream to launch on: the current one of the tensors' device."""
    if device.index is None:
        raise SbnError("stream", 2, f"the tensors must be on a GPU, not on {device}")
    c = _torch()._C
    if c._cuda_getDevice() != device.index:
        raise SbnError("stream", 2, f"the tensors are on {device}, which is not the current device")
    return c._cuda_getCurrentRawStream(device.index)   # torch.cuda.current_stream() without its Stream object


def _scratch(kind: str, nbytes: int, device, raw: int):
    """The package's grow-only workspace of (kind, device, the device's current stream)
    of the calling thread; under capture one of its own, which belongs to the graph."""
    torch = _torch()
    if raw and torch._C._cuda_isCurrentStreamCapturing():   # the null stream cannot be captured
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    key = (kind, device, raw)
    buf = _WS.kept.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = _WS.kept[key] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    return buf


def _given(ws, device, fn: str):
    """A workspace of the caller's has no gaps and is on the tensors' device."""
    if ws.device != device or not ws.is_contiguous():
        raise SbnError(fn, 2, f"ws must be contiguous on {device}, got {ws.device}")


# ------------------------------------------------------------------ RMS norm
def _norm_args(fn, X, gain, residual, H, rstd):
    torch = _torch()
    _matrix(X, "X", fn)
    dt = _dtype(X, "X", fn)
    gdt = _dtype(gain, "gain", fn)
    T, K = X.shape
    _vector(gain, "gain", K, gain.dtype, X.device, fn)
    if residual is not None:
        _rows(residual, "residual", X, fn)
        if H is None:
            H = X.new_empty((T, K))
        else:
            _rows(H, "H", X, fn)
    elif H is not None:
        raise SbnError(fn, 2, "H is written only with a residual (without one, h is X)")
    if rstd is None:
        rstd = X.new_empty(T, dtype=torch.float32)
    else:
        _vector(rstd, "rstd", T, torch.float32, X.device, fn)
    return dt, gdt, T, K, H, rstd


def sbn_rmsnorm(X, gain, *, residual=None, eps: float = 1e-6, H=None, Y=None, rstd=None, stream=None):
    """h = X + residual and its RMS norm Y = h * rstd * gain, X [T, K] bf16 or
    float32.  Returns (Y, H, rstd); H is X itself without a residual."""
    if stream is not None:
        return _on(stream, sbn_rmsnorm, locals())
    fn = "sbn_rmsnorm"
    dt, gdt, T, K, H, rstd = _norm_args(fn, X, gain, residual, H, rstd)
    if Y is None:
        Y = X.new_empty((T, K))
    else:
        _rows(Y, "Y", X, fn)
    if T:
        _check(fn, _so().sbn_rmsnorm(X.data_ptr(), _ld(X), _addr(residual), 0 if residual is None else _ld(residual),
                                     dt, gain.data_ptr(), gdt, T, K, eps, _addr(H), 0 if H is None else _ld(H),
                                     Y.data_ptr(), _ld(Y), rstd.data_ptr(), _raw_stream(X.device)))
    return Y, X if H is None else H, rstd


def sbn_rmsnorm_quant(X, gain, *, residual=None, eps: float = 1e-6, H=None, Xq=None, s_x=None, rstd=None, stream=None):
    """The norm of h = X + residual as the layer's activations: per-token absmax
    int8 codes Xq and scales s_x.  Returns (Xq, s_x, H, rstd); H is X itself
    without a residual."""
    if stream is not None:
        return _on(stream, sbn_rmsnorm_quant, locals())
    fn = "sbn_rmsnorm_quant"
    torch = _torch()
    dt, gdt, T, K, H, rstd = _norm_args(fn, X, gain, residual, H, rstd)
    if Xq is None:
        Xq = X.new_empty((T, K), dtype=torch.int8)
    else:
        _req(Xq, "Xq", "i8", True, fn)
        if Xq.shape != X.shape or Xq.device != X.device:
            raise SbnError(fn, 2, f"Xq must be {tuple(X.shape)} on {X.device}")
    if s_x is None:
        s_x = X.new_empty(T, dtype=torch.float32)
    else:
        _vector(s_x, "s_x", T, torch.float32, X.device, fn)
    if T:
        _check(fn, _so().sbn_rmsnorm_quant(X.data_ptr(), _ld(X), _addr(residual),
                                           0 if residual is None else _ld(residual), dt, gain.data_ptr(), gdt, T, K,
                                           eps, _addr(H), 0 if H is None else _ld(H), Xq.data_ptr(), s_x.data_ptr(),
                                           rstd.data_ptr(), _raw_stream(X.device)))
    return Xq, s_x, X if H is None else H, rstd


@functools.lru_cache(maxsize=1024)
def _norm_scratch_bytes(T: int, K: int) -> int:
    b = _sz()
    fn = "sbn_rmsnorm_backward_workspace_bytes"
    _check(fn, _so().sbn_rmsnorm_backward_workspace_bytes(T, K, ctypes.byref(b)))
    return b.value


def sbn_rmsnorm_backward(dY, H, gain, rstd, *, dH=None, dX=None, dgain=None, ws=None, stream=None):
    """Gradient of sbn_rmsnorm and sbn_rmsnorm_quant from the forward's H and
    rstd; dH is the gradient that reaches h along the residual stream.
    Returns (dX, dgain): dX is the gradient of X and of the residual alike."""
    if stream is not None:
        return _on(stream, sbn_rmsnorm_backward, locals())
    fn = "sbn_rmsnorm_backward"
    torch = _torch()
    _matrix(H, "H", fn)
    dt, gdt = _dtype(H, "H", fn), _dtype(gain, "gain", fn)
    T, K = H.shape
    _rows(dY, "dY", H, fn)
    _vector(gain, "gain", K, gain.dtype, H.device, fn)
    _vector(rstd, "rstd", T, torch.float32, H.device, fn)
    if dH is not None:
        _rows(dH, "dH", H, fn)
    if dX is None:
        dX = H.new_empty((T, K))
    else:
        _rows(dX, "dX", H, fn)
    if dgain is None:
        dgain = H.new_empty(K, dtype=torch.float32)
    else:
        _vector(dgain, "dgain", K, torch.float32, H.device, fn)
    if ws is not None:
        _given(ws, H.device, fn)
    raw = _raw_stream(H.device)
    if ws is None:
        ws = _scratch("rmsnorm_backward", _norm_scratch_bytes(T, K), H.device, raw)
    _check(fn, _so().sbn_rmsnorm_backward(dY.data_ptr(), _ld(dY), H.data_ptr(), _ld(H), _addr(dH),
                                          0 if dH is None else _ld(dH), dt, gain.data_ptr(), gdt, rstd.data_ptr(), T, K,
                                          dX.data_ptr(), _ld(dX), dgain.data_ptr(), ws.data_ptr(), ws.numel(), raw))
    return dX, dgain


# ------------------------------------------------------------------ cross entropy of the head
def _head_args(fn, X, W, labels):
    torch = _torch()
    _matrix(X, "X", fn)
    _matrix(W, "W", fn)
    _req(X, "X", "bf16", False, fn)
    _req(W, "W", "bf16", False, fn)
    if labels.dtype not in (torch.int64, torch.int32):
        raise SbnError(fn, 6, f"labels must be int64 or int32, got {labels.dtype}")
    T, K = X.shape
    V = W.shape[0]
    if W.shape[1] != K or W.device != X.device:
        raise SbnError(fn, 2, f"W {tuple(W.shape)} on {W.device} does not go with X {tuple(X.shape)} on {X.device}")
    _vector(labels, "labels", T, labels.dtype, X.device, fn)
    return T, V, K, 8 if labels.dtype == torch.int64 else 4


@functools.lru_cache(maxsize=1024)
def sbn_cross_entropy_workspace_bytes(T: int, V: int, K: int, backward: bool = False) -> int:
    fn = "sbn_cross_entropy_backward_workspace_bytes" if backward else "sbn_cross_entropy_workspace_bytes"
    b = _sz()
    _check(fn, getattr(_so(), fn)(T, V, K, ctypes.byref(b)))
    return b.value


def sbn_cross_entropy(X, W, labels, *, loss=None, lse=None, ws=None, stream=None):
    """Per-token softmax cross entropy of the logits X W^T, X [T, K] and W
    [V, K] bf16, labels [T] int64 or int32 (outside [0, V): no target, loss 0).
    Returns (loss, lse), float32 [T]; the mean over tokens is the caller's."""
    if stream is not None:
        return _on(stream, sbn_cross_entropy, locals())
    fn = "sbn_cross_entropy"
    torch = _torch()
    T, V, K, lb = _head_args(fn, X, W, labels)
    if loss is None:
        loss = X.new_empty(T, dtype=torch.float32)
    else:
        _vector(loss, "loss", T, torch.float32, X.device, fn)
    if lse is None:
        lse = X.new_empty(T, dtype=torch.float32)
    else:
        _vector(lse, "lse", T, torch.float32, X.device, fn)
    if ws is not None:
        _given(ws, X.device, fn)
    raw = _raw_stream(X.device)
    if ws is None:
        ws = _scratch("cross_entropy", sbn_cross_entropy_workspace_bytes(T, V, K), X.device, raw)
    _check(fn, _so().sbn_cross_entropy(X.data_ptr(), _ld(X), W.data_ptr(), _ld(W), labels.data_ptr(), lb, T, V, K,
                                       loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), raw))
    return loss, lse


def _head_grad_out(t, name, need, dt, like, fn):
    """A gradient of the head's, of type `dt` and the shape of `like`: `t`, checked, or a new one."""
    torch = _torch()
    types = {SBN_BF16: torch.bfloat16, SBN_F32: torch.float32, SBN_F32_FINE: torch.float32}
    if dt not in types:
        raise SbnError(fn, 6, f"{name}'s type must be SBN_BF16, SBN_F32 or SBN_F32_FINE, got {dt}")
    if not need:
        return None
    if t is None:
        return torch.empty(like.shape, dtype=types[dt], device=like.device)
    if t.dtype != types[dt]:
        raise SbnError(fn, 6, f"{name} must be {types[dt]}, got {t.dtype}")
    if t.shape != like.shape or t.device != like.device:
        raise SbnError(fn, 2, f"{name} must be {tuple(like.shape)} on {like.device}")
    _matrix(t, name, fn)
    return t


def sbn_cross_entropy_backward(X, W, labels, lse, dloss, *, dxdt: int = SBN_BF16, dwdt: int = SBN_BF16, dX=None,
                               dW=None, need_dX: bool = True, need_dW: bool = True, ws=None, stream=None):
    """Gradients of the hidden states and of the head's weights from the
    forward's lse and dloss [T], the gradient of each token's loss (float32).
    SBN_F32_FINE: float32, from logit gradients of 16 bits instead of 8, at
    twice the time of that gradient's product.
    Returns (dX, dW), each None where it is not needed."""
    if stream is not None:
        return _on(stream, sbn_cross_entropy_backward, locals())
    fn = "sbn_cross_entropy_backward"
    torch = _torch()
    T, V, K, lb = _head_args(fn, X, W, labels)
    _vector(lse, "lse", T, torch.float32, X.device, fn)
    _vector(dloss, "dloss", T, torch.float32, X.device, fn)
    dX = _head_grad_out(dX, "dX", need_dX, dxdt, X, fn)
    dW = _head_grad_out(dW, "dW", need_dW, dwdt, W, fn)
    if ws is not None:
        _given(ws, X.device, fn)
    raw = _raw_stream(X.device)
    if ws is None:
        ws = _scratch("cross_entropy_backward", sbn_cross_entropy_workspace_bytes(T, V, K, True), X.device, raw)
    _check(fn, _so().sbn_cross_entropy_backward(X.data_ptr(), _ld(X), W.data_ptr(), _ld(W), labels.data_ptr(), lb,
                                                lse.data_ptr(), dloss.data_ptr(), T, V, K, _addr(dX), dxdt,
                                                0 if dX is None else _ld(dX), _addr(dW), dwdt,
                                                0 if dW is None else _ld(dW), ws.data_ptr(), ws.numel(), raw))
    return dX, dW


# ------------------------------------------------------------------ AdamW
class _AdamWEntry(ctypes.Structure):
    _fields_ = [("p", _vp), ("grad", _vp), ("m", _vp), ("v", _vp), ("m_scale", _vp), ("v_scale", _vp),
                ("shadow", _vp), ("n", _i64), ("weight_decay", _f32), ("reserved", _f32)]


class AdamWTable:
    """The tensors of an AdamW step, as a table in device memory, built once and
    used by every sbn_adamw_step: lists of equal length of parameters and
    gradients (each list of one type, bfloat16 or float32, contiguous) and of
    the states, float32 or in 8 bits (m int8, v uint8, with float32 scales, one
    per SBN_ADAMW_BLOCK elements).  `shadows`: bf16 copies of float32
    parameters, written by the step.  `weight_decay`: one number, or one per
    tensor.  No element may be in two of the tensors that the step writes.  The
    table refers to the tensors' memory and keeps them alive."""

    def __init__(self, params, grads, ms, vs, *, m_scales=None, v_scales=None, shadows=None, weight_decay=0.0):
        torch = _torch()
        fn = "AdamWTable"
        count = len(params)
        if count < 1:
            raise SbnError(fn, 2, "no tensors")
        wds = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * count
        if m_scales is None and v_scales is None:
            self.state_bits = 32
        elif m_scales is not None and v_scales is not None:
            self.state_bits = 8
        else:
            raise SbnError(fn, 2, "8-bit states need both m_scales and v_scales")
        none = [None] * count
        lists = {"grads": grads, "ms": ms, "vs": vs, "m_scales": m_scales or none, "v_scales": v_scales or none,
                 "shadows": shadows or none, "weight_decay": wds}
        for name, v in lists.items():
            if len(v) != count:
                raise SbnError(fn, 2, f"{name} has {len(v)} entries for {count} parameters")
        dev = params[0].device
        pt, gt = params[0].dtype, grads[0].dtype
        self.pdt, self.gdt = _dtype(params[0], "params[0]", fn), _dtype(grads[0], "grads[0]", fn)
        mt, vt = (torch.int8, torch.uint8) if self.state_bits == 8 else (torch.float32, torch.float32)
        entries = (_AdamWEntry * count)()
        state = 1 if self.state_bits == 8 else 4
        sizes = {"params": params[0].element_size(), "grads": grads[0].element_size(), "ms": state, "vs": state,
                 "m_scales": 4, "v_scales": 4, "shadows": 2}
        spans = []                                   # first and past the last byte, whether written, name

        def put(t, name, i, dtype, n, shape=None):
            if t is None:
                return None
            if t.dtype != dtype:
                raise SbnError(fn, 6, f"{name}[{i}] must be {dtype}, got {t.dtype}")
            if t.numel() != n or t.device != dev or not t.is_contiguous():
                raise SbnError(fn, 2, f"{name}[{i}] must be contiguous, with {n} elements on {dev}")
            at = t.data_ptr()
            if n:
                spans.append((at, at + n * sizes[name], name != "grads", name, i))
            return at

        for i in range(count):
            n = params[i].numel()
            e = entries[i]
            e.p, e.grad = put(params[i], "params", i, pt, n), put(grads[i], "grads", i, gt, n)
            e.m, e.v = put(ms[i], "ms", i, mt, n), put(vs[i], "vs", i, vt, n)
            ns = -(-n // SBN_ADAMW_BLOCK)
            e.m_scale = put(lists["m_scales"][i], "m_scales", i, torch.float32, ns)
            e.v_scale = put(lists["v_scales"][i], "v_scales", i, torch.float32, ns)
            e.shadow = put(lists["shadows"][i], "shadows", i, torch.bfloat16, n)
            e.n, e.weight_decay = n, wds[i]
        spans.sort()
        read = written = (0, 0)                      # of the spans so far, the one that reaches furthest
        for s in spans:
            if s[0] < written[1] or (s[2] and s[0] < read[1]):
                o = written if s[0] < written[1] else read
                raise SbnError(fn, 2, f"{o[3]}[{o[4]}] and {s[3]}[{s[4]}] share memory that the step writes")
            if s[2]:
                written = s if s[1] > written[1] else written
            else:
                read = s if s[1] > read[1] else read
        blocks = _i64()
        plan = _so().sbn_adamw_plan
        _check("sbn_adamw_plan", plan(entries, count, self.pdt, self.gdt, self.state_bits, None, ctypes.byref(blocks)))
        self.blocks = blocks.value
        mp = torch.empty(max(2 * self.blocks, 2), dtype=torch.int32)
        _check("sbn_adamw_plan", plan(entries, count, self.pdt, self.gdt, self.state_bits, mp.data_ptr(),
                                      ctypes.byref(blocks)))
        raw = torch.frombuffer(bytearray(bytes(entries)), dtype=torch.uint8)
        self.entries, self.map = raw.to(dev), mp.to(dev)
        self.tensors = (list(params), list(grads), list(ms), list(vs), lists["m_scales"], lists["v_scales"],
                        lists["shadows"])


def sbn_adamw_step(table, *, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                   dyn=None, stream=None):
    """One AdamW step on every tensor of `table` (AdamWTable), in place.  `dyn`:
    4 floats in device memory in the place of lr, 1 - beta1^step,
    1 - beta2^step and the gradients' factor 1, for steps replayed from a graph
    (lr and step are then not used, but checked)."""
    if stream is not None:
        return _on(stream, sbn_adamw_step, locals())
    fn = "sbn_adamw_step"
    if not isinstance(table, AdamWTable):
        raise SbnError(fn, 2, "table must be an AdamWTable")
    if dyn is not None:
        _vector(dyn, "dyn", 4, _torch().float32, table.map.device, fn)
    _check(fn, _so().sbn_adamw_step(table.entries.data_ptr(), table.map.data_ptr(), table.blocks, table.pdt, table.gdt,
                                    table.state_bits, lr, beta1, beta2, eps, step, _addr(dyn),
                                    _raw_stream(table.map.device)))


def _decode(codes, scale, second, out, stream):
    if stream is not None:
        return _on(stream, _decode, locals())
    fn = "sbn_adamw_decode_state"
    torch = _torch()
    n = codes.numel()
    _req(codes, "codes", "u8" if second else "i8", True, fn)
    _vector(scale, "scale", -(-n // SBN_ADAMW_BLOCK), torch.float32, codes.device, fn)
    if out is None:
        out = torch.empty(codes.shape, dtype=torch.float32, device=codes.device)
    else:
        _req(out, "out", "f32", True, fn)
        if out.numel() != n or out.device != codes.device:
            raise SbnError(fn, 2, f"out must have {n} elements on {codes.device}")
    _check(fn, _so().sbn_adamw_decode_state(codes.data_ptr(), scale.data_ptr(), n, second, out.data_ptr(),
                                            _raw_stream(codes.device)))
    return out


def sbn_adamw_decode_m(codes, scale, *, out=None, stream=None):
    """The float32 values of an 8-bit first moment (int8 codes, one scale per block)."""
    return _decode(codes, scale, 0, out, stream)


def sbn_adamw_decode_v(codes, scale, *, out=None, stream=None):
    """The float32 values of an 8-bit second moment (uint8 codes, one scale per block)."""
    return _decode(codes, scale, 1, out, stream)


def _encode(x, second, codes, scale, stream):
    if stream is not None:
        return _on(stream, _encode, locals())
    fn = "sbn_adamw_encode_state"
    torch = _torch()
    _req(x, "x", "f32", True, fn)
    n = x.numel()
    dt = torch.uint8 if second else torch.int8
    if codes is None:
        codes = torch.empty(x.shape, dtype=dt, device=x.device)
    else:
        _req(codes, "codes", "u8" if second else "i8", True, fn)
        if codes.numel() != n or codes.device != x.device:
            raise SbnError(fn, 2, f"codes must have {n} elements on {x.device}")
    ns = -(-n // SBN_ADAMW_BLOCK)
    if scale is None:
        scale = torch.empty(ns, dtype=torch.float32, device=x.device)
    else:
        _vector(scale, "scale", ns, torch.float32, x.device, fn)
    _check(fn, _so().sbn_adamw_encode_state(x.data_ptr(), n, second, codes.data_ptr(), scale.data_ptr(),
                                            _raw_stream(x.device)))
    return codes, scale


def sbn_adamw_encode_m(x, *, codes=None, scale=None, stream=None):
    """(int8 codes, scales) of a float32 first moment."""
    return _encode(x, 0, codes, scale, stream)


def sbn_adamw_encode_v(x, *, codes=None, scale=None, stream=None):
    """(uint8 codes, scales) of a float32 second moment."""
    return _encode(x, 1, codes, scale, stream)
