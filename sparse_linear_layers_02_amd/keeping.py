"""Binding of the calls declared in ``include/sbn_keep.h``: 8-bit checkpoints of
what a training step keeps for its backward pass, the RMS norm and the activation
of a feed-forward block that write them, and their gradients from them.

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
from typing import NamedTuple

from . import _SIGNATURES, SBN_BF16, SBN_F32, PKG_DIR, SbnError, _check, _req
from .training import _addr, _dtype, _given, _ld, _matrix, _on, _raw_stream, _rows, _scratch, _so, _sz, _torch, _vector

KEEP_HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "sbn_keep.h")
SBN_KEEP_BLOCK = 128
SBN_RELU2, SBN_SILU = 0, 1

_i64, _int, _vp, _f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float
_SIGNATURES.update({
    "sbn_keep8_encode": ([_vp, _i64, _int, _i64, _i64, _vp, _vp, _vp], _int),
    "sbn_keep8_decode": ([_vp, _vp, _i64, _i64, _vp, _i64, _int, _vp], _int),
    "sbn_rmsnorm_quant_keep": ([_vp, _i64, _vp, _i64, _int, _vp, _int, _i64, _i64, _f32, _vp, _i64, _vp, _vp, _vp, _vp,
                                _vp], _int),
    "sbn_rmsnorm_backward_kept_workspace_bytes": ([_i64, _i64, ctypes.POINTER(_sz)], _int),
    "sbn_rmsnorm_backward_kept": ([_vp, _i64, _vp, _i64, _int, _vp, _vp, _vp, _int, _i64, _i64, _f32, _vp, _i64, _vp,
                                   _vp, _sz, _vp], _int),
    "sbn_activation_quant": ([_vp, _i64, _vp, _i64, _int, _int, _vp, _int, _i64, _i64, _f32, _vp, _vp, _vp, _vp, _vp,
                              _vp, _vp], _int),
    "sbn_activation_backward_workspace_bytes": ([_i64, _i64, ctypes.POINTER(_sz)], _int),
    "sbn_activation_backward": ([_vp, _i64, _int, _vp, _vp, _vp, _vp, _int, _vp, _int, _i64, _i64, _f32, _vp, _i64, _vp,
                                 _i64, _vp, _vp, _sz, _vp], _int),
})


def keep_header_symbols() -> list[str]:
    """Names of the functions declared in include/sbn_keep.h."""
    text = open(KEEP_HEADER_PATH).read()
    return sorted(set(re.findall(r"^\s*sbn_status\s+(sbn_\w+)\s*\(", text, re.M)))


class Kept8(NamedTuple):
    """A matrix [T, K] in 8 bits: int8 codes [T, K], and a float32 scale for each
    SBN_KEEP_BLOCK neighbours of a row, [T, ceil(K / SBN_KEEP_BLOCK)].  A value is
    code * scale."""
    codes: object
    scales: object


def _kept(kept, name: str, shape, device, fn: str):
    """`kept` is a checkpoint of a matrix of `shape` (None: of any) on `device`."""
    torch = _torch()
    try:
        codes, scales = kept
    except (TypeError, ValueError):
        raise SbnError(fn, 2, f"{name} must be a Kept8, or a pair of codes and scales") from None
    if codes.dtype is not torch.int8 or scales.dtype is not torch.float32:
        raise SbnError(fn, 6, f"{name} must be int8 codes and float32 scales, got {codes.dtype} and {scales.dtype}")
    if codes.dim() != 2 or (shape is not None and codes.shape != shape) or codes.device != device:
        raise SbnError(fn, 2, f"{name}'s codes must be {'[T, K]' if shape is None else list(shape)} on {device}, "
                              f"got {list(codes.shape)} on {codes.device}")
    T, K = codes.shape
    if scales.shape != (T, -(-K // SBN_KEEP_BLOCK)) or scales.device != device:
        raise SbnError(fn, 2, f"{name}'s scales must be {[T, -(-K // SBN_KEEP_BLOCK)]} on {device}, "
                              f"got {list(scales.shape)} on {scales.device}")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise SbnError(fn, 2, f"{name} must be contiguous")
    return codes, scales


def _kept_out(kept, name: str, like, fn: str):
    """A checkpoint of `like` to write: `kept`, checked, or a new one."""
    if kept is not None:
        return _kept(kept, name, like.shape, like.device, fn)
    T, K = like.shape
    torch = _torch()
    return (like.new_empty((T, K), dtype=torch.int8),
            like.new_empty((T, -(-K // SBN_KEEP_BLOCK)), dtype=torch.float32))


def _codes_out(Xq, s_x, like, fn):
    """The layer's activations, allocated or checked."""
    torch = _torch()
    T = like.shape[0]
    if Xq is None:
        Xq = like.new_empty(like.shape, dtype=torch.int8)
    else:
        _req(Xq, "Xq", "i8", True, fn)
        if Xq.shape != like.shape or Xq.device != like.device:
            raise SbnError(fn, 2, f"Xq must be {tuple(like.shape)} on {like.device}")
    if s_x is None:
        s_x = like.new_empty(T, dtype=torch.float32)
    else:
        _vector(s_x, "s_x", T, torch.float32, like.device, fn)
    return Xq, s_x


def sbn_keep8_encode(X, *, kept=None, stream=None):
    """The 8-bit checkpoint of X [T, K], bf16 or float32, as a Kept8 (`kept`: one to write)."""
    if stream is not None:
        return _on(stream, sbn_keep8_encode, locals())
    fn = "sbn_keep8_encode"
    _matrix(X, "X", fn)
    dt = _dtype(X, "X", fn)
    T, K = X.shape
    codes, scales = _kept_out(kept, "kept", X, fn)
    _check(fn, _so().sbn_keep8_encode(X.data_ptr(), _ld(X) if T else K, dt, T, K, codes.data_ptr(), scales.data_ptr(),
                                      _raw_stream(X.device)))
    return Kept8(codes, scales)


def sbn_keep8_decode(kept, *, dt: int = SBN_F32, Y=None, stream=None):
    """The values of a checkpoint, as SBN_F32 or SBN_BF16, or of Y's type into Y."""
    if stream is not None:
        return _on(stream, sbn_keep8_decode, locals())
    fn = "sbn_keep8_decode"
    torch = _torch()
    if not isinstance(kept, (tuple, list)) or len(kept) != 2:
        raise SbnError(fn, 2, "kept must be a Kept8, or a pair of codes and scales")
    codes, scales = _kept(kept, "kept", None, kept[0].device, fn)
    T, K = codes.shape
    if Y is None:
        if dt not in (SBN_F32, SBN_BF16):
            raise SbnError(fn, 6, f"dt must be SBN_F32 or SBN_BF16, got {dt}")
        Y = torch.empty((T, K), dtype=torch.float32 if dt == SBN_F32 else torch.bfloat16, device=codes.device)
    else:
        dt = _dtype(Y, "Y", fn)
        _matrix(Y, "Y", fn)
        if Y.shape != codes.shape or Y.device != codes.device:
            raise SbnError(fn, 2, f"Y must be {tuple(codes.shape)} on {codes.device}")
    _check(fn, _so().sbn_keep8_decode(codes.data_ptr(), scales.data_ptr(), T, K, Y.data_ptr(), _ld(Y) if T else K, dt,
                                      _raw_stream(codes.device)))
    return Y


def sbn_rmsnorm_quant_keep(X, gain, *, residual=None, eps: float = 1e-6, H=None, Xq=None, s_x=None, kept=None,
                           stream=None):
    """sbn_rmsnorm_quant, and the 8-bit checkpoint of h = X + residual for
    sbn_rmsnorm_backward_kept.  Returns (Xq, s_x, H, kept); H is X itself without
    a residual."""
    if stream is not None:
        return _on(stream, sbn_rmsnorm_quant_keep, locals())
    fn = "sbn_rmsnorm_quant_keep"
    _matrix(X, "X", fn)
    dt, gdt = _dtype(X, "X", fn), _dtype(gain, "gain", fn)
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
    Xq, s_x = _codes_out(Xq, s_x, X, fn)
    codes, scales = _kept_out(kept, "kept", X, fn)
    if T:
        _check(fn, _so().sbn_rmsnorm_quant_keep(
            X.data_ptr(), _ld(X), _addr(residual), 0 if residual is None else _ld(residual), dt, gain.data_ptr(), gdt, T,
            K, eps, _addr(H), 0 if H is None else _ld(H), Xq.data_ptr(), s_x.data_ptr(), codes.data_ptr(),
            scales.data_ptr(), _raw_stream(X.device)))
    return Xq, s_x, X if H is None else H, Kept8(codes, scales)


@functools.lru_cache(maxsize=1024)
def _scratch_bytes(T: int, K: int, fn: str) -> int:
    b = _sz()
    _check(fn, getattr(_so(), fn)(T, K, ctypes.byref(b)))
    return b.value


def _out(t, name, like, fn):
    if t is None:
        return like.new_empty(like.shape)
    _rows(t, name, like, fn)
    return t


def sbn_rmsnorm_backward_kept(dY, kept, gain, *, eps: float = 1e-6, dH=None, dX=None, dgain=None, ws=None, stream=None):
    """Gradient of sbn_rmsnorm_quant_keep at the values it kept; dH is the
    gradient that reaches h along the residual stream, eps the forward's.
    Returns (dX, dgain): dX is the gradient of X and of the residual alike, of dY's type."""
    if stream is not None:
        return _on(stream, sbn_rmsnorm_backward_kept, locals())
    fn = "sbn_rmsnorm_backward_kept"
    torch = _torch()
    _matrix(dY, "dY", fn)
    dt, gdt = _dtype(dY, "dY", fn), _dtype(gain, "gain", fn)
    T, K = dY.shape
    codes, scales = _kept(kept, "kept", dY.shape, dY.device, fn)
    _vector(gain, "gain", K, gain.dtype, dY.device, fn)
    if dH is not None:
        _rows(dH, "dH", dY, fn)
    dX = _out(dX, "dX", dY, fn)
    if dgain is None:
        dgain = dY.new_empty(K, dtype=torch.float32)
    else:
        _vector(dgain, "dgain", K, torch.float32, dY.device, fn)
    if ws is not None:
        _given(ws, dY.device, fn)
    raw = _raw_stream(dY.device)
    if ws is None:
        ws = _scratch("kept_backward", _scratch_bytes(T, K, "sbn_rmsnorm_backward_kept_workspace_bytes"), dY.device,
                      raw)
    _check(fn, _so().sbn_rmsnorm_backward_kept(dY.data_ptr(), _ld(dY), _addr(dH), 0 if dH is None else _ld(dH), dt,
                                               codes.data_ptr(), scales.data_ptr(), gain.data_ptr(), gdt, T, K, eps,
                                               dX.data_ptr(), _ld(dX), dgain.data_ptr(), ws.data_ptr(), ws.numel(), raw))
    return dX, dgain


def sbn_activation_quant(A, B=None, *, act: int, gain=None, eps: float = 1e-6, keep: bool = True, Xq=None, s_x=None,
                         kept_A=None, kept_B=None, stream=None):
    """u = f(A) * B (f(A) without B), f = SBN_RELU2 or SBN_SILU, as the next
    layer's int8 activations; with a gain, of u's RMS norm.  Returns
    (Xq, s_x, kept_A, kept_B): the 8-bit checkpoints for sbn_activation_backward,
    None with keep=False (inference), kept_B also without B."""
    if stream is not None:
        return _on(stream, sbn_activation_quant, locals())
    fn = "sbn_activation_quant"
    _matrix(A, "A", fn)
    dt = _dtype(A, "A", fn)
    T, K = A.shape
    if B is not None:
        _rows(B, "B", A, fn)
    gdt = SBN_F32
    if gain is not None:
        gdt = _dtype(gain, "gain", fn)
        _vector(gain, "gain", K, gain.dtype, A.device, fn)
    Xq, s_x = _codes_out(Xq, s_x, A, fn)
    none = (None, None)
    ka = kb = none
    if keep:
        ka = _kept_out(kept_A, "kept_A", A, fn)
        if B is not None:
            kb = _kept_out(kept_B, "kept_B", A, fn)
    if (kept_A is not None and ka is none) or (kept_B is not None and kb is none):
        raise SbnError(fn, 2, "a checkpoint to write that the call does not keep")
    if T:
        _check(fn, _so().sbn_activation_quant(
            A.data_ptr(), _ld(A), _addr(B), 0 if B is None else _ld(B), dt, act, _addr(gain), gdt, T, K, eps,
            Xq.data_ptr(), s_x.data_ptr(), _addr(ka[0]), _addr(ka[1]), _addr(kb[0]), _addr(kb[1]),
            _raw_stream(A.device)))
    return Xq, s_x, None if ka is none else Kept8(*ka), None if kb is none else Kept8(*kb)


def sbn_activation_backward(dY, kept_A, kept_B=None, *, act: int, gain=None, eps: float = 1e-6, dA=None, dB=None,
                            dgain=None, ws=None, stream=None):
    """Gradient of sbn_activation_quant at the values it kept; act, gain and eps
    are the forward's.  Returns (dA, dB, dgain), of dY's type and float32; dB is
    None without kept_B, dgain without a gain."""
    if stream is not None:
        return _on(stream, sbn_activation_backward, locals())
    fn = "sbn_activation_backward"
    torch = _torch()
    _matrix(dY, "dY", fn)
    dt = _dtype(dY, "dY", fn)
    T, K = dY.shape
    ca, sa = _kept(kept_A, "kept_A", dY.shape, dY.device, fn)
    cb = sb = None
    dA = _out(dA, "dA", dY, fn)
    if kept_B is not None:
        cb, sb = _kept(kept_B, "kept_B", dY.shape, dY.device, fn)
        dB = _out(dB, "dB", dY, fn)
    elif dB is not None:
        raise SbnError(fn, 2, "dB goes with kept_B")
    gdt = SBN_F32
    if gain is not None:
        gdt = _dtype(gain, "gain", fn)
        _vector(gain, "gain", K, gain.dtype, dY.device, fn)
        if dgain is None:
            dgain = dY.new_empty(K, dtype=torch.float32)
        else:
            _vector(dgain, "dgain", K, torch.float32, dY.device, fn)
    elif dgain is not None:
        raise SbnError(fn, 2, "dgain goes with a gain")
    if ws is not None:
        _given(ws, dY.device, fn)
    raw = _raw_stream(dY.device)
    if ws is None and gain is not None:
        ws = _scratch("kept_backward", _scratch_bytes(T, K, "sbn_activation_backward_workspace_bytes"), dY.device, raw)
    _check(fn, _so().sbn_activation_backward(
        dY.data_ptr(), _ld(dY), dt, ca.data_ptr(), sa.data_ptr(), _addr(cb), _addr(sb), act, _addr(gain), gdt, T, K, eps,
        dA.data_ptr(), _ld(dA), _addr(dB), 0 if dB is None else _ld(dB), _addr(dgain), _addr(ws),
        0 if ws is None else ws.numel(), raw))
    return dA, dB, dgain
