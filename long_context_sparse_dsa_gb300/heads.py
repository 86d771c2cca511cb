"""Norm and rotation of every head of q and k, and their gradient: binding of ``include/dsa_heads.h``.

For models that normalise or rotate their heads: ``qk_norm_rotate`` before the layer (or before the decode calls, with
``positions``), ``qk_norm_rotate_bwd`` behind ``layer_bwd``, whose fp32 gradients it takes.  Checks types and shapes.
"""
from __future__ import annotations

import ctypes

import long_context_sparse_dsa_gb300 as _dsa
from long_context_sparse_dsa_gb300 import decode as _dec


def _fail(func, name, t, want):
    got = type(t).__name__ if not hasattr(t, "stride") else f"{t.dtype}, {tuple(t.shape)}, strides {t.stride()}, {t.device}"
    raise ValueError(f"{func}: {name} must be {want} (got {got})")


def _need(func, dev, *specs):
    """Raise for the first of `specs` (name, tensor or None, dtype, shape) that is not contiguous, of that type, shape, device."""
    for name, t, dtype, shape in specs:
        if t is not None and not (t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
            _fail(func, name, t, f"a contiguous {dtype} of shape {shape} on cuda:{dev}")


def _device(func, t):
    dev = t.get_device()
    if dev < 0 or dev != _dec.torch.cuda.current_device():
        raise ValueError(f"{func}: the tensors must be on the current CUDA device (got {t.device})")
    return dev


def _heads(func, dims, q, k):
    """(device, tokens, q's stride, k's): the heads of a token are contiguous, tokens any distance apart."""
    first = q if q is not None else k
    if first is None:
        raise ValueError(f"{func}: neither q nor k is given")
    _dec._need_torch()
    dev, n, dt = _device(func, first), first.shape[0], _dec._DTYPES[dims.dtype]
    strides = []
    for name, t, shape in (("q", q, (n, dims.Hq, dims.d)), ("k", k, (n, dims.d))):
        if t is None:
            strides.append(0)
            continue
        inner = (dims.d, 1) if t.dim() == 3 else (1,)
        if not (t.dtype is dt and t.shape == shape and t.get_device() == dev and
                (t.stride()[1:] == inner or n == 0 or name == "q" and dims.Hq == 1 and t.stride()[2] == 1)):
            _fail(func, name, t, f"a {dt} of shape {shape} on cuda:{dev} whose rows are contiguous")
        row = dims.Hq * dims.d if name == "q" else dims.d
        strides.append(t.stride(0) if n > 1 else row)
    return dev, n, strides[0], strides[1]


def _p(t):
    return None if t is None else t.data_ptr()


def _turns(func, rotation, dev):
    if rotation is None:
        return None
    if rotation.turns.get_device() != dev:
        raise ValueError(f"{func}: the rotation is on {rotation.turns.device}, not on cuda:{dev}")
    return rotation._ref


def qk_norm_rotate(dims, q, k, q_out, k_out, eps, q_weight=None, k_weight=None, rotation=None, positions=None, stream=None):
    """q_out [T, Hq, d] and k_out [T, d] = the heads of q and k divided by their root mean square, times the weights [d]
    (fp32; None: 1), rotated to positions [T] int32 (None: token t is at t).  q and k may be slices of a wider tensor (any
    distance between tokens); either pair may be None.  The outputs may be q and k themselves where these are contiguous."""
    dev, n, qs, ks = _heads("qk_norm_rotate", dims, q, k)
    dt, f32 = _dec._DTYPES[dims.dtype], _dec.torch.float32
    _need("qk_norm_rotate", dev, ("q_out", q_out, dt, (n, dims.Hq, dims.d)), ("k_out", k_out, dt, (n, dims.d)),
          ("q_weight", q_weight, f32, (dims.d,)), ("k_weight", k_weight, f32, (dims.d,)),
          ("positions", positions, _dec.torch.int32, (n,)))
    if (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("qk_norm_rotate: an input without its output, or the reverse")
    st = _dsa._load().dsa_qk_norm_rotate(
        ctypes.byref(dims), n, _p(q), qs, _p(k), ks, _p(q_weight), _p(k_weight), eps,
        _turns("qk_norm_rotate", rotation, dev), _p(positions), _p(q_out), _p(k_out), _dec._raw_stream(stream, dev))
    if st:
        _dsa._check(st, "dsa_qk_norm_rotate")


def qk_norm_bwd_workspace_bytes(dims, n_tokens: int) -> int:
    return int(_dsa._load().dsa_qk_norm_bwd_workspace_bytes(ctypes.byref(dims), int(n_tokens)))


def qk_norm_rotate_bwd(dims, q, k, dq_out, dk_out, dq, dk, eps, ws, q_weight=None, k_weight=None, dq_weight=None,
                       dk_weight=None, rotation=None, positions=None, stream=None):
    """Gradients of ``qk_norm_rotate``: dq, dk (fp32; may be dq_out, dk_out themselves) of its inputs q, k, and, where
    given, dq_weight, dk_weight [d] fp32 (written, not added to).  dq_out, dk_out: fp32, as ``layer_bwd`` leaves them."""
    dev, n, qs, ks = _heads("qk_norm_rotate_bwd", dims, q, k)
    f32 = _dec.torch.float32
    heads, row = (n, dims.Hq, dims.d), (n, dims.d)
    _need("qk_norm_rotate_bwd", dev, ("dq_out", dq_out, f32, heads), ("dk_out", dk_out, f32, row), ("dq", dq, f32, heads),
          ("dk", dk, f32, row), ("q_weight", q_weight, f32, (dims.d,)), ("k_weight", k_weight, f32, (dims.d,)),
          ("dq_weight", dq_weight, f32, (dims.d,)), ("dk_weight", dk_weight, f32, (dims.d,)),
          ("positions", positions, _dec.torch.int32, (n,)), ("ws", ws, _dec.torch.uint8, ws.shape if ws is not None else None))
    if any((x is None) != (y is None) for x, y in ((q, dq_out), (q, dq), (k, dk_out), (k, dk))):
        raise ValueError("qk_norm_rotate_bwd: an input without its gradients, or the reverse")
    st = _dsa._load().dsa_qk_norm_rotate_bwd(
        ctypes.byref(dims), n, _p(q), qs, _p(k), ks, _p(q_weight), _p(k_weight), eps,
        _turns("qk_norm_rotate_bwd", rotation, dev), _p(positions), _p(dq_out), _p(dk_out), _p(dq), _p(dk), _p(dq_weight),
        _p(dk_weight), _p(ws), 0 if ws is None else ws.nbytes, _dec._raw_stream(stream, dev))
    if st:
        _dsa._check(st, "dsa_qk_norm_rotate_bwd")


def _signatures(D):
    P, i64, size, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    R = ctypes.POINTER(_dec._CRotation)
    return {
        "dsa_qk_norm_rotate": ([D, i64, P, i64, P, i64, P, P, f32, R, P, P, P, P], ctypes.c_int),
        "dsa_qk_norm_bwd_workspace_bytes": ([D, i64], size),
        "dsa_qk_norm_rotate_bwd": ([D, i64, P, i64, P, i64, P, P, f32, R, P, P, P, P, P, P, P, P, size, P], ctypes.c_int),
    }
