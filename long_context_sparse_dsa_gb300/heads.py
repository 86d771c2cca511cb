"""Norm and rotation of every head of q and k, and their gradient: binding of ``include/dsa_heads.h``.

For models that normalise or rotate their heads: ``qk_norm_rotate`` before the layer (or before the decode calls, with
``positions``), ``qk_norm_rotate_bwd`` behind ``layer_bwd``, whose fp32 gradients it takes.  Checks types and shapes.
"""
from __future__ import annotations

import ctypes

import long_context_sparse_dsa_gb300 as _dsa
from long_context_sparse_dsa_gb300 import decode as _dec


def _refuse(func, dims, *specs):
    """Raise for the first of `specs` (name, tensor, dtype, shape, rows) that is not what the call takes; rows: any distance
    between tokens will do."""
    dev = _dec.torch.cuda.current_device()
    for name, t, dtype, shape, rows in specs:
        if t is None:
            continue
        if not hasattr(t, "get_device") or t.get_device() != dev:
            raise ValueError(f"{func}: {name} must be a tensor on the current device, cuda:{dev} (got {getattr(t, 'device', type(t))})")
        if t.dtype is not dtype or t.shape != shape or not (t.is_contiguous() or rows and len(t) and t[0].is_contiguous()):
            raise ValueError(f"{func}: {name} must be a {dtype} of shape {shape}, {'its tokens' if rows else 'all'} contiguous "
                             f"(got {t.dtype}, {tuple(t.shape)}, strides {t.stride()})")
    raise ValueError(f"{func}: unusable arguments")


def _rows(t, n, dt, shape, row, dev):
    """(fits, distance between tokens) of q or k: the heads of a token are contiguous, tokens any distance apart."""
    if t.dtype is not dt or t.shape != shape or t.get_device() != dev:
        return False, 0
    if t.is_contiguous():
        return True, row
    st = t.stride()
    return st[-1] == 1 and (len(st) == 2 or st[1] == shape[2] or shape[1] == 1), st[0]


def _heads(func, dims, q, k):
    """(device, tokens, layer dtype, fits, q's distance, k's)"""
    first = q if q is not None else k
    if first is None:
        raise ValueError(f"{func}: neither q nor k is given")
    _dec._need_torch()
    dev, n, dt, d = first.get_device(), first.shape[0], _dec._DTYPES[dims.dtype], dims.d
    ok, qs, ks = dev == _dec.torch.cuda.current_device(), 0, 0
    if q is not None and ok:
        ok, qs = _rows(q, n, dt, (n, dims.Hq, d), dims.Hq * d, dev)
    if k is not None and ok:
        ok, ks = _rows(k, n, dt, (n, d), d, dev)
    return dev, n, dt, ok, qs, ks


def _is(t, dtype, shape, dev):
    return t is None or t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


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
    dev, n, dt, ok, qs, ks = _heads("qk_norm_rotate", dims, q, k)
    f32, i32, heads, row, w = _dec.torch.float32, _dec.torch.int32, (n, dims.Hq, dims.d), (n, dims.d), (dims.d,)
    if not (ok and _is(q_out, dt, heads, dev) and _is(k_out, dt, row, dev) and _is(q_weight, f32, w, dev) and
            _is(k_weight, f32, w, dev) and _is(positions, i32, (n,), dev)):
        _refuse("qk_norm_rotate", dims, ("q", q, dt, heads, True), ("k", k, dt, row, True), ("q_out", q_out, dt, heads, False),
                ("k_out", k_out, dt, row, False), ("q_weight", q_weight, f32, w, False), ("k_weight", k_weight, f32, w, False),
                ("positions", positions, i32, (n,), False))
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
    dev, n, dt, ok, qs, ks = _heads("qk_norm_rotate_bwd", dims, q, k)
    f32, i32, heads, row, w = _dec.torch.float32, _dec.torch.int32, (n, dims.Hq, dims.d), (n, dims.d), (dims.d,)
    if not (ok and _is(dq_out, f32, heads, dev) and _is(dk_out, f32, row, dev) and _is(dq, f32, heads, dev) and
            _is(dk, f32, row, dev) and _is(q_weight, f32, w, dev) and _is(k_weight, f32, w, dev) and
            _is(dq_weight, f32, w, dev) and _is(dk_weight, f32, w, dev) and _is(positions, i32, (n,), dev) and
            (ws is None or ws.get_device() == dev and ws.is_contiguous())):
        _refuse("qk_norm_rotate_bwd", dims, ("q", q, dt, heads, True), ("k", k, dt, row, True),
                ("dq_out", dq_out, f32, heads, False), ("dk_out", dk_out, f32, row, False), ("dq", dq, f32, heads, False),
                ("dk", dk, f32, row, False), ("q_weight", q_weight, f32, w, False), ("k_weight", k_weight, f32, w, False),
                ("dq_weight", dq_weight, f32, w, False), ("dk_weight", dk_weight, f32, w, False),
                ("positions", positions, i32, (n,), False), ("ws", ws, ws.dtype if ws is not None else None,
                                                             ws.shape if ws is not None else None, False))
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
