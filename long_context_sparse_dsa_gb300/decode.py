"""Decoding with the DSA layer from a paged cache: binding of ``include/dsa_decode.h``.

Like the package's other entry points these calls only check and marshal their arguments; the caller owns
every tensor.  Unlike them they also check types and shapes, since a decoder's integer arguments (lengths,
block tables) are easily of another type.

A decoder keeps a ``PagedCache``, a workspace (``alloc_decode_workspace``) and, if its model rotates keys and
queries, a ``Rotation``; per step it advances ``lens`` and calls ``decode_step``, or the three calls it is made
of: ``cache_append``, ``decode_indexer_topk``, ``decode_attn``.  All of them can be captured into a CUDA graph.
``cache_append`` and ``decode_step`` take a sequence once per call; the draft tokens of a sequence are appended together
(offsets) and then are a row each, with the same block-table row and growing lens, for the other two.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass, field

import long_context_sparse_dsa_gb300 as _dsa

torch = _DTYPES = None   # set by _need_torch(): importing the package (to build it, say) does not need torch


def _need_torch():
    """Every call of this module needs an object made by one of the functions that call this."""
    global torch, _DTYPES
    if torch is None:
        import torch as t
        _DTYPES = {_dsa.DSA_FP32: t.float32, _dsa.DSA_BF16: t.bfloat16}
        torch = t


class _CCache(ctypes.Structure):
    """Mirror of ``dsa_paged_cache``."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("kpool", ctypes.c_void_p),
                ("ktail", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32)]


class _CRotation(ctypes.Structure):
    """Mirror of ``dsa_rotation``."""
    _fields_ = [("turns", ctypes.c_void_p), ("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


@dataclass(frozen=True, eq=False)
class PagedCache:
    """k, v [pages, page_size, d], kpool [pages, page_size / 4, di], ktail [pages, 3, di], in the layer dtype.

    An array that no call uses may be None (``decode_attn`` reads k and v, ``decode_indexer_topk`` kpool,
    ``cache_append`` writes all four)."""
    k: object = None
    v: object = None
    kpool: object = None
    ktail: object = None
    pages: int = field(init=False)
    page_size: int = field(init=False)
    _c: object = field(init=False, repr=False)

    def __post_init__(self):
        _need_torch()
        given = [t for t in (self.k, self.v, self.kpool, self.ktail) if t is not None]
        if not given or (self.k is None and self.kpool is None):
            raise ValueError("a paged cache has k and v, or kpool, or all of k, v, kpool and ktail")
        first = given[0]
        for t in given:
            _dsa._ptr(t)    # CUDA, contiguous
            if t.dim() != 3 or t.shape[0] != first.shape[0] or t.dtype != first.dtype or t.device != first.device:
                raise ValueError("the cache's arrays are 3-dimensional, with the same pages, dtype and device")
        page = self.k.shape[1] if self.k is not None else 4 * self.kpool.shape[1]
        if page < 4 or page % 4:
            raise ValueError(f"page_size must be a positive multiple of 4 (got {page})")
        if (self.k is None) != (self.v is None) or (self.k is not None and self.k.shape != self.v.shape):
            raise ValueError("k and v have one shape")
        if self.kpool is not None and self.kpool.shape[1] != page // 4:
            raise ValueError("kpool has page_size / 4 rows per page")
        if self.ktail is not None and (self.ktail.shape[1] != 3 or self.kpool is None or
                                       self.ktail.shape[2] != self.kpool.shape[2]):
            raise ValueError("ktail is [pages, 3, di], beside a kpool of the same di")
        put = object.__setattr__
        put(self, "pages", int(first.shape[0]))
        put(self, "page_size", int(page))
        put(self, "_device", first.get_device())
        put(self, "_dtype", first.dtype)
        put(self, "_d", None if self.k is None else int(self.k.shape[2]))
        put(self, "_di", None if self.kpool is None else int(self.kpool.shape[2]))
        put(self, "_c", _CCache(_dsa._ptr(self.k), _dsa._ptr(self.v), _dsa._ptr(self.kpool), _dsa._ptr(self.ktail),
                                self.pages, self.page_size))
        put(self, "_ref", ctypes.byref(self._c))


def alloc_paged_cache(dims, pages: int, page_size: int = 64, device="cuda") -> PagedCache:
    """Uninitialised arrays of a cache of `pages` pages for the layer `dims` (nothing in them needs a value)."""
    _need_torch()
    _dsa._check(validate_decode_dims(dims), "dsa_validate_decode_dims")
    dt = _DTYPES[dims.dtype]
    e = lambda *shape: torch.empty(shape, dtype=dt, device=device)
    return PagedCache(k=e(pages, page_size, dims.d), v=e(pages, page_size, dims.d),
                      kpool=e(pages, page_size // 4, dims.di), ktail=e(pages, 3, dims.di))


class Rotation:
    """Position rotation of the first 2 * len(freq) channels: see ``make_rotation``.  turns: the frequencies as turns per
    position in units of 2^-64, an int64 tensor."""

    def __init__(self, turns, interleaved: bool):
        _need_torch()
        if not (isinstance(turns, torch.Tensor) and turns.dtype is torch.int64 and turns.dim() == 1 and
                turns.is_contiguous() and turns.numel() and turns.numel() % 8 == 0):
            raise ValueError("a rotation's turns are a contiguous int64 tensor of a multiple of 8 frequencies")
        self.turns = turns
        self.dim = 2 * turns.numel()
        self._c = _CRotation(turns.data_ptr(), self.dim, int(bool(interleaved)))
        self._ref = ctypes.byref(self._c)


def make_rotation(freq, interleaved: bool = False, device="cuda") -> Rotation:
    """freq: the pairs' frequencies in radians per position, e.g. ``base ** (-arange(0, dim, 2) / dim)``, as a float64
    tensor or a sequence of numbers.  Pair i is channels (i, i + dim/2), or (2i, 2i+1) when interleaved."""
    _need_torch()
    values = [float(f) for f in (freq.tolist() if hasattr(freq, "tolist") else freq)]
    if not values or len(values) % 8 or not all(math.isfinite(f) for f in values):
        raise ValueError("a rotation has a multiple of 8 finite frequencies")
    # turns per position in units of 2^-64, modulo a whole turn, as the int64 of the same bits
    turns = [int(round((f / (2.0 * math.pi)) % 1.0 * 2.0 ** 64)) % 2 ** 64 for f in values]
    turns = [t - 2 ** 64 if t >= 2 ** 63 else t for t in turns]
    return Rotation(torch.tensor(turns, dtype=torch.int64, device=device), interleaved)


# A decoder makes these calls for every token, so each checks its tensors in one plain condition (a few attribute
# reads per tensor) and only looks for what is wrong when it fails.


def _refuse(func, dims, cache, *specs):
    """Raise for the first of `specs` (name, tensor, dtype, shape) that is not what the call takes."""
    device = cache._device
    if device != torch.cuda.current_device():
        raise ValueError(f"{func}: the cache is on cuda:{device}, not on the current device")
    if cache._dtype is not _DTYPES[dims.dtype]:
        raise ValueError(f"{func}: the cache is not of the layer's dtype")
    if cache._d not in (None, dims.d) or cache._di not in (None, dims.di):
        raise ValueError(f"{func}: the cache is of d = {cache._d}, di = {cache._di}, the layer of {dims.d}, {dims.di}")
    for name, t, dtype, shape in specs:
        if t is not None and (t.get_device() != device or not t.is_contiguous() or
                              dtype is not None and (t.dtype is not dtype or t.shape != shape)):
            raise ValueError(f"{func}: {name} must be a contiguous {dtype or 'tensor'} of shape {shape} on cuda:{device} "
                             f"(got {t.dtype}, {tuple(t.shape)}, strides {t.stride()}, {t.device})")
    raise ValueError(f"{func}: unusable arguments")


def _cache_ok(dims, cache, dt):
    return (cache._device == torch.cuda.current_device() and cache._dtype is dt and
            (cache._d is None or cache._d == dims.d) and (cache._di is None or cache._di == dims.di))


def _raw_stream(stream, device):
    if stream is None:   # what torch.cuda.current_stream().cuda_stream gives, without a Stream object per call
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def validate_decode_dims(dims) -> int:
    return _dsa._load().dsa_validate_decode_dims(ctypes.byref(dims))


def decode_workspace_bytes(dims, batch: int) -> int:
    return int(_dsa._load().dsa_decode_workspace_bytes(ctypes.byref(dims), int(batch)))


def alloc_decode_workspace(dims, batch: int, device="cuda"):
    """Scratch of the decode calls for up to `batch` rows; calls that may overlap on the GPU need one each."""
    _need_torch()
    n = decode_workspace_bytes(dims, batch)
    if n == 0:
        _dsa._check(validate_decode_dims(dims), "dsa_decode_workspace_bytes")
        raise _dsa.DSAError(_dsa.DSA_ERR_INVALID_ARG, "dsa_decode_workspace_bytes", f"batch {batch}")
    return torch.empty((n,), dtype=torch.uint8, device=device)


def cache_append(dims, cache, lens, block_table, k, v, k_idx, offsets=None, rotation=None, q=None, q_out=None,
                 k_out=None, stream=None):
    """New tokens into the cache; lens [batch] int32 count them.  Without offsets one token per row, with offsets
    [batch + 1] int32 rows offsets[b] .. offsets[b+1]-1 of k, v, k_idx (q) are row b's.  With a rotation, k enters the
    cache rotated to its position (and goes to k_out), and q goes to q_out rotated.  No two rows append to the same page."""
    dt, i32, dev = _DTYPES[dims.dtype], torch.int32, cache._device
    batch, n, d = lens.numel(), k.shape[0], dims.d
    cols = -(-dims.L // cache.page_size)
    row, index = (n, d), (n, dims.di)
    ok = (_cache_ok(dims, cache, dt) and
          lens.dtype is i32 and lens.shape == (batch,) and lens.get_device() == dev and lens.is_contiguous() and
          block_table.dtype is i32 and block_table.shape == (batch, cols) and block_table.get_device() == dev and
          block_table.is_contiguous() and
          k.dtype is dt and k.shape == row and k.get_device() == dev and k.is_contiguous() and
          v.dtype is dt and v.shape == row and v.get_device() == dev and v.is_contiguous() and
          k_idx.dtype is dt and k_idx.shape == index and k_idx.get_device() == dev and k_idx.is_contiguous())
    po = pr = pq = pqo = pko = None
    if offsets is not None:
        ok = (ok and offsets.dtype is i32 and offsets.shape == (batch + 1,) and offsets.get_device() == dev and
              offsets.is_contiguous())
        po = offsets.data_ptr()
    if rotation is not None:
        ok = ok and rotation.turns.get_device() == dev
        pr = rotation._ref
    if q is not None:
        heads = (n, dims.Hq, d)
        ok = ok and q.dtype is dt and q.shape == heads and q.get_device() == dev and q.is_contiguous()
        pq = q.data_ptr()
    if q_out is not None:
        heads = (n, dims.Hq, d)
        ok = ok and q_out.dtype is dt and q_out.shape == heads and q_out.get_device() == dev and q_out.is_contiguous()
        pqo = q_out.data_ptr()
    if k_out is not None:
        ok = ok and k_out.dtype is dt and k_out.shape == row and k_out.get_device() == dev and k_out.is_contiguous()
        pko = k_out.data_ptr()
    if not ok:
        heads = (n, dims.Hq, d)
        _refuse("cache_append", dims, cache, ("lens", lens, i32, (batch,)), ("block_table", block_table, i32, (batch, cols)),
                ("k", k, dt, row), ("v", v, dt, row), ("k_idx", k_idx, dt, index), ("offsets", offsets, i32, (batch + 1,)),
                ("q", q, dt, heads), ("q_out", q_out, dt, heads), ("k_out", k_out, dt, row),
                ("the rotation", None if rotation is None else rotation.turns, None, None))
    st = _dsa._load().dsa_cache_append(
        ctypes.byref(dims), cache._ref, batch, lens.data_ptr(), block_table.data_ptr(), n, po, k.data_ptr(), v.data_ptr(),
        k_idx.data_ptr(), pr, pq, pqo, pko, _raw_stream(stream, dev))
    if st:
        _dsa._check(st, "dsa_cache_append")


def decode_indexer_topk(dims, cache, lens, block_table, q_idx, w, idx, ws, stream=None):
    """The min(k, lens[b] // 4) best complete pools of every row, ascending, then -1, into idx [batch, k] int32."""
    dt, i32, f32, dev, batch = _DTYPES[dims.dtype], torch.int32, torch.float32, cache._device, lens.numel()
    cols = -(-dims.L // cache.page_size)
    queries, weights, chosen = (batch, dims.Hi, dims.di), (batch, dims.Hi), (batch, dims.k)
    if not (_cache_ok(dims, cache, dt) and
            lens.dtype is i32 and lens.shape == (batch,) and lens.get_device() == dev and lens.is_contiguous() and
            block_table.dtype is i32 and block_table.shape == (batch, cols) and block_table.get_device() == dev and
            block_table.is_contiguous() and
            q_idx.dtype is dt and q_idx.shape == queries and q_idx.get_device() == dev and q_idx.is_contiguous() and
            w.dtype is f32 and w.shape == weights and w.get_device() == dev and w.is_contiguous() and
            idx.dtype is i32 and idx.shape == chosen and idx.get_device() == dev and idx.is_contiguous() and
            (ws is None or ws.get_device() == dev and ws.is_contiguous())):
        _refuse("decode_indexer_topk", dims, cache, ("lens", lens, i32, (batch,)),
                ("block_table", block_table, i32, (batch, cols)), ("q_idx", q_idx, dt, queries), ("w", w, f32, weights),
                ("idx", idx, i32, chosen), ("ws", ws, None, None))
    pw, nw = (None, 0) if ws is None else (ws.data_ptr(), ws.nbytes)
    st = _dsa._load().dsa_decode_indexer_topk(
        ctypes.byref(dims), cache._ref, batch, lens.data_ptr(), block_table.data_ptr(), q_idx.data_ptr(), w.data_ptr(),
        idx.data_ptr(), pw, nw, _raw_stream(stream, dev))
    if st:
        _dsa._check(st, "dsa_decode_indexer_topk")


def decode_attn(dims, cache, lens, block_table, q, o, lse, ws, idx=None, stream=None):
    """Attention of one query per row: over the pools of idx [batch, k] and the row's partial pool, or, without idx, over
    all of the row's tokens.  o [batch, Hq, d], lse [batch, Hq] fp32."""
    dt, i32, f32, dev, batch = _DTYPES[dims.dtype], torch.int32, torch.float32, cache._device, lens.numel()
    cols, heads = -(-dims.L // cache.page_size), (batch, dims.Hq, dims.d)
    if not (_cache_ok(dims, cache, dt) and
            lens.dtype is i32 and lens.shape == (batch,) and lens.get_device() == dev and lens.is_contiguous() and
            block_table.dtype is i32 and block_table.shape == (batch, cols) and block_table.get_device() == dev and
            block_table.is_contiguous() and
            (idx is None or idx.dtype is i32 and idx.shape == (batch, dims.k) and idx.get_device() == dev and
             idx.is_contiguous()) and
            q.dtype is dt and q.shape == heads and q.get_device() == dev and q.is_contiguous() and
            o.dtype is dt and o.shape == heads and o.get_device() == dev and o.is_contiguous() and
            lse.dtype is f32 and lse.shape == heads[:2] and lse.get_device() == dev and lse.is_contiguous() and
            (ws is None or ws.get_device() == dev and ws.is_contiguous())):
        _refuse("decode_attn", dims, cache, ("lens", lens, i32, (batch,)), ("block_table", block_table, i32, (batch, cols)),
                ("idx", idx, i32, (batch, dims.k)), ("q", q, dt, heads), ("o", o, dt, heads), ("lse", lse, f32, heads[:2]),
                ("ws", ws, None, None))
    pw, nw = (None, 0) if ws is None else (ws.data_ptr(), ws.nbytes)
    st = _dsa._load().dsa_decode_attn(
        ctypes.byref(dims), cache._ref, batch, lens.data_ptr(), block_table.data_ptr(),
        None if idx is None else idx.data_ptr(), q.data_ptr(), o.data_ptr(), lse.data_ptr(), pw, nw,
        _raw_stream(stream, dev))
    if st:
        _dsa._check(st, "dsa_decode_attn")


def decode_step(dims, cache, lens, block_table, q, k, v, q_idx, k_idx, w, o, lse, idx, ws, rotation=None, stream=None):
    """One decode step: append one token per row, select its pools (idx), attend to them (o, lse).  No two rows append to
    the same page."""
    dt, i32, f32, dev, batch = _DTYPES[dims.dtype], torch.int32, torch.float32, cache._device, lens.numel()
    specs = (("lens", lens, i32, (batch,)), ("block_table", block_table, i32, (batch, -(-dims.L // cache.page_size))),
             ("q", q, dt, (batch, dims.Hq, dims.d)), ("k", k, dt, (batch, dims.d)), ("v", v, dt, (batch, dims.d)),
             ("q_idx", q_idx, dt, (batch, dims.Hi, dims.di)), ("k_idx", k_idx, dt, (batch, dims.di)),
             ("w", w, f32, (batch, dims.Hi)), ("o", o, dt, (batch, dims.Hq, dims.d)), ("lse", lse, f32, (batch, dims.Hq)),
             ("idx", idx, i32, (batch, dims.k)))
    ok = _cache_ok(dims, cache, dt)
    for _, t, dtype, shape in specs:
        ok = ok and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()
    pr = None
    if rotation is not None:
        ok = ok and rotation.turns.get_device() == dev
        pr = rotation._ref
    if not ok or ws is not None and not (ws.get_device() == dev and ws.is_contiguous()):
        _refuse("decode_step", dims, cache, *specs, ("ws", ws, None, None),
                ("the rotation", None if rotation is None else rotation.turns, None, None))
    pw, nw = (None, 0) if ws is None else (ws.data_ptr(), ws.nbytes)
    st = _dsa._load().dsa_decode_step(
        ctypes.byref(dims), cache._ref, batch, lens.data_ptr(), block_table.data_ptr(), q.data_ptr(), k.data_ptr(),
        v.data_ptr(), q_idx.data_ptr(), k_idx.data_ptr(), w.data_ptr(), pr, o.data_ptr(), lse.data_ptr(),
        idx.data_ptr(), pw, nw, _raw_stream(stream, dev))
    if st:
        _dsa._check(st, "dsa_decode_step")


def _signatures(D):
    P, i64, size = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    C, R = ctypes.POINTER(_CCache), ctypes.POINTER(_CRotation)
    return {
        "dsa_validate_decode_dims": ([D], ctypes.c_int),
        "dsa_decode_workspace_bytes": ([D, i64], size),
        "dsa_cache_append": ([D, C, i64, P, P, i64, P, P, P, P, R, P, P, P, P], ctypes.c_int),
        "dsa_decode_indexer_topk": ([D, C, i64, P, P, P, P, P, P, size, P], ctypes.c_int),
        "dsa_decode_attn": ([D, C, i64, P, P, P, P, P, P, P, size, P], ctypes.c_int),
        "dsa_decode_step": ([D, C, i64, P, P, P, P, P, P, P, P, R, P, P, P, P, size, P], ctypes.c_int),
    }
