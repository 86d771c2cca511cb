"""Drafted tokens judged in one pass, and the pages behind them: binding of ``include/dsa_tree.h`` and ``include/dsa_pages.h``.

``decode_tree_attn`` attends with every node of each row's draft tree to the row's cached tokens and the node's
ancestors; ``cache_commit`` appends the accepted path.  ``cache_reserve``, ``cache_fork``, ``cache_release``,
``cache_compact`` and ``cache_copy_pages`` keep account of a ``PagedCache``'s pages in an int32 tensor ``refs`` [pages]
that the caller owns (zeros for an empty cache).  Everything the calls read lies on the device: all can be captured into
a CUDA graph.  Types and shapes are checked as in ``decode.py``.
"""
from __future__ import annotations

import ctypes

import long_context_sparse_dsa_gb300 as _dsa
from long_context_sparse_dsa_gb300 import decode as _dec

MAX_TREE_NODES = 128


def _ok(t, dtype, shape, dev):
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _check_all(func, dims, cache, specs, ws=None):
    """`specs`: (name, tensor or None, dtype, shape)."""
    dev = cache._device
    ok = _dec._cache_ok(dims, cache, _dec._DTYPES[dims.dtype])
    for _, t, dtype, shape in specs:
        ok = ok and (t is None or _ok(t, dtype, shape, dev))
    if not ok or ws is not None and not (ws.get_device() == dev and ws.is_contiguous()):
        _dec._refuse(func, dims, cache, *specs, ("ws", ws, None, None))


def _cols(dims, cache):
    return -(-dims.L // cache.page_size)


def _p(t):
    return None if t is None else t.data_ptr()


def _ws(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.nbytes)


def tree_workspace_bytes(dims, batch: int, n_nodes: int) -> int:
    return int(_dsa._load().dsa_tree_workspace_bytes(ctypes.byref(dims), int(batch), int(n_nodes)))


def alloc_tree_workspace(dims, batch: int, n_nodes: int, device="cuda"):
    """Scratch of ``decode_tree_attn`` for up to `batch` rows with `n_nodes` nodes in all."""
    _dec._need_torch()
    n = tree_workspace_bytes(dims, batch, n_nodes)
    if n == 0:
        _dsa._check(_dec.validate_decode_dims(dims), "dsa_tree_workspace_bytes")
        raise _dsa.DSAError(_dsa.DSA_ERR_INVALID_ARG, "dsa_tree_workspace_bytes", f"batch {batch}, n_nodes {n_nodes}")
    return _dec.torch.empty((n,), dtype=_dec.torch.uint8, device=device)


def decode_tree_attn(dims, cache, lens, block_table, offsets, parents, q, k, v, o, lse, ws, idx=None, stream=None):
    """Attention of the nodes of each row's draft tree.  lens [batch] int32: the row's cached tokens, drafts not included;
    offsets [batch + 1] int32: row b's nodes are rows offsets[b] .. offsets[b+1]-1 (at most 128) of the node tensors;
    parents [T] int32: a node's parent within its row, -1 for the cached tokens' end (None: chains).  Node t attends to
    the row's tokens (or, with idx [T, k], to the pools named and the row's partial pool), its ancestors and itself.
    q [T, Hq, d], k, v [T, d] -> o [T, Hq, d], lse [T, Hq] fp32."""
    i32, f32, batch, n = _dec.torch.int32, _dec.torch.float32, lens.numel(), q.shape[0]
    dt, heads = _dec._DTYPES[dims.dtype], (n, dims.Hq, dims.d)
    _check_all("decode_tree_attn", dims, cache, (
        ("lens", lens, i32, (batch,)), ("block_table", block_table, i32, (batch, _cols(dims, cache))),
        ("offsets", offsets, i32, (batch + 1,)), ("parents", parents, i32, (n,)), ("idx", idx, i32, (n, dims.k)),
        ("q", q, dt, heads), ("k", k, dt, (n, dims.d)), ("v", v, dt, (n, dims.d)), ("o", o, dt, heads),
        ("lse", lse, f32, heads[:2])), ws)
    pw, nw = _ws(ws)
    st = _dsa._load().dsa_decode_tree_attn(
        ctypes.byref(dims), cache._ref, batch, lens.data_ptr(), block_table.data_ptr(), n, offsets.data_ptr(), _p(parents),
        _p(idx), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), pw, nw,
        _dec._raw_stream(stream, cache._device))
    if st:
        _dsa._check(st, "dsa_decode_tree_attn")


def cache_commit(dims, cache, lens, block_table, offsets, parents, accepted, k, v, k_idx, lens_out, stream=None):
    """The path from the root to node accepted[b] ([batch] int32; -1: nothing) of each row's draft tree becomes the row's
    next tokens, from position lens[b] on: k, v [T, d] and k_idx [T, di] of its nodes enter the cache.  lens_out [batch]
    int32 (may be lens): the new lengths.  offsets, parents: as in ``decode_tree_attn``."""
    i32, batch, n = _dec.torch.int32, lens.numel(), k.shape[0]
    dt = _dec._DTYPES[dims.dtype]
    _check_all("cache_commit", dims, cache, (
        ("lens", lens, i32, (batch,)), ("block_table", block_table, i32, (batch, _cols(dims, cache))),
        ("offsets", offsets, i32, (batch + 1,)), ("parents", parents, i32, (n,)), ("accepted", accepted, i32, (batch,)),
        ("k", k, dt, (n, dims.d)), ("v", v, dt, (n, dims.d)), ("k_idx", k_idx, dt, (n, dims.di)),
        ("lens_out", lens_out, i32, (batch,))))
    st = _dsa._load().dsa_cache_commit(
        ctypes.byref(dims), cache._ref, batch, lens.data_ptr(), block_table.data_ptr(), n, offsets.data_ptr(), _p(parents),
        accepted.data_ptr(), k.data_ptr(), v.data_ptr(), k_idx.data_ptr(), lens_out.data_ptr(),
        _dec._raw_stream(stream, cache._device))
    if st:
        _dsa._check(st, "dsa_cache_commit")


def page_workspace_bytes(dims, cache, batch: int) -> int:
    return int(_dsa._load().dsa_page_workspace_bytes(ctypes.byref(dims), cache._ref, int(batch)))


def alloc_page_workspace(dims, cache, batch: int):
    """Scratch of ``cache_reserve`` and ``cache_compact`` for up to `batch` rows."""
    n = page_workspace_bytes(dims, cache, batch)
    if n == 0:
        _dsa._check(_dec.validate_decode_dims(dims), "dsa_page_workspace_bytes")
        raise _dsa.DSAError(_dsa.DSA_ERR_INVALID_ARG, "dsa_page_workspace_bytes", f"batch {batch}")
    return _dec.torch.empty((n,), dtype=_dec.torch.uint8, device=f"cuda:{cache._device}")


def cache_reserve(dims, cache, refs, lens, new_lens, block_table, missing, ws, stream=None):
    """Pages for rows to grow from lens [batch] to new_lens [batch] int32: free ones, ascending, into block_table, and a
    page of its own, with a copy, for a row whose next token would go to a page that others hold too.  Nothing is changed
    where missing [1] int32 comes back above 0: so many pages are wanting."""
    i32, batch = _dec.torch.int32, lens.numel()
    _check_all("cache_reserve", dims, cache, (
        ("refs", refs, i32, (cache.pages,)), ("lens", lens, i32, (batch,)), ("new_lens", new_lens, i32, (batch,)),
        ("block_table", block_table, i32, (batch, _cols(dims, cache))), ("missing", missing, i32, (1,))), ws)
    pw, nw = _ws(ws)
    st = _dsa._load().dsa_cache_reserve(
        ctypes.byref(dims), cache._ref, refs.data_ptr(), batch, lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
        missing.data_ptr(), pw, nw, _dec._raw_stream(stream, cache._device))
    if st:
        _dsa._check(st, "dsa_cache_reserve")


def cache_fork(dims, cache, refs, lens, block_table, parents, lens_out, table_out, stream=None):
    """Row i of table_out, lens_out shares the pages of row parents[i] ([n_out] int32; -1: an empty row) of block_table, lens."""
    i32, batch, n = _dec.torch.int32, lens.numel(), parents.numel()
    cols = _cols(dims, cache)
    _check_all("cache_fork", dims, cache, (
        ("refs", refs, i32, (cache.pages,)), ("lens", lens, i32, (batch,)), ("block_table", block_table, i32, (batch, cols)),
        ("parents", parents, i32, (n,)), ("lens_out", lens_out, i32, (n,)), ("table_out", table_out, i32, (n, cols))))
    st = _dsa._load().dsa_cache_fork(
        ctypes.byref(dims), cache._ref, refs.data_ptr(), batch, lens.data_ptr(), block_table.data_ptr(), n,
        parents.data_ptr(), lens_out.data_ptr(), table_out.data_ptr(), _dec._raw_stream(stream, cache._device))
    if st:
        _dsa._check(st, "dsa_cache_fork")


def cache_release(dims, cache, refs, lens, block_table, keep=None, stream=None):
    """Rows give back the pages behind their first keep [batch] int32 tokens (None: all of them)."""
    i32, batch = _dec.torch.int32, lens.numel()
    _check_all("cache_release", dims, cache, (
        ("refs", refs, i32, (cache.pages,)), ("lens", lens, i32, (batch,)), ("keep", keep, i32, (batch,)),
        ("block_table", block_table, i32, (batch, _cols(dims, cache)))))
    st = _dsa._load().dsa_cache_release(
        ctypes.byref(dims), cache._ref, refs.data_ptr(), batch, lens.data_ptr(), _p(keep), block_table.data_ptr(),
        _dec._raw_stream(stream, cache._device))
    if st:
        _dsa._check(st, "dsa_cache_release")


def cache_compact(dims, cache, refs, lens, block_table, remap, used, ws, stream=None):
    """The used pages to the front of the cache; the rows' tables follow.  remap [pages] int32: a page's new number, -1 for
    free ones; used [1] int32: how many are in use."""
    i32, batch = _dec.torch.int32, lens.numel()
    _check_all("cache_compact", dims, cache, (
        ("refs", refs, i32, (cache.pages,)), ("lens", lens, i32, (batch,)),
        ("block_table", block_table, i32, (batch, _cols(dims, cache))), ("remap", remap, i32, (cache.pages,)),
        ("used", used, i32, (1,))), ws)
    pw, nw = _ws(ws)
    st = _dsa._load().dsa_cache_compact(
        ctypes.byref(dims), cache._ref, refs.data_ptr(), batch, lens.data_ptr(), block_table.data_ptr(), remap.data_ptr(),
        used.data_ptr(), pw, nw, _dec._raw_stream(stream, cache._device))
    if st:
        _dsa._check(st, "dsa_cache_compact")


def cache_copy_pages(dims, source, target, src, dst, stream=None):
    """Page src[i] of the cache `source` to page dst[i] of `target` (which may be the same), [n] int32."""
    i32, n = _dec.torch.int32, src.numel()
    specs = (("src", src, i32, (n,)), ("dst", dst, i32, (n,)))
    _check_all("cache_copy_pages", dims, source, specs)
    _check_all("cache_copy_pages", dims, target, specs)
    if n == 0:
        return
    st = _dsa._load().dsa_cache_copy_pages(
        ctypes.byref(dims), source._ref, target._ref, n, src.data_ptr(), dst.data_ptr(),
        _dec._raw_stream(stream, source._device))
    if st:
        _dsa._check(st, "dsa_cache_copy_pages")


def _signatures(D):
    P, i64, size = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    C = ctypes.POINTER(_dec._CCache)
    i = ctypes.c_int
    return {
        "dsa_tree_workspace_bytes": ([D, i64, i64], size),
        "dsa_decode_tree_attn": ([D, C, i64, P, P, i64, P, P, P, P, P, P, P, P, P, size, P], i),
        "dsa_cache_commit": ([D, C, i64, P, P, i64, P, P, P, P, P, P, P, P], i),
        "dsa_page_workspace_bytes": ([D, C, i64], size),
        "dsa_cache_reserve": ([D, C, P, i64, P, P, P, P, P, size, P], i),
        "dsa_cache_fork": ([D, C, P, i64, P, P, i64, P, P, P, P], i),
        "dsa_cache_release": ([D, C, P, i64, P, P, P, P], i),
        "dsa_cache_compact": ([D, C, P, i64, P, P, P, P, P, size, P], i),
        "dsa_cache_copy_pages": ([D, C, C, i64, P, P, P], i),
    }
