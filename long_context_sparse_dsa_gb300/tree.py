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


# As in decode.py, the calls that a decoder makes for every step check their tensors in one plain condition and look for
# what is wrong only when it fails.


def _check_all(func, dims, cache, specs, ws=None):
    """`specs`: (name, tensor or None, dtype, shape)."""
    dev = cache._device
    ok = _dec._cache_ok(dims, cache, _dec._DTYPES[dims.dtype])
    for _, t, dtype, shape in specs:
        ok = ok and (t is None or t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous())
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
    torch, dev, batch, n, d = _dec.torch, cache._device, lens.numel(), q.shape[0], dims.d
    i32, dt, heads, cols = torch.int32, _dec._DTYPES[dims.dtype], (n, dims.Hq, d), -(-dims.L // cache.page_size)
    if not (_dec._cache_ok(dims, cache, dt) and
            lens.dtype is i32 and lens.shape == (batch,) and lens.get_device() == dev and lens.is_contiguous() and
            block_table.dtype is i32 and block_table.shape == (batch, cols) and block_table.get_device() == dev and
            block_table.is_contiguous() and
            offsets.dtype is i32 and offsets.shape == (batch + 1,) and offsets.get_device() == dev and
            offsets.is_contiguous() and
            (parents is None or parents.dtype is i32 and parents.shape == (n,) and parents.get_device() == dev and
             parents.is_contiguous()) and
            (idx is None or idx.dtype is i32 and idx.shape == (n, dims.k) and idx.get_device() == dev and
             idx.is_contiguous()) and
            q.dtype is dt and q.shape == heads and q.get_device() == dev and q.is_contiguous() and
            k.dtype is dt and k.shape == (n, d) and k.get_device() == dev and k.is_contiguous() and
            v.dtype is dt and v.shape == (n, d) and v.get_device() == dev and v.is_contiguous() and
            o.dtype is dt and o.shape == heads and o.get_device() == dev and o.is_contiguous() and
            lse.dtype is torch.float32 and lse.shape == heads[:2] and lse.get_device() == dev and lse.is_contiguous() and
            (ws is None or ws.get_device() == dev and ws.is_contiguous())):
        _dec._refuse("decode_tree_attn", dims, cache, ("lens", lens, i32, (batch,)), ("block_table", block_table, i32, (batch, cols)),
                     ("offsets", offsets, i32, (batch + 1,)), ("parents", parents, i32, (n,)), ("idx", idx, i32, (n, dims.k)),
                     ("q", q, dt, heads), ("k", k, dt, (n, d)), ("v", v, dt, (n, d)), ("o", o, dt, heads),
                     ("lse", lse, torch.float32, heads[:2]), ("ws", ws, None, None))
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
    i32, dev, batch, n, d = _dec.torch.int32, cache._device, lens.numel(), k.shape[0], dims.d
    dt, cols = _dec._DTYPES[dims.dtype], -(-dims.L // cache.page_size)
    if not (_dec._cache_ok(dims, cache, dt) and
            lens.dtype is i32 and lens.shape == (batch,) and lens.get_device() == dev and lens.is_contiguous() and
            block_table.dtype is i32 and block_table.shape == (batch, cols) and block_table.get_device() == dev and
            block_table.is_contiguous() and
            offsets.dtype is i32 and offsets.shape == (batch + 1,) and offsets.get_device() == dev and
            offsets.is_contiguous() and
            (parents is None or parents.dtype is i32 and parents.shape == (n,) and parents.get_device() == dev and
             parents.is_contiguous()) and
            accepted.dtype is i32 and accepted.shape == (batch,) and accepted.get_device() == dev and
            accepted.is_contiguous() and
            k.dtype is dt and k.shape == (n, d) and k.get_device() == dev and k.is_contiguous() and
            v.dtype is dt and v.shape == (n, d) and v.get_device() == dev and v.is_contiguous() and
            k_idx.dtype is dt and k_idx.shape == (n, dims.di) and k_idx.get_device() == dev and k_idx.is_contiguous() and
            lens_out.dtype is i32 and lens_out.shape == (batch,) and lens_out.get_device() == dev and
            lens_out.is_contiguous()):
        _dec._refuse("cache_commit", dims, cache, ("lens", lens, i32, (batch,)), ("block_table", block_table, i32, (batch, cols)),
                     ("offsets", offsets, i32, (batch + 1,)), ("parents", parents, i32, (n,)),
                     ("accepted", accepted, i32, (batch,)), ("k", k, dt, (n, d)), ("v", v, dt, (n, d)),
                     ("k_idx", k_idx, dt, (n, dims.di)), ("lens_out", lens_out, i32, (batch,)))
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
    where missing [1] int32 comes back above 0: so many pages are wanting.  Room that a row did not use is given back before
    the next reserve: ``cache_release`` with lens = the reserved lengths, keep = the rows' own."""
    i32, dev, batch, cols = _dec.torch.int32, cache._device, lens.numel(), -(-dims.L // cache.page_size)
    if not (_dec._cache_ok(dims, cache, _dec._DTYPES[dims.dtype]) and
            refs.dtype is i32 and refs.shape == (cache.pages,) and refs.get_device() == dev and refs.is_contiguous() and
            lens.dtype is i32 and lens.shape == (batch,) and lens.get_device() == dev and lens.is_contiguous() and
            new_lens.dtype is i32 and new_lens.shape == (batch,) and new_lens.get_device() == dev and
            new_lens.is_contiguous() and
            block_table.dtype is i32 and block_table.shape == (batch, cols) and block_table.get_device() == dev and
            block_table.is_contiguous() and
            missing.dtype is i32 and missing.shape == (1,) and missing.get_device() == dev and
            (ws is None or ws.get_device() == dev and ws.is_contiguous())):
        _dec._refuse("cache_reserve", dims, cache, ("refs", refs, i32, (cache.pages,)), ("lens", lens, i32, (batch,)),
                     ("new_lens", new_lens, i32, (batch,)), ("block_table", block_table, i32, (batch, cols)),
                     ("missing", missing, i32, (1,)), ("ws", ws, None, None))
    pw, nw = _ws(ws)
    st = _dsa._load().dsa_cache_reserve(
        ctypes.byref(dims), cache._ref, refs.data_ptr(), batch, lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
        missing.data_ptr(), pw, nw, _dec._raw_stream(stream, cache._device))
    if st:
        _dsa._check(st, "dsa_cache_reserve")


def cache_fork(dims, cache, refs, lens, block_table, parents, lens_out, table_out, stream=None):
    """Row i of table_out, lens_out shares the pages of row parents[i] ([n_out] int32; -1: an empty row) of block_table, lens."""
    i32, dev, batch, n = _dec.torch.int32, cache._device, lens.numel(), parents.numel()
    cols = -(-dims.L // cache.page_size)
    if not (_dec._cache_ok(dims, cache, _dec._DTYPES[dims.dtype]) and
            refs.dtype is i32 and refs.shape == (cache.pages,) and refs.get_device() == dev and refs.is_contiguous() and
            lens.dtype is i32 and lens.shape == (batch,) and lens.get_device() == dev and lens.is_contiguous() and
            block_table.dtype is i32 and block_table.shape == (batch, cols) and block_table.get_device() == dev and
            block_table.is_contiguous() and
            parents.dtype is i32 and parents.shape == (n,) and parents.get_device() == dev and parents.is_contiguous() and
            lens_out.dtype is i32 and lens_out.shape == (n,) and lens_out.get_device() == dev and lens_out.is_contiguous() and
            table_out.dtype is i32 and table_out.shape == (n, cols) and table_out.get_device() == dev and
            table_out.is_contiguous()):
        _dec._refuse("cache_fork", dims, cache, ("refs", refs, i32, (cache.pages,)), ("lens", lens, i32, (batch,)),
                     ("block_table", block_table, i32, (batch, cols)), ("parents", parents, i32, (n,)),
                     ("lens_out", lens_out, i32, (n,)), ("table_out", table_out, i32, (n, cols)))
    st = _dsa._load().dsa_cache_fork(
        ctypes.byref(dims), cache._ref, refs.data_ptr(), batch, lens.data_ptr(), block_table.data_ptr(), n,
        parents.data_ptr(), lens_out.data_ptr(), table_out.data_ptr(), _dec._raw_stream(stream, cache._device))
    if st:
        _dsa._check(st, "dsa_cache_fork")


def cache_release(dims, cache, refs, lens, block_table, keep=None, stream=None):
    """Rows give back the pages behind their first keep [batch] int32 tokens (None: all of them).  lens: the rows' lengths or,
    of rows with room that is not used, the reserved ones."""
    i32, dev, batch, cols = _dec.torch.int32, cache._device, lens.numel(), -(-dims.L // cache.page_size)
    if not (_dec._cache_ok(dims, cache, _dec._DTYPES[dims.dtype]) and
            refs.dtype is i32 and refs.shape == (cache.pages,) and refs.get_device() == dev and refs.is_contiguous() and
            lens.dtype is i32 and lens.shape == (batch,) and lens.get_device() == dev and lens.is_contiguous() and
            (keep is None or keep.dtype is i32 and keep.shape == (batch,) and keep.get_device() == dev and
             keep.is_contiguous()) and
            block_table.dtype is i32 and block_table.shape == (batch, cols) and block_table.get_device() == dev and
            block_table.is_contiguous()):
        _dec._refuse("cache_release", dims, cache, ("refs", refs, i32, (cache.pages,)), ("lens", lens, i32, (batch,)),
                     ("keep", keep, i32, (batch,)), ("block_table", block_table, i32, (batch, cols)))
    st = _dsa._load().dsa_cache_release(
        ctypes.byref(dims), cache._ref, refs.data_ptr(), batch, lens.data_ptr(), _p(keep), block_table.data_ptr(),
        _dec._raw_stream(stream, cache._device))
    if st:
        _dsa._check(st, "dsa_cache_release")


def cache_compact(dims, cache, refs, lens, block_table, remap, used, ws, stream=None):
    """The used pages to the front of the cache; the rows' tables follow, as far as lens (reserved lengths, where rows have room
    that is not used).  remap [pages] int32: a page's new number, -1 for free ones; used [1] int32: how many are in use."""
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
