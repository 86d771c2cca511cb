"""Host-only checks of the draft tree, page and head calls: what they refuse before any launch (no call below reaches a GPU),
and their workspace sizes."""
import ctypes

import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from long_context_sparse_dsa_gb300 import build as dsa_build
from long_context_sparse_dsa_gb300 import decode

P, ODD, BIG = ctypes.c_void_p(256), ctypes.c_void_p(264), 1 << 40
INV, UNS, WS = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.library()


def _dims(**kw):
    return dsa.make_dims(**{**dict(L=4096, Hq=16, d=128, Hi=8, di=64, k=512, dtype="bf16"), **kw})


def _cache(**kw):
    base = {**dict(k=256, v=256, kpool=256, ktail=256, num_pages=10, page_size=64), **kw}
    return decode._CCache(*(base[n] for n, _ in decode._CCache._fields_))


def _tree(lib, d=None, c=None, batch=2, n=5, size=BIG, **kw):
    a = dict(lens=P, table=P, offsets=P, parents=P, idx=P, q=P, k=P, v=P, o=P, lse=P, ws=P)
    a.update(kw)
    return lib.dsa_decode_tree_attn(ctypes.byref(d or _dims()), ctypes.byref(c or _cache()), batch, a["lens"], a["table"], n,
                                    a["offsets"], a["parents"], a["idx"], a["q"], a["k"], a["v"], a["o"], a["lse"], a["ws"],
                                    size, None)


def _commit(lib, d=None, c=None, batch=2, n=5, **kw):
    a = dict(lens=P, table=P, offsets=P, parents=P, accepted=P, k=P, v=P, k_idx=P, lens_out=P)
    a.update(kw)
    return lib.dsa_cache_commit(ctypes.byref(d or _dims()), ctypes.byref(c or _cache()), batch, a["lens"], a["table"], n,
                                a["offsets"], a["parents"], a["accepted"], a["k"], a["v"], a["k_idx"], a["lens_out"], None)


BAD_COMMON = [(dict(batch=0), INV), (dict(batch=1 << 16), UNS), (dict(lens=None), INV), (dict(table=ODD), INV), (dict(d=_dims(d=96)), UNS),
              (dict(c=_cache(page_size=6)), INV), (dict(c=_cache(num_pages=0)), INV), (dict(c=_cache(num_pages=1 << 31)), UNS)]


@pytest.mark.parametrize("kw,status", BAD_COMMON + [
    (dict(n=-1), INV), (dict(n=(1 << 24) + 1), INV), (dict(offsets=None), INV), (dict(offsets=ODD), INV), (dict(parents=ODD), INV),
    (dict(idx=ODD), INV), (dict(q=None), INV), (dict(k=ODD), INV), (dict(v=None), INV), (dict(o=ODD), INV), (dict(lse=None), INV),
    (dict(ws=None), WS), (dict(size=100), WS), (dict(ws=ODD), INV), (dict(c=_cache(v=None)), INV), (dict(c=_cache(k=264)), INV)])
def test_tree_attn_refuses(lib, kw, status):
    assert _tree(lib, **kw) == status


def test_tree_attn_of_no_nodes_launches_nothing(lib):
    assert _tree(lib, n=0, q=None, k=None, v=None, o=None, lse=None, ws=None, size=0) == dsa.DSA_OK


@pytest.mark.parametrize("kw,status", BAD_COMMON + [
    (dict(n=-1), INV), (dict(offsets=None), INV), (dict(parents=ODD), INV), (dict(accepted=None), INV), (dict(k=None), INV),
    (dict(v=ODD), INV), (dict(k_idx=None), INV), (dict(lens_out=ODD), INV), (dict(lens_out=None), INV),
    (dict(c=_cache(kpool=None)), INV), (dict(c=_cache(ktail=264)), INV)])
def test_commit_refuses(lib, kw, status):
    assert _commit(lib, **kw) == status


def test_workspaces(lib):
    d = _dims()
    assert dsa.tree_workspace_bytes(d, 2, 0) > 0 and dsa.tree_workspace_bytes(d, 0, 5) == 0 and dsa.tree_workspace_bytes(d, 2, -1) == 0
    assert dsa.tree_workspace_bytes(d, 2, 1000) >= 32 * 1000 and dsa.tree_workspace_bytes(d, 2, (1 << 24) + 1) == 0
    n = lambda c, b=3, d=d: lib.dsa_page_workspace_bytes(ctypes.byref(d), ctypes.byref(c), b)  # noqa: E731
    assert n(_cache(num_pages=100000)) >= 800000 and n(_cache(), b=65535) >= 16 * 65535
    assert n(_cache(page_size=2)) == n(_cache(num_pages=0)) == n(_cache(), b=0) == n(_cache(), d=_dims(di=32)) == 0
    assert dsa.qk_norm_bwd_workspace_bytes(d, 5) > 0 and dsa.qk_norm_bwd_workspace_bytes(d, -1) == 0
    assert dsa.qk_norm_bwd_workspace_bytes(_dims(Hq=33), 5) == 0


@pytest.mark.parametrize("kw,status", BAD_COMMON + [
    (dict(refs=None), INV), (dict(new=ODD), INV), (dict(new=None), INV), (dict(missing=None), INV), (dict(ws=None), WS), (dict(size=64), WS),
    (dict(ws=ODD), INV), (dict(c=_cache(v=None)), INV), (dict(c=_cache(k=None, v=None, kpool=None)), INV),
    (dict(c=_cache(k=None, v=None, kpool=None, ktail=None)), INV), (dict(c=_cache(kpool=264)), INV),
    (dict(c=_cache(page_size=1 << 21, num_pages=4)), UNS)])
def test_reserve_and_compact_refuse(lib, kw, status):
    a = {**dict(d=_dims(), c=_cache(), batch=2, refs=P, lens=P, new=P, table=P, missing=P, ws=P, size=BIG), **kw}
    head = (ctypes.byref(a["d"]), ctypes.byref(a["c"]), a["refs"], a["batch"], a["lens"])
    assert lib.dsa_cache_reserve(*head, a["new"], a["table"], a["missing"], a["ws"], a["size"], None) == status
    assert lib.dsa_cache_compact(*head, a["table"], a["new"], a["missing"], a["ws"], a["size"], None) == status


@pytest.mark.parametrize("kw,status", BAD_COMMON + [(dict(refs=ODD), INV), (dict(extra=ODD), INV)])
def test_fork_and_release_refuse(lib, kw, status):
    a = {**dict(d=_dims(), c=_cache(), batch=2, refs=P, lens=P, table=P, extra=P), **kw}
    head = (ctypes.byref(a["d"]), ctypes.byref(a["c"]), a["refs"], a["batch"], a["lens"])
    Q = ctypes.c_void_p(512)
    assert lib.dsa_cache_fork(*head, a["table"], 3, a["extra"], Q, Q, None) == status
    assert lib.dsa_cache_release(*head, a["extra"], a["table"], None) == status


def test_fork_refuses_the_old_rows_as_new_ones(lib):
    head = (ctypes.byref(_dims()), ctypes.byref(_cache()), P, 2, P, P)
    Q = ctypes.c_void_p(512)
    assert lib.dsa_cache_fork(*head, 3, P, P, Q, None) == INV and lib.dsa_cache_fork(*head, 3, P, Q, P, None) == INV
    assert lib.dsa_cache_fork(*head, 0, P, Q, Q, None) == INV and lib.dsa_cache_fork(*head, 1 << 16, P, Q, Q, None) == UNS
    assert lib.dsa_cache_fork(*head, 3, None, Q, Q, None) == INV and lib.dsa_cache_fork(*head, 3, P, None, Q, None) == INV


@pytest.mark.parametrize("to,n,src,status", [
    (_cache(page_size=32), 1, P, INV), (_cache(k=None, v=None), 1, P, INV), (_cache(ktail=None), 1, P, INV), (_cache(), -1, P, INV),
    (_cache(), 1 << 31, P, INV), (_cache(), 1, None, INV), (_cache(), 1, ODD, INV), (_cache(num_pages=0), 1, P, INV)])
def test_copy_pages_refuses(lib, to, n, src, status):
    assert lib.dsa_cache_copy_pages(ctypes.byref(_dims()), ctypes.byref(_cache()), ctypes.byref(to), n, src, P, None) == status


def test_copy_pages_names_what_it_refuses(lib):
    ref = ctypes.byref(_cache())
    for src, dst, name in ((None, P, "src is NULL"), (P, ODD, "dst is not 16-byte aligned")):
        assert lib.dsa_cache_copy_pages(ctypes.byref(_dims()), ref, ref, 1, src, dst, None) == INV
        with pytest.raises(dsa.DSAError, match=name):
            dsa._check(INV, "dsa_cache_copy_pages")


def _norm(lib, **kw):
    a = {**dict(d=_dims(), n=3, q=P, qs=2048, k=P, ks=128, qw=P, kw=P, eps=1e-6, rot=None, pos=P, qo=P, ko=P), **kw}
    return lib.dsa_qk_norm_rotate(ctypes.byref(a["d"]), a["n"], a["q"], a["qs"], a["k"], a["ks"], a["qw"], a["kw"], a["eps"],
                                  None if a["rot"] is None else ctypes.byref(a["rot"]), a["pos"], a["qo"], a["ko"], None)


def _norm_bwd(lib, **kw):
    a = {**dict(d=_dims(), n=3, q=P, qs=2048, k=P, ks=128, qw=P, kw=P, eps=1e-6, rot=None, pos=P, dqo=P, dko=P, dq=P, dk=P,
                dqw=P, dkw=P, ws=P, size=BIG), **kw}
    return lib.dsa_qk_norm_rotate_bwd(ctypes.byref(a["d"]), a["n"], a["q"], a["qs"], a["k"], a["ks"], a["qw"], a["kw"], a["eps"],
                                      None if a["rot"] is None else ctypes.byref(a["rot"]), a["pos"], a["dqo"], a["dko"], a["dq"],
                                      a["dk"], a["dqw"], a["dkw"], a["ws"], a["size"], None)


HEADS = [(dict(d=_dims(Hq=33)), UNS), (dict(n=-1), INV), (dict(n=1 << 31), INV), (dict(q=ODD), INV), (dict(k=ODD), INV), (dict(qs=2040), INV),
         (dict(qs=2052), INV), (dict(ks=64), INV), (dict(ks=132), INV), (dict(qw=ODD), INV), (dict(kw=ODD), INV), (dict(eps=0.0), INV),
         (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(pos=ODD), INV), (dict(q=None), INV), (dict(k=None), INV),
         (dict(rot=decode._CRotation(256, 144, 0)), INV), (dict(rot=decode._CRotation(256, 8, 0)), INV),
         (dict(rot=decode._CRotation(None, 16, 0)), INV)]


@pytest.mark.parametrize("kw,status", HEADS + [
    (dict(qo=None), INV), (dict(ko=ODD), INV), (dict(q=None, qo=None, k=None, ko=None), INV),
    (dict(qs=2176, qo=P), INV), (dict(ks=256, ko=P), INV)])     # in place, but not contiguous
def test_norm_refuses(lib, kw, status):
    Q = ctypes.c_void_p(1 << 20)
    assert _norm(lib, **{**dict(qo=Q, ko=Q), **kw}) == status


@pytest.mark.parametrize("kw,status", HEADS + [
    (dict(dqo=None), INV), (dict(dk=None), INV), (dict(dq=ODD), INV), (dict(dkw=ODD), INV), (dict(ws=None), WS), (dict(size=8), WS),
    (dict(ws=ODD), INV), (dict(q=None, dqo=None, dq=None), INV)])     # a weight's gradient without its heads
def test_norm_gradient_refuses(lib, kw, status):
    assert _norm_bwd(lib, **kw) == status


def test_bindings_refuse_what_they_cannot_pass_on():
    """Tensors on the CPU stand in for any that are not as the calls want them."""
    d = _dims(L=64, Hq=4)
    z = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError)):
        dsa.qk_norm_rotate(d, z, z[:, 0].contiguous(), z, z[:, 0].contiguous(), 1e-6)
    with pytest.raises(ValueError):
        dsa.qk_norm_rotate(d, None, None, None, None, 1e-6)
