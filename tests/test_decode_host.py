"""Host-only checks of the paged decode calls: what they refuse before any launch (no call below reaches a GPU),
the workspace sizes, the rotation's integer angles and the kernels' page division."""
import ctypes
import math
import random
from fractions import Fraction

import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from long_context_sparse_dsa_gb300 import build as dsa_build
from long_context_sparse_dsa_gb300 import decode


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.library()


def _dims(**kw):
    base = dict(L=4096, Hq=16, d=128, Hi=8, di=64, k=512, dtype="bf16")
    base.update(kw)
    return dsa.make_dims(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(), dsa.DSA_OK),
    (dict(Hq=1, Hi=1), dsa.DSA_OK),              # any head count the tiles hold, unlike the training kernels
    (dict(Hq=5, Hi=3, dtype="fp32"), dsa.DSA_OK),
    (dict(L=4094), dsa.DSA_ERR_INVALID_ARG),
    (dict(L=0), dsa.DSA_ERR_INVALID_ARG),
    (dict(L=1 << 31), dsa.DSA_ERR_UNSUPPORTED),
    (dict(k=0), dsa.DSA_ERR_INVALID_ARG),
    (dict(k=1025), dsa.DSA_ERR_UNSUPPORTED),
    (dict(scale=0.0), dsa.DSA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), dsa.DSA_ERR_INVALID_ARG),
    (dict(d=96), dsa.DSA_ERR_UNSUPPORTED),
    (dict(di=32), dsa.DSA_ERR_UNSUPPORTED),
    (dict(Hq=33), dsa.DSA_ERR_UNSUPPORTED),
    (dict(Hq=0), dsa.DSA_ERR_UNSUPPORTED),
    (dict(Hi=9), dsa.DSA_ERR_UNSUPPORTED),
    (dict(pool=8), dsa.DSA_ERR_UNSUPPORTED),
])
def test_validate_decode_dims(lib, kw, status):
    assert dsa.validate_decode_dims(_dims(**kw)) == status
    assert (dsa.decode_workspace_bytes(_dims(**kw), 3) > 0) == (status == dsa.DSA_OK)


def test_workspace_bytes(lib):
    d = _dims()
    assert dsa.decode_workspace_bytes(d, 0) == 0 and dsa.decode_workspace_bytes(d, 1 << 16) == 0
    # the score block of a long row, and the rotated queries, fit
    big = _dims(L=1 << 20)
    assert dsa.decode_workspace_bytes(big, 7) >= 7 * (1 << 18) * 4 + 7 * 16 * 128 * 2


def _cache(**kw):
    base = dict(k=256, v=256, kpool=256, ktail=256, num_pages=10, page_size=64)
    base.update(kw)
    return decode._CCache(*(base[n] for n, _ in decode._CCache._fields_))


P, ODD = ctypes.c_void_p(256), ctypes.c_void_p(264)
BIG = 1 << 40


def _append(lib, d=None, c=None, batch=2, n=2, rot=None, **kw):
    a = dict(lens=P, table=P, offsets=None, k=P, v=P, k_idx=P, q=None, q_out=None, k_out=None)
    a.update(kw)
    return lib.dsa_cache_append(ctypes.byref(d or _dims()), ctypes.byref(c or _cache()), batch, a["lens"], a["table"], n,
                                a["offsets"], a["k"], a["v"], a["k_idx"], None if rot is None else ctypes.byref(rot),
                                a["q"], a["q_out"], a["k_out"], None)


def _topk(lib, d=None, c=None, batch=2, size=BIG, **kw):
    a = dict(lens=P, table=P, q_idx=P, w=P, idx=P, ws=P)
    a.update(kw)
    return lib.dsa_decode_indexer_topk(ctypes.byref(d or _dims()), ctypes.byref(c or _cache()), batch, a["lens"], a["table"],
                                       a["q_idx"], a["w"], a["idx"], a["ws"], size, None)


def _attn(lib, d=None, c=None, batch=2, size=BIG, **kw):
    a = dict(lens=P, table=P, idx=P, q=P, o=P, lse=P, ws=P)
    a.update(kw)
    return lib.dsa_decode_attn(ctypes.byref(d or _dims()), ctypes.byref(c or _cache()), batch, a["lens"], a["table"], a["idx"],
                               a["q"], a["o"], a["lse"], a["ws"], size, None)


def _step(lib, d=None, c=None, batch=2, size=BIG, rot=None, **kw):
    a = dict(lens=P, table=P, q=P, k=P, v=P, q_idx=P, k_idx=P, w=P, o=P, lse=P, idx=P, ws=P)
    a.update(kw)
    return lib.dsa_decode_step(ctypes.byref(d or _dims()), ctypes.byref(c or _cache()), batch, a["lens"], a["table"], a["q"],
                               a["k"], a["v"], a["q_idx"], a["k_idx"], a["w"], None if rot is None else ctypes.byref(rot),
                               a["o"], a["lse"], a["idx"], a["ws"], size, None)


CALLS = {
    "append": (_append, ["lens", "table", "k", "v", "k_idx"], ["k", "v", "kpool", "ktail"]),
    "topk": (_topk, ["lens", "table", "q_idx", "w", "idx"], ["kpool"]),
    "attn": (_attn, ["lens", "table", "q", "o", "lse"], ["k", "v"]),
    "step": (_step, ["lens", "table", "q", "k", "v", "q_idx", "k_idx", "w", "o", "lse", "idx"],
             ["k", "v", "kpool", "ktail"]),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_arguments_are_refused_before_any_launch(lib, name):
    call, ptrs, arrays = CALLS[name]
    for p in ptrs:
        assert call(lib, **{p: None}) == dsa.DSA_ERR_INVALID_ARG, p
        assert b"NULL" in lib.dsa_last_error_message()
        assert call(lib, **{p: ODD}) == dsa.DSA_ERR_INVALID_ARG, p
        assert b"aligned" in lib.dsa_last_error_message()
    for p in arrays:
        assert call(lib, c=_cache(**{p: None})) == dsa.DSA_ERR_INVALID_ARG, p
        assert b"cache->" in lib.dsa_last_error_message()
        assert call(lib, c=_cache(**{p: 264})) == dsa.DSA_ERR_INVALID_ARG, p
    for bad in (dict(page_size=0), dict(page_size=6), dict(page_size=-4), dict(num_pages=0)):
        assert call(lib, c=_cache(**bad)) == dsa.DSA_ERR_INVALID_ARG, bad
    assert call(lib, c=_cache(num_pages=(1 << 25) + 1)) == dsa.DSA_ERR_UNSUPPORTED     # more than 2^31 tokens
    assert call(lib, d=_dims(d=96)) == dsa.DSA_ERR_UNSUPPORTED
    assert call(lib, batch=0, **({"n": 0} if name == "append" else {})) == dsa.DSA_ERR_INVALID_ARG
    assert call(lib, batch=1 << 16, **({"n": 1 << 16} if name == "append" else {})) == dsa.DSA_ERR_UNSUPPORTED
    if name != "append":
        need = dsa.decode_workspace_bytes(_dims(), 2)
        assert call(lib, ws=None) == dsa.DSA_ERR_WORKSPACE
        assert call(lib, size=need - 1) == dsa.DSA_ERR_WORKSPACE
        assert call(lib, ws=ODD) == dsa.DSA_ERR_INVALID_ARG


def test_append_refusals(lib):
    rot = decode._CRotation(256, 64, 0)
    assert _append(lib, n=3) == dsa.DSA_ERR_INVALID_ARG            # one token per row without offsets
    assert _append(lib, n=-1, offsets=P) == dsa.DSA_ERR_INVALID_ARG
    assert _append(lib, n=3, offsets=ODD) == dsa.DSA_ERR_INVALID_ARG
    assert _append(lib, q=P, rot=rot) == dsa.DSA_ERR_INVALID_ARG   # q without q_out
    assert _append(lib, q_out=P, rot=rot) == dsa.DSA_ERR_INVALID_ARG
    assert _append(lib, q=P, q_out=P) == dsa.DSA_ERR_INVALID_ARG   # without a rotation
    assert _append(lib, k_out=P) == dsa.DSA_ERR_INVALID_ARG
    assert _append(lib, q=P, q_out=ODD, rot=rot) == dsa.DSA_ERR_INVALID_ARG
    assert _append(lib, k_out=ODD, rot=rot) == dsa.DSA_ERR_INVALID_ARG
    for turns, dim in ((None, 64), (264, 64), (256, 0), (256, 24), (256, 144), (256, -16)):
        assert _append(lib, rot=decode._CRotation(turns, dim, 0)) == dsa.DSA_ERR_INVALID_ARG, (turns, dim)
        assert _step(lib, rot=decode._CRotation(turns, dim, 0)) == dsa.DSA_ERR_INVALID_ARG, (turns, dim)
    # no new tokens: nothing to do, and the token tensors may be empty
    assert _append(lib, n=0, offsets=P, k=None, v=None, k_idx=None) == dsa.DSA_OK


def test_attn_optional_selection(lib):
    assert _attn(lib, idx=ODD) == dsa.DSA_ERR_INVALID_ARG


def test_cache_handle_refusals():
    with pytest.raises(ValueError):
        dsa.PagedCache()
    with pytest.raises(ValueError):       # a CPU tensor
        dsa.PagedCache(k=torch.zeros(2, 16, 64), v=torch.zeros(2, 16, 64))
    with pytest.raises(ValueError):
        dsa.make_rotation([0.1] * 7, device="cpu")
    with pytest.raises(ValueError):
        dsa.make_rotation([0.1] * 7 + [math.inf], device="cpu")


def test_rotation_turns_are_exact_fractions():
    """turns / 2^64 is freq / 2 pi modulo 1 to the double's own rounding; negative frequencies turn backwards, and the
    64-bit product of a position wraps to the angle's fraction."""
    freq = [10000.0 ** (-i / 8) for i in range(8)] + [-0.25, 7.0, 1e-9, 2 * math.pi, 0.0, 1.0, -1.0, 3.5]
    r = dsa.make_rotation(freq, device="cpu")
    assert r.dim == 32
    for f, t in zip(freq, r.turns.tolist()):
        t %= 1 << 64
        want = Fraction(f / (2 * math.pi)) % 1
        assert abs(Fraction(t, 1 << 64) - want) % 1 in (0, 1) or \
            min(abs(Fraction(t, 1 << 64) - want) % 1, 1 - abs(Fraction(t, 1 << 64) - want) % 1) <= Fraction(1, 1 << 52)
        for pos in (0, 1, 131071, (1 << 20) + 7, (1 << 31) - 4):
            a = 2 * math.pi * ((pos * t % (1 << 64)) / 2.0 ** 64)
            err = abs(math.remainder(a - math.fmod(pos * f, 2 * math.pi), 2 * math.pi))
            # the fraction's rounding times the position, the double product's rounding, and the final few operations
            assert err <= pos * 2.0 ** -50 + abs(pos * f) * 2.0 ** -52 + 1e-14


def test_page_division_is_exact():
    """The multiplier and shift of decode.h divide every pool index below 2^29 by any pools-per-page."""
    rng = random.Random(5)
    for ppp in list(range(1, 70)) + [100, 255, 256, 257, 1000, 4096, 65537, (1 << 28) - 1, 1 << 28, (1 << 29) - 1]:
        s = 0
        while (1 << s) < ppp:
            s += 1
        mul, shift = (1 << (29 + s)) // ppp + 1, 29 + s
        assert mul < 1 << 32
        ps = [0, 1, (1 << 29) - 1, (1 << 29) - 2] + [rng.randrange(1 << 29) for _ in range(200)]
        for q in [rng.randrange((1 << 29) // ppp + 1) for _ in range(200)]:
            ps += [q * ppp, q * ppp - 1, q * ppp + 1]
        for p in ps:
            if 0 <= p < 1 << 29:
                assert p * mul < 1 << 64 and (p * mul) >> shift == p // ppp, (p, ppp)
