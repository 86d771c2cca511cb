"""Attention over whole caches in the form that lists all rows' steps and joins the rows that straddle CTAs.

Which form a call takes follows from the batch and the rows' capacity (test_gpu_decode's whole caches of short rows are
mostly of the other form, one cluster per row).  Here the capacity is far above the lengths, and every test asserts that the
list was taken: it makes two launches, the other form one.  References and tolerances are those of test_gpu_decode.
"""
import ctypes

import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from test_gpu_decode import DEV, LENS, Paged, _built, _check_attn, _junk_ws  # noqa: F401

pytestmark = pytest.mark.gpu


def _launches(call):
    """Kernel launches of call(stream), counted in a captured graph that is not run."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    handle, graph, n = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p(), ctypes.c_size_t()
    torch.cuda.synchronize()
    relaxed = 2
    assert cu.cuStreamBeginCapture_v2(handle, relaxed) == 0
    try:
        call(stream)
    finally:
        assert cu.cuStreamEndCapture(handle, ctypes.byref(graph)) == 0
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    assert cu.cuGraphDestroy(graph) == 0
    return n.value


def _whole(pg, Hq, d, launches):
    dims = dsa.make_dims(pg.cap, Hq, d, 8, 64, 8, dtype=pg.dtype)
    B = len(pg.lens_list)
    q = torch.randn(B, Hq, d, generator=pg.g).to(pg.dt)
    lens, table = pg.args()
    o, lse = torch.full((B, Hq, d), 7.0, dtype=pg.dt, device=DEV), torch.full((B, Hq), 7.0, device=DEV)
    cache, ws, qd = pg.cache(), _junk_ws(dims, B), q.to(DEV)
    call = lambda stream=None: dsa.decode_attn(dims, cache, lens, table, qd, o, lse, ws, stream=stream)
    call()
    dsa.check_device_error()
    first = o.clone(), lse.clone()
    assert _launches(call) == launches
    o.fill_(7.0)
    call()
    assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    _check_attn(pg, q, o, lse, d ** -0.5)
    dsa.check_device_error()


VARIANTS = [
    ("bf16", 16, 128, 64), ("bf16", 32, 128, 16), ("bf16", 16, 64, 4), ("bf16", 32, 64, 100), ("bf16", 1, 128, 12),
    ("bf16", 5, 64, 128), ("bf16", 17, 128, 64), ("bf16", 31, 64, 20),
    ("fp32", 8, 64, 16), ("fp32", 8, 128, 64), ("fp32", 16, 128, 12), ("fp32", 16, 64, 20), ("fp32", 32, 128, 64),
    ("fp32", 32, 64, 100), ("fp32", 1, 64, 4), ("fp32", 5, 128, 100)]


@pytest.mark.parametrize("dtype,Hq,d,page", VARIANTS)
def test_list_of_all_lengths(dtype, Hq, d, page):
    _whole(Paged(LENS, page, d=d, dtype=dtype, seed=Hq + d + page, cap=60000).fill(), Hq, d, 2)


@pytest.mark.parametrize("dtype,Hq,d", [("bf16", 16, 128), ("bf16", 32, 128), ("bf16", 32, 64), ("fp32", 8, 64), ("fp32", 8, 128),
                                        ("fp32", 16, 128), ("fp32", 32, 128)])
@pytest.mark.parametrize("batch,most", [(3, 9001), (40, 2001), (129, 613), (150, 301), (700, 97)])
def test_list_of_ragged_batches(dtype, Hq, d, batch, most):
    """Few rows cut into many pieces; rows that begin and end anywhere in a CTA's range; more rows than the cut sums up at
    once (128); more rows than CTAs, so that a CTA has several whole rows and at most one to be joined.  Some idle."""
    lens = [1 + (b * 7919 + 61) % most if b % 9 else 0 for b in range(batch)]
    lens[0] = most
    _whole(Paged(lens, 20, d=d, dtype=dtype, seed=batch + Hq, cap=60000).fill(), Hq, d, 2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[700] * 70, [1] * 600, [0] * 5, [0] * 500, [3001] + [0] * 200, [0] * 200 + [3001]])
def test_list_of_even_rows_and_idle_ones(dtype, lens):
    _whole(Paged(lens, 64, d=64, dtype=dtype, seed=3, cap=60000).fill(), 16, 64, 2)


@pytest.mark.parametrize("dtype,Hq", [("bf16", 16), ("bf16", 32), ("fp32", 8)])
def test_short_capacities_take_one_launch(dtype, Hq):
    """The other side: rows that cannot be long are a cluster each."""
    _whole(Paged([(b * 61) % 300 for b in range(45)], 16, d=64, dtype=dtype, seed=5).fill(), Hq, 64, 1)
