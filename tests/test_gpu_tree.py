"""Attention of draft trees over the paged cache, and the accepted path's way into it, against plain forms in 64 bits.

Caches start full of NaN, and so do workspaces.  Tolerances are those of test_gpu_decode (_check_attn): the same sums over
the same kinds of products, two bf16 terms of the weights.  What enters the cache is compared bit for bit with
cache_append's.
"""
import math
import random

import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from test_gpu_decode import DEV, HALF, Paged, _built, _freq  # noqa: F401
from test_gpu_decode_contract import _reports

pytestmark = pytest.mark.gpu


class Trees:
    """A random tree of the given number of nodes behind each row of a Paged."""

    def __init__(self, pg, nodes, Hq, chain=False, seed=0, wide=4):
        r, g = random.Random(seed), torch.Generator().manual_seed(seed)
        self.pg, self.nodes, self.Hq, self.chain = pg, nodes, Hq, chain
        self.off = [sum(nodes[:b]) for b in range(len(nodes) + 1)]
        self.up = [[i - 1 if chain else r.randint(max(-1, i - wide), i - 1) for i in range(n)] for n in nodes]
        d, di, T = pg.K[0].shape[1], pg.KI[0].shape[1], sum(nodes)
        draw = lambda *s: torch.randn(*s, generator=g).to(pg.dt)  # noqa: E731
        self.q, self.k, self.v = draw(T, Hq, d), draw(T, d), draw(T, d)
        self.ki = torch.randint(-3, 4, (T, di), generator=g).to(pg.dt)

    def line(self, b, i):
        """Node i's ancestors and itself, from the root on, as rows of the node tensors."""
        out = []
        while i >= 0:
            out.insert(0, self.off[b] + i)
            i = self.up[b][i]
        return out

    def args(self):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        parents = None if self.chain else i32([p for row in self.up for p in row])
        return i32(self.off), parents


def _dims(pg, Hq, k=8):
    return dsa.make_dims(pg.cap, Hq, pg.K[0].shape[1], 8, pg.KI[0].shape[1], k, dtype=pg.dtype)


def _ws(dims, B, T):
    return torch.full((dsa.tree_workspace_bytes(dims, B, T),), 0xFF, dtype=torch.uint8, device=DEV)


def _run(pg, tr, dims, idx=None, **kw):
    T, Hq, d = tr.q.shape
    lens, table = pg.args()
    off, parents = tr.args()
    o, lse = torch.full((T, Hq, d), 7.0, dtype=pg.dt, device=DEV), torch.full((T, Hq), 7.0, device=DEV)
    dsa.decode_tree_attn(dims, kw.get("cache") or pg.cache(), lens, table, off, parents, tr.q.to(DEV), tr.k.to(DEV), tr.v.to(DEV),
                         o, lse, _ws(dims, len(pg.lens_list), T), idx=None if idx is None else idx.to(DEV))
    return o, lse


def _check(pg, tr, o, lse, scale, idx=None, rows=None, nodes=None):
    d, u = tr.q.shape[2], HALF[pg.dtype]
    o, lse = o.double().cpu(), lse.double().cpu()
    for b in range(len(tr.nodes)) if rows is None else rows:
        for i in range(tr.nodes[b]) if nodes is None else nodes:
            t, line = tr.off[b] + i, tr.line(b, i)
            at = pg.keys(b, None if idx is None else {b: idx[t]})
            k = torch.cat([pg.K[b][at], tr.k[line]]).double()
            v = torch.cat([pg.V[b][at], tr.v[line]]).double()
            qq = tr.q[t].double()
            s = qq @ k.T * scale
            ref_l = torch.logsumexp(s, -1)
            p = (s - ref_l[:, None]).exp()
            ref = p @ v
            ds = (d + 4) * 2.0 ** -23 * scale * (qq.abs() @ k.abs().T).amax(-1)
            n = len(k)
            tol = (4 * ds[:, None] + 2.0 ** -18 + n * 2.0 ** -23) * (p @ v.abs()) + u * ref.abs()
            if pg.dtype == "bf16":
                tol += 2.0 ** -16 * (p @ v.abs())
            assert torch.all((o[t] - ref).abs() <= tol), (b, i, ((o[t] - ref).abs() / tol).max())
            ltol = 2 * ds + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * ref_l.abs()
            assert torch.all((lse[t] - ref_l).abs() <= ltol), (b, i, ((lse[t] - ref_l).abs() / ltol).max())


def _selection(pg, tr, k, seed=3):
    g = torch.Generator().manual_seed(seed)
    idx = torch.full((sum(tr.nodes), k), -1, dtype=torch.int32)
    for b, n in enumerate(tr.nodes):
        for i in range(n):
            e = pg.lens_list[b] // 4
            m = min(k, e)
            idx[tr.off[b] + i, :m] = torch.randperm(e, generator=g)[:m].sort().values.to(torch.int32)
    return idx


@pytest.fixture(params=[None, 60000], ids=["near", "far"])
def cap(request):
    """The rows' capacity: by it a call goes through whole caches node by node or, where it is far above these lengths, by rows
    on the tensor cores."""
    return request.param


LENS = [0, 1, 3, 4, 17, 64, 127, 128, 129, 300, 515, 1003]
NODES = [3, 0, 1, 2, 8, 9, 16, 17, 33, 128, 5, 64]
SHAPES = [("bf16", 16, 128, 64), ("bf16", 32, 128, 16), ("bf16", 16, 64, 4), ("bf16", 1, 128, 12), ("bf16", 5, 64, 100),
          ("bf16", 31, 64, 20), ("fp32", 8, 64, 16), ("fp32", 32, 128, 64), ("fp32", 3, 128, 100)]


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype,Hq,d,page", SHAPES)
@pytest.mark.parametrize("form", ["all", "chains", "selected"])
def test_tree_attention(dtype, Hq, d, page, form, cap):
    pg = Paged(LENS, page, d=d, dtype=dtype, seed=Hq + d + page, cap=cap).fill()
    tr = Trees(pg, NODES, Hq, chain=form == "chains", seed=page)
    dims = _dims(pg, Hq, k=9)
    idx = _selection(pg, tr, 9) if form == "selected" else None
    o, lse = _run(pg, tr, dims, idx)
    dsa.check_device_error()
    _check(pg, tr, o, lse, dims.scale, idx)


@pytest.mark.parametrize("dtype,Hq", [("bf16", 16), ("bf16", 32), ("bf16", 24), ("fp32", 8)])
@pytest.mark.parametrize("lens,nodes", [([20011], [16]), ([9001, 3, 0, 12289], [7, 1, 0, 12]), ([700] * 40, [3] * 40),
                                        ([130] * 300, [1] * 300), ([2500, 40], [100, 128]), ([0] * 5, [2] * 5), ([6000], [1])])
def test_tree_attention_batches(dtype, Hq, lens, nodes, cap):
    pg = Paged(lens, 16, dtype=dtype, seed=len(lens) + Hq, cap=cap).fill()
    tr = Trees(pg, nodes, Hq, seed=5)
    dims = _dims(pg, Hq)
    o, lse = _run(pg, tr, dims)
    dsa.check_device_error()
    _check(pg, tr, o, lse, dims.scale, rows=range(0, len(lens), 1 + len(lens) // 30))


@pytest.mark.parametrize("batch", [1, 17, 60, 150])
def test_tree_attention_of_selected_pools_in_batches(batch):
    pg = Paged([(b * 997) % 3000 + 1 for b in range(batch)], 64, seed=batch).fill()
    tr = Trees(pg, [1 + b % 6 for b in range(batch)], 16, seed=batch)
    dims = _dims(pg, 16, k=129)
    idx = _selection(pg, tr, 129)
    o, lse = _run(pg, tr, dims, idx)
    dsa.check_device_error()
    _check(pg, tr, o, lse, dims.scale, idx, rows=range(0, batch, 1 + batch // 20))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("how", ["large", "rising", "lowest"])
def test_tree_attention_of_awkward_scores(dtype, how, cap):
    """Scores far apart, rising along the keys (the running maximum moves all the time), and at the type's lowest values."""
    pg = Paged([900, 77], 16, dtype=dtype, seed=31, cap=cap)
    tr = Trees(pg, [20, 3], 16, seed=32)
    if how == "large":
        tr.q = (tr.q.float() * 40).to(pg.dt)
    elif how == "rising":
        for K in pg.K:
            K[:, 0] = torch.linspace(-60, 60, len(K)).to(pg.dt)
        tr.q[:, :, 0] = 30
    else:   # every cached score is about -1e30
        for K in pg.K:
            K.zero_()
            K[:, 0] = -1e15
        tr.q[:, :, 0] = 1e16
        tr.k[:, 0] = 0
    pg.fill()
    dims = _dims(pg, 16)
    o, lse = _run(pg, tr, dims)
    dsa.check_device_error()
    if how == "lowest":   # the cached keys weigh nothing
        pg.lens_list = [0, 0]
    _check(pg, tr, o, lse, dims.scale)


@pytest.mark.parametrize("dtype,Hq", [("bf16", 16), ("bf16", 32), ("fp32", 8)])
@pytest.mark.parametrize("selected", [False, True])
def test_other_branches_may_hold_anything(dtype, Hq, selected, cap):
    """NaN and infinities in the keys and values of nodes that are no ancestors change nothing; descendants get them."""
    pg = Paged([300, 9], 16, dtype=dtype, seed=41, cap=cap).fill()
    tr = Trees(pg, [40, 40], Hq, seed=42)
    tr.up = [[-1] + [i - 2 if i > 1 else -1 for i in range(1, 40)] for _ in range(2)]   # two branches: even and odd nodes
    sound = Trees(pg, [40, 40], Hq, seed=42)
    sound.up = tr.up
    for b in range(2):
        rows = torch.arange(1, 40, 2) + 40 * b
        tr.k[rows[5:]], tr.v[rows[3:]] = math.nan, math.inf
        tr.v[rows[7], ::2] = math.nan
    dims = _dims(pg, Hq, k=7)
    idx = _selection(pg, tr, 7) if selected else None
    got, want = _run(pg, tr, dims, idx), _run(pg, sound, dims, idx)
    dsa.check_device_error()
    _check(pg, sound, *want, dims.scale, idx)
    for b in range(2):
        even, odd = torch.arange(0, 40, 2) + 40 * b, torch.arange(1, 40, 2) + 40 * b
        for x, y in zip(got, want):
            assert torch.equal(x[even], y[even])
            assert torch.equal(x[odd[:3]], y[odd[:3]])
        assert not torch.any(torch.isfinite(got[0][odd[3:]]))      # an infinite value
        assert torch.equal(got[1][odd[3:5]], want[1][odd[3:5]])    # of a sound key
        assert torch.all(torch.isnan(got[1][odd[5:]]))


@pytest.mark.parametrize("dtype,Hq", [("bf16", 16), ("fp32", 8)])
def test_values_behind_a_row_are_not_read(dtype, Hq, cap):
    """Keys behind a row's length are NaN in the cache, also on its last page: test_tree_attention has that everywhere; here
    infinities of the row itself reach its nodes only (as infinities or NaN, the header says)."""
    pg = Paged([40, 200, 40], 16, dtype=dtype, seed=43, cap=cap)
    pg.V[1][100] = math.inf
    pg.fill()
    tr = Trees(pg, [4, 4, 4], Hq, seed=44)
    dims = _dims(pg, Hq)
    o, lse = _run(pg, tr, dims)
    dsa.check_device_error()
    assert not torch.any(torch.isfinite(o[4:8]))
    _check(pg, tr, o, lse, dims.scale, rows=[0, 2])


@pytest.mark.parametrize("dtype,Hq", [("bf16", 16), ("bf16", 32), ("fp32", 8)])
@pytest.mark.parametrize("selected", [False, True])
def test_bad_rows_are_skipped_and_reported(dtype, Hq, selected, cap):
    lens = [100, 50, 70, 33, 20, 64]
    nodes = [4, 129, 3, 5, 6, 2]
    pg = Paged(lens, 16, dtype=dtype, seed=51, cap=cap).fill()
    tr = Trees(pg, nodes, Hq, seed=52)
    dims = _dims(pg, Hq, k=5)
    idx = _selection(pg, tr, 5) if selected else None
    T, d = sum(nodes), 128
    run = lambda lens, table, off, parents: (  # noqa: E731
        dsa.decode_tree_attn(dims, pg.cache(), lens, table, off, parents, tr.q.to(DEV), tr.k.to(DEV), tr.v.to(DEV), o, lse,
                             _ws(dims, 6, T), idx=None if idx is None else idx.to(DEV)))
    fresh = lambda: (torch.full((T, Hq, d), 7.0, dtype=pg.dt, device=DEV), torch.full((T, Hq), 7.0, device=DEV))  # noqa: E731
    lens_d, table = pg.args()
    off, parents = tr.args()
    # row 1 has too many nodes
    o, lse = fresh()
    run(lens_d, table, off, parents)
    _reports(dsa.DSA_ERR_BAD_PAGE)
    assert torch.all(o[4:133] == 7) and torch.all(lse[4:133] == 7)
    _check(pg, tr, o, lse, dims.scale, idx, rows=[0, 2, 3, 4, 5])
    # parents out of range are roots; row 3 of a bad length is empty; nodes outside the offsets are left alone
    o, lse = fresh()
    bad_up = parents.clone()
    bad_up[tr.off[2] + 1], bad_up[tr.off[4]], bad_up[tr.off[4] + 5] = 1, -2, 77
    off2 = off.clone()
    off2[0], off2[6] = 2, T - 1
    bad_len = lens_d.clone()
    bad_len[3] = pg.cap + 1
    run(bad_len, table, off2, bad_up)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error()
    assert e.value.status in (dsa.DSA_ERR_BAD_INDEX, dsa.DSA_ERR_BAD_PAGE)
    assert torch.all(o[:2] == 7) and torch.all(o[T - 1] == 7) and torch.all(lse[T - 1] == 7) and torch.all(o[4:133] == 7)
    old = tr.up[2][1], tr.up[4][0], tr.up[4][5], pg.lens_list[3]
    tr.up[2][1], tr.up[4][0], tr.up[4][5], pg.lens_list[3] = -1, -1, -1, 0
    _check(pg, tr, o, lse, dims.scale, idx, rows=[2, 4])
    if idx is None:
        _check(pg, tr, o, lse, dims.scale, idx, rows=[3])
    tr.up[2][1], tr.up[4][0], tr.up[4][5], pg.lens_list[3] = old
    # offsets that descend
    o, lse = fresh()
    off3 = off.clone()
    off3[3] = off3[2] - 5
    run(lens_d, table, off3, parents)
    with pytest.raises(dsa.DSAError):   # row 3, which begins earlier, has other rows' parents too
        dsa.check_device_error()
    _check(pg, tr, o, lse, dims.scale, idx, rows=[0, 4, 5])
    # a bad page: its tokens are missing, nothing else
    o, lse = fresh()
    table2 = table.clone()
    table2[0, 2] = pg.pages
    run(lens_d, table2, off, parents)
    _reports(dsa.DSA_ERR_BAD_PAGE)
    _check(pg, tr, o, lse, dims.scale, idx, rows=[2, 3, 4, 5])
    if not selected:
        keep = torch.cat([torch.arange(32), torch.arange(48, 100)])
        K, V = pg.K[0], pg.V[0]
        pg.K[0], pg.V[0], pg.lens_list[0] = K[keep], V[keep], 84
        _check(pg, tr, o, lse, dims.scale, rows=[0])


def test_no_nodes_and_no_rows(cap):
    pg = Paged([20, 5], 16, seed=53, cap=cap).fill()
    dims = _dims(pg, 16)
    tr = Trees(pg, [0, 0], 16)
    o, lse = _run(pg, tr, dims)
    # node tensors that no row claims
    lens, table = pg.args()
    o, lse = torch.full((3, 16, 128), 7.0, dtype=pg.dt, device=DEV), torch.full((3, 16), 7.0, device=DEV)
    z = torch.zeros(3, 16, 128, dtype=pg.dt, device=DEV)
    dsa.decode_tree_attn(dims, pg.cache(), lens, table, torch.tensor([1, 1, 1], dtype=torch.int32, device=DEV), None, z,
                         z[:, 0].contiguous(), z[:, 0].contiguous(), o, lse, _ws(dims, 2, 3))
    dsa.check_device_error()
    assert torch.all(o == 7) and torch.all(lse == 7)


def test_calls_at_the_same_time(cap):
    """Calls on two streams, each with its own workspace, in flight together, give the bits that one alone gives."""
    pg = Paged([900, 1500, 4, 260], 16, seed=59, cap=cap).fill()
    Hq = 16
    dims = _dims(pg, Hq)
    trees = [Trees(pg, n, Hq, seed=57 + i) for i, n in enumerate(([40, 7, 1, 90], [3, 120, 0, 12]))]
    alone = [_run(pg, tr, dims) for tr in trees]
    cache, (lens, table) = pg.cache(), pg.args()
    args = [(*tr.args(), tr.q.to(DEV), tr.k.to(DEV), tr.v.to(DEV)) for tr in trees]
    outs = [[(torch.zeros_like(o), torch.zeros_like(l)) for _ in range(12)] for o, l in alone]
    ws = [_ws(dims, 4, tr.q.shape[0]) for tr in trees]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(12):
        for j in (0, 1):
            with torch.cuda.stream(streams[j]):
                dsa.decode_tree_attn(dims, cache, lens, table, *args[j], *outs[j][i], ws[j])
    torch.cuda.synchronize()
    dsa.check_device_error()
    for j in (0, 1):
        for o, lse in outs[j]:
            assert torch.equal(o, alone[j][0]) and torch.equal(lse, alone[j][1])


def test_graph_replay_other_streams_and_reproducibility(cap):
    pg = Paged([2000, 150, 0, 31], 16, seed=61, cap=cap).fill()
    Hq = 16
    dims = _dims(pg, Hq)
    trees = [Trees(pg, n, Hq, seed=62 + i) for i, n in enumerate(([9, 30, 2, 7], [20, 0, 25, 3], [1, 1, 1, 45]))]
    T = 48
    lens, table = pg.args()
    cache, ws = pg.cache(), _ws(dims, 4, T)
    q, k, v = (torch.zeros(T, *s, dtype=pg.dt, device=DEV) for s in ((Hq, 128), (128,), (128,)))
    off, up = torch.zeros(5, dtype=torch.int32, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    o, lse = torch.zeros(T, Hq, 128, dtype=pg.dt, device=DEV), torch.zeros(T, Hq, device=DEV)

    def load(tr):
        o_, p_ = tr.args()
        off.copy_(o_)
        up.copy_(p_)
        for a, b in ((q, tr.q), (k, tr.k), (v, tr.v)):
            a.copy_(b)

    call = lambda: dsa.decode_tree_attn(dims, cache, lens, table, off, up, q, k, v, o, lse, ws)  # noqa: E731
    load(trees[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    first = o.clone()
    _check(pg, trees[0], o, lse, dims.scale)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for tr in trees:
        load(tr)
        o.zero_()
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        _check(pg, tr, o, lse, dims.scale)
    load(trees[0])
    call()
    assert torch.equal(o, first)
    dsa.check_device_error()


@pytest.mark.parametrize("Hq,chain", [(16, False), (16, True)])
def test_cache_beyond_32_bit_offsets(Hq, chain, cap):
    """The same row at the far end of a cache of 4.6 GB a tensor gives the same bits."""
    page, d = 128, 128
    pages = (1 << 31) // (page * d) + 8
    pg = Paged([1000], page, seed=71, cap=cap).fill()
    tr = Trees(pg, [20], Hq, chain=chain, seed=72)
    dims = _dims(pg, Hq)
    near = _run(pg, tr, dims)
    k, v = (torch.full((pages, page, d), math.nan, dtype=pg.dt, device=DEV) for _ in range(2))
    old = pg.table.clone()
    new = torch.full_like(old, -7)
    for c in range(8):
        new[0, c] = pages - 1 - c
        k[pages - 1 - c], v[pages - 1 - c] = pg.k_c[old[0, c].long()].to(DEV), pg.v_c[old[0, c].long()].to(DEV)
    pg.table = new
    far = _run(pg, tr, dims, cache=dsa.PagedCache(k=k, v=v))
    dsa.check_device_error()
    assert torch.equal(near[0], far[0]) and torch.equal(near[1], far[1])


def test_rows_may_share_pages(cap):
    """Two rows with one table row: each as if it were alone."""
    pg = Paged([517, 517], 64, seed=73, cap=cap).fill()
    pg.table[1], pg.K[1], pg.V[1] = pg.table[0], pg.K[0], pg.V[0]
    tr = Trees(pg, [7, 11], 16, seed=74)
    dims = _dims(pg, 16)
    o, lse = _run(pg, tr, dims)
    dsa.check_device_error()
    _check(pg, tr, o, lse, dims.scale)


# ---------------------------------------------------------------- commit
@pytest.mark.parametrize("dtype,d,di,page", [("bf16", 128, 64, 64), ("bf16", 64, 128, 4), ("fp32", 128, 128, 12), ("fp32", 64, 64, 16)])
@pytest.mark.parametrize("chain", [False, True])
def test_commit_is_an_append(dtype, d, di, page, chain):
    lens = [0, 1, 2, 3, 4, 5, 6, 7, 30, 31, 62, 100, 101, 203]
    r = random.Random(page)
    nodes = [r.choice([1, 2, 5, 9, 40, 128]) for _ in lens]
    nodes[3] = 0
    pg = Paged([n + m for n, m in zip(lens, nodes)], page, d=d, di=di, dtype=dtype, seed=81 + page).fill(lens)
    tr = Trees(pg, nodes, 2, chain=chain, seed=82)
    acc = [r.randint(-1, n - 1) for n in nodes]
    acc[0], acc[13] = nodes[0] - 1, nodes[13] - 1
    dims = _dims(pg, 2)
    table = pg.table.to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    lines = [tr.line(b, a) for b, a in enumerate(acc)]
    after = [n + len(x) for n, x in zip(lens, lines)]
    want, got = pg.cache(), pg.cache()
    rows = torch.tensor([t for x in lines for t in x])
    off = i32([sum(map(len, lines[:b])) for b in range(len(lens) + 1)])
    dsa.cache_append(dims, want, i32(after), table, tr.k[rows].to(DEV), tr.v[rows].to(DEV), tr.ki[rows].to(DEV), offsets=off)
    offsets, parents = tr.args()
    lens_d = i32(lens)
    dsa.cache_commit(dims, got, lens_d, table, offsets, parents, i32(acc), tr.k.to(DEV), tr.v.to(DEV), tr.ki.to(DEV), lens_d)
    dsa.check_device_error()
    assert lens_d.tolist() == after
    view = torch.int16 if dtype == "bf16" else torch.int32
    for x in ("k", "v", "kpool", "ktail"):
        assert torch.equal(getattr(got, x).view(view), getattr(want, x).view(view)), x


def test_commit_skips_and_reports_bad_rows():
    lens, nodes = [10, 20, 30, 61, 9, 7], [4, 4, 4, 6, 130, 4]
    pg = Paged([64] * 6, 16, seed=83).fill(lens)
    tr = Trees(pg, nodes, 2, chain=True, seed=84)
    dims = _dims(pg, 2)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    offsets, _ = tr.args()
    kw = (tr.k.to(DEV), tr.v.to(DEV), tr.ki.to(DEV))

    def go(lens, acc, parents=None, table=None):
        cache, out = pg.cache(), torch.full((6,), -5, dtype=torch.int32, device=DEV)
        dsa.cache_commit(dims, cache, i32(lens), (pg.table if table is None else table).to(DEV), offsets, parents, i32(acc), *kw, out)
        return cache, out.tolist()

    # an accepted node that is not there; row 4 has too many nodes
    cache, out = go(lens, [4, -2, 1, -1, 3, 2])
    with pytest.raises(dsa.DSAError):
        dsa.check_device_error()
    assert out == [10, 20, 32, 61, 9, 10]
    clean = torch.isnan(cache.k.float()).any(-1)
    assert int((~clean).sum()) == sum(lens) + 2 + 3
    # a path past the capacity, a bad length
    cache, out = go([10, 70, 30, 61, -3, 7], [-1, 2, -1, 5, -1, -1])
    _reports(dsa.DSA_ERR_BAD_PAGE)
    assert out == [10, 70, 30, 61, -3, 7]
    # a bad parent on the path is the root
    up = torch.tensor([p for row in tr.up for p in row], dtype=torch.int32, device=DEV)
    up[2] = 3
    cache, out = go(lens, [3, -1, -1, -1, -1, -1], parents=up)
    with pytest.raises(dsa.DSAError):
        dsa.check_device_error()
    assert out[0] == 12
    # a token whose page is bad counts but does not enter
    table = pg.table.clone()
    table[1, 1] = -1
    cache, out = go(lens, [-1, 3, -1, -1, -1, -1], table=table)
    _reports(dsa.DSA_ERR_BAD_PAGE)
    assert out[1] == 24
    assert int((~torch.isnan(cache.k.float()).any(-1)).sum()) == sum(lens)


# ---------------------------------------------------------------- as they are used
@pytest.mark.parametrize("dtype,Hq", [("bf16", 16), ("fp32", 8)])
def test_a_chain_of_drafts_sees_what_single_steps_see(dtype, Hq):
    """Drafts judged at once attend as the same tokens appended one after the other and attended to with decode_attn do."""
    pg = Paged([130, 41], 16, dtype=dtype, seed=91, cap=152).fill([121, 32])
    # rows of the sequences' own next tokens as drafts
    tr = Trees(pg, [9, 9], Hq, chain=True, seed=92)
    tr.k, tr.v = (torch.cat([x[0][121:130], x[1][32:41]]) for x in (pg.K, pg.V))
    dims = _dims(pg, Hq)
    full = list(pg.lens_list)
    pg.lens_list = [121, 32]
    o, lse = _run(pg, tr, dims)
    _check(pg, tr, o, lse, dims.scale)
    pg.fill(full)
    rows = torch.arange(9).repeat(2)
    lens = (torch.tensor([121] * 9 + [32] * 9) + rows + 1).to(torch.int32).to(DEV)
    table = pg.table[[0] * 9 + [1] * 9].contiguous().to(DEV)
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    dsa.decode_attn(dims, pg.cache(), lens, table, tr.q.to(DEV), o2, lse2,
                    torch.empty(dsa.decode_workspace_bytes(dims, 18), dtype=torch.uint8, device=DEV))
    dsa.check_device_error()
    # each is within _check's tolerance of the same numbers, about 2^-16 of values of order 1, and rounded: a step apart at most
    step = 2 * HALF[dtype]
    assert torch.all((o.double() - o2.double()).abs() <= step * o.double().abs() + 1e-3 * step + 2.0 ** -13)
    assert torch.all((lse - lse2).abs() <= 1e-4)
