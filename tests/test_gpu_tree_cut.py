"""Draft trees by rows whose cut gives a CTA the end of one small group and then a single tile of the next
(test_tree_cut_host): every node against a plain form in 64 bits, and the same bits every time.  Tolerances: those of
test_gpu_decode."""
import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from test_gpu_decode import DEV, HALF, Paged, _built  # noqa: F401
from test_gpu_decode_forms import _launches
from test_gpu_tree import Trees, _dims, _ws
from test_tree_cut_host import SHAPES, hand_overs

pytestmark = pytest.mark.gpu


def _check_rows(pg, tr, o, lse, scale):
    """test_gpu_tree's _check, all nodes of a row at once and on the GPU."""
    d, u = tr.q.shape[2], HALF[pg.dtype]
    q, nk, nv = (x.to(DEV).double() for x in (tr.q, tr.k, tr.v))
    for b, n in enumerate(tr.nodes):
        if n == 0:
            continue
        at, L = slice(tr.off[b], tr.off[b] + n), pg.lens_list[b]
        sees = torch.zeros(n, n, dtype=torch.bool)
        for i in range(n):
            sees[i, [t - tr.off[b] for t in tr.line(b, i)]] = True
        k, v = torch.cat([pg.K[b].to(DEV).double(), nk[at]]), torch.cat([pg.V[b].to(DEV).double(), nv[at]])
        s = q[at] @ k.T * scale
        hidden = torch.cat([torch.zeros(n, L, dtype=torch.bool), ~sees], 1)[:, None].to(DEV)
        ds = (d + 4) * 2.0 ** -23 * scale * (q[at].abs() @ k.abs().T).masked_fill(hidden, 0).amax(-1)
        s.masked_fill_(hidden, -torch.inf)
        ref_l = torch.logsumexp(s, -1)
        p = (s - ref_l[..., None]).exp()
        ref, size, m = p @ v, p @ v.abs(), L + n
        two_terms = 2.0 ** -16 if pg.dtype == "bf16" else 0.0
        tol = (4 * ds[..., None] + 2.0 ** -18 + m * 2.0 ** -23 + two_terms) * size + u * ref.abs()
        err = (o[at].double() - ref).abs()
        assert torch.all(err <= tol), (b, (err / tol).max())
        err, tol = (lse[at].double() - ref_l).abs(), 2 * ds + 2.0 ** -20 + m * 2.0 ** -23 + 2.0 ** -22 * ref_l.abs()
        assert torch.all(err <= tol), (b, (err / tol).max())


@pytest.mark.parametrize("name", SHAPES)
def test_small_groups_behind_one_another(name):
    lens, nodes, Hq, d = SHAPES[name]
    assert hand_overs(lens, nodes, Hq) > 0
    pg = Paged(lens, 16, d=d, seed=len(lens) + d, cap=60000).fill()
    tr = Trees(pg, nodes, Hq, seed=3)
    dims, T = _dims(pg, Hq), sum(nodes)
    (n, table), (off, parents), cache, ws = pg.args(), tr.args(), pg.cache(), _ws(dims, len(lens), T)
    q, k, v = tr.q.to(DEV), tr.k.to(DEV), tr.v.to(DEV)
    outs = [(torch.full((T, Hq, d), 7.0, dtype=pg.dt, device=DEV), torch.full((T, Hq), 7.0, device=DEV)) for _ in range(50)]
    call = lambda o, lse, stream=None: dsa.decode_tree_attn(dims, cache, n, table, off, parents, q, k, v, o, lse, ws,  # noqa: E731
                                                            stream=stream)
    for x in outs:
        call(*x)
    dsa.check_device_error()
    assert _launches(lambda stream: call(*outs[0], stream=stream)) == 2   # by rows: the kernel and the join
    _check_rows(pg, tr, *outs[0], dims.scale)
    for x in outs[1:]:
        assert torch.equal(x[0], outs[0][0]) and torch.equal(x[1], outs[0][1])


@pytest.mark.parametrize("dtype,selected", [("bf16", True), ("fp32", True), ("fp32", False), ("bf16", False)])
def test_more_nodes_than_a_grid_has_rows(dtype, selected):
    """70000 nodes and some that no row claims; by nodes that is more than one launch.  A selection of all of a row's pools
    is the whole row."""
    B, n, Hq, d, pad = 700, 100, 2, 64, 9
    pg = Paged([(b * 7) % 30 for b in range(B)], 16, d=d, dtype=dtype, seed=4).fill()
    tr = Trees(pg, [n] * B, Hq, seed=5)
    dims, T = _dims(pg, Hq, k=8), n * B
    (lens, table), (off, parents) = pg.args(), tr.args()
    z = lambda x: torch.cat([x, torch.full((pad, *x.shape[1:]), torch.nan, dtype=x.dtype)]).to(DEV)  # noqa: E731
    parents = torch.cat([parents, torch.full((pad,), 5, dtype=torch.int32, device=DEV)])
    idx = None
    if selected:
        p = torch.arange(8, dtype=torch.int32)
        idx = torch.cat([torch.where(p < n_ // 4, p, -1).repeat(n, 1) for n_ in pg.lens_list] + [p.repeat(pad, 1)]).to(torch.int32).to(DEV)
    o, lse = torch.full((T + pad, Hq, d), 7.0, dtype=pg.dt, device=DEV), torch.full((T + pad, Hq), 7.0, device=DEV)
    dsa.decode_tree_attn(dims, pg.cache(), lens, table, off, parents, z(tr.q), z(tr.k), z(tr.v), o, lse, _ws(dims, B, T + pad), idx=idx)
    dsa.check_device_error()
    assert torch.all(o[T:] == 7) and torch.all(lse[T:] == 7)
    tr.nodes = [m if b % 50 in (0, 29, 49) else 0 for b, m in enumerate(tr.nodes)]   # the rows that are checked
    _check_rows(pg, tr, o[:T], lse[:T], dims.scale)
