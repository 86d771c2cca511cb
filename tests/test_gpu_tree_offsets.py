"""Draft trees of many rows some of whose offsets are bad, against plain forms in 64 bits (test_gpu_tree's)."""
import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from test_gpu_decode import DEV, Paged, _built  # noqa: F401
from test_gpu_tree import Trees, _check, _dims, _selection, _ws, cap  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,selected", [("bf16", False), ("bf16", True), ("fp32", False), ("fp32", True)])
def test_bad_offsets_among_many_rows(dtype, selected, cap):
    """More rows than are all looked at for a node at once: offsets that descend, that are far too large or negative cost the rows
    that they belong to, and no other; nodes that no row claims are left alone."""
    B, Hq = 700, 4
    pg = Paged([(b * 13) % 40 for b in range(B)], 16, d=64, dtype=dtype, seed=95, cap=cap).fill()
    tr = Trees(pg, [b % 3 for b in range(B)], Hq, seed=96)
    dims = _dims(pg, Hq, k=3)
    idx = _selection(pg, tr, 3) if selected else None
    (lens, table), (off, parents), T = pg.args(), tr.args(), sum(tr.nodes)
    for bad in ({1: 2 ** 30}, {350: 0}, {349: -5, 500: 2 ** 31 - 1}, {0: 40}, {B: 600}, {176: 690, 525: 1}, {b: 0 for b in range(2, 340, 2)}):
        off2 = off.clone()
        for b, x in bad.items():
            off2[b] = x
        claims, o2 = [[] for _ in range(T)], off2.tolist()
        for b in range(B):
            if 0 <= o2[b] <= o2[b + 1] <= T and o2[b + 1] - o2[b] <= 128:
                for t in range(o2[b], o2[b + 1]):
                    claims[t].append(b)
        o, lse = torch.full((T, Hq, 64), 7.0, dtype=pg.dt, device=DEV), torch.full((T, Hq), 7.0, device=DEV)
        dsa.decode_tree_attn(dims, pg.cache(), lens, table, off2, parents, tr.q.to(DEV), tr.k.to(DEV), tr.v.to(DEV), o, lse,
                             _ws(dims, B, T), idx=None if idx is None else idx.to(DEV))
        with pytest.raises(dsa.DSAError):   # bad rows; rows that begin elsewhere have parents of others
            dsa.check_device_error()
        good = [b for b in range(B) if not {b, b + 1} & set(bad) and o2[0] <= tr.off[b] and tr.off[b + 1] <= o2[B] and
                all(claims[t] == [b] for t in range(tr.off[b], tr.off[b + 1]))]
        assert len(good) > B // 4
        _check(pg, tr, o, lse, dims.scale, idx, rows=good)
        free = torch.tensor([not c for c in claims], device=DEV)
        assert torch.all(o[free] == 7) and torch.all(lse[free] == 7)
