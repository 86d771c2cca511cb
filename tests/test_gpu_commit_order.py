"""Commits of indexer keys whose sums show the order of their additions, bit for bit against cache_append's."""
import random

import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from test_gpu_decode import DEV, Paged, _built  # noqa: F401
from test_gpu_tree import Trees, _dims

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,di,page", [("bf16", 64, 16), ("bf16", 128, 4), ("fp32", 64, 12), ("fp32", 128, 64)])
def test_commit_adds_keys_in_the_order_of_an_append(dtype, di, page):
    """test_commit_is_an_append's keys are small integers, whose sums are exact in any order.  Of these a quarter is 2^30 or -2^30, so that
    what is left of a pool's other keys, even in bf16, goes with the order."""
    lens = [0, 1, 2, 3, 4, 5, 6, 7, 30, 31, 62, 101]
    r, g = random.Random(di + page), torch.Generator().manual_seed(di + page)
    nodes = [r.choice([4, 5, 9, 40, 128]) for _ in lens]
    pg = Paged([n + m for n, m in zip(lens, nodes)], page, di=di, dtype=dtype, seed=97).fill(lens)
    def real(*s):
        x = torch.randn(*s, generator=g) * 2.0 ** torch.randint(-8, 9, s, generator=g)
        big = 2.0 ** 30 * (2 * torch.randint(0, 2, s, generator=g) - 1)
        return torch.where(torch.rand(*s, generator=g) < 0.25, big, x).to(pg.dt)

    pg.kt_c = real(*pg.kt_c.shape)
    tr = Trees(pg, nodes, 2, seed=98, wide=2)
    tr.ki = real(*tr.ki.shape)
    acc = [n - 1 - i % 3 for i, n in enumerate(nodes)]
    dims, table = _dims(pg, 2), pg.table.to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    lines = [tr.line(b, a) for b, a in enumerate(acc)]
    want, got = pg.cache(), pg.cache()
    rows = torch.tensor([t for x in lines for t in x])
    off = i32([sum(map(len, lines[:b])) for b in range(len(lens) + 1)])
    dsa.cache_append(dims, want, i32([n + len(x) for n, x in zip(lens, lines)]), table, tr.k[rows].to(DEV), tr.v[rows].to(DEV),
                     tr.ki[rows].to(DEV), offsets=off)
    offsets, parents = tr.args()
    dsa.cache_commit(dims, got, i32(lens), table, offsets, parents, i32(acc), tr.k.to(DEV), tr.v.to(DEV), tr.ki.to(DEV), i32(lens))
    dsa.check_device_error()
    view = torch.int16 if dtype == "bf16" else torch.int32
    for x in ("k", "v", "kpool", "ktail"):
        assert torch.equal(getattr(got, x).view(view), getattr(want, x).view(view)), x
    # the order of additions can be seen in these keys
    b = 8
    keys = torch.cat([pg.kt_c[pg.table[b, 29 // page], :2], tr.ki[lines[b]]])[:4].float()
    fwd, back = (((k[0] + k[1]) + k[2] + k[3]).to(pg.dt) for k in (keys, keys.flip(0)))
    assert torch.any(fwd != back)
