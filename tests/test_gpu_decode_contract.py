"""What the header of the paged decode operators promises beside the ordinary calls.  Caches, references and tolerances are
those of test_gpu_decode.
"""
import math

import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from test_gpu_decode import (DEV, Paged, _built, _check_attn, _close_rotated, _freq, _junk_ws, _ref_topk,  # noqa: F401
                             _rotate)

pytestmark = pytest.mark.gpu


def _reports(status):
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error()
    assert e.value.status == status


# ---------------------------------------------------------------- the newest token's page is bad
@pytest.mark.parametrize("dtype,Hq,inter", [("bf16", 16, False), ("bf16", 32, True), ("fp32", 8, False)])
def test_step_of_a_row_whose_newest_page_is_bad(dtype, Hq, inter):
    """Rows 0 and 2 begin a page that is not there: only the new token is missing from their results, which are those of
    their own, rotated query whatever the workspace held."""
    k, page, d = 6, 16, 128
    pg = Paged([161, 90, 49, 33], page, dtype=dtype, seed=110 + Hq).fill([160, 89, 48, 32])
    dims = dsa.make_dims(pg.cap, Hq, d, 8, 64, k, dtype=dtype)
    lens, table = pg.args()
    bad = table.clone()
    bad[0, 10], bad[2, 3] = pg.pages, -1
    rot = dsa.make_rotation(_freq(64), interleaved=inter)
    g = pg.g
    q = torch.randn(4, Hq, d, generator=g).to(pg.dt)
    qi = torch.randint(-3, 4, (4, 8, 64), generator=g).to(pg.dt)
    w = torch.randint(1, 5, (4, 8), generator=g).float()
    last = lambda xs: torch.stack([x[-1] for x in xs]).to(DEV)
    o, lse = torch.full((4, Hq, d), 7.0, dtype=pg.dt, device=DEV), torch.full((4, Hq), 7.0, device=DEV)
    idx = torch.full((4, k), -9, dtype=torch.int32, device=DEV)
    cache = pg.cache()
    dsa.decode_step(dims, cache, lens, bad, q.to(DEV), last(pg.K), last(pg.V), qi.to(DEV), last(pg.KI), w.to(DEV), o, lse, idx,
                    _junk_ws(dims, 4), rotation=rot)
    _reports(dsa.DSA_ERR_BAD_PAGE)
    assert torch.equal(idx.cpu(), _ref_topk(pg, qi, w, k))
    # the queries as an append with a sound table rotates them; where the new key went in, it is the rotated one
    q_rot = torch.full((4, Hq, d), 7.0, dtype=pg.dt, device=DEV)
    dsa.cache_append(dims, pg.cache(), lens, table, last(pg.K), last(pg.V), last(pg.KI), rotation=rot, q=q.to(DEV), q_out=q_rot)
    dsa.check_device_error()
    for b in (1, 3):
        at, r = pg.where(b, lens[b].item() - 1)
        pg.K[b][-1] = cache.k[at, r].cpu()
    pg.lens_list = [160, 90, 48, 33]         # what rows 0 and 2 have left
    _check_attn(pg, q_rot.cpu(), o, lse, d ** -0.5, idx.cpu())


@pytest.mark.parametrize("with_offsets", [False, True])
def test_append_to_a_bad_page_still_rotates(with_offsets):
    """q_out and k_out of a token whose page is bad are its rotated rows; nothing of it enters the cache."""
    pg = Paged([17, 40], 16, seed=112)
    dims = dsa.make_dims(pg.cap, 5, 128, 8, 64, 8)
    lens, table = pg.args()
    table[0, 1] = pg.pages
    q = torch.randn(2, 5, 128, generator=pg.g).to(torch.bfloat16)
    k = torch.stack([x[-1] for x in pg.K])
    q_out, k_out = torch.full_like(q, 7.0).to(DEV), torch.full_like(k, 7.0).to(DEV)
    off = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV) if with_offsets else None
    cache = pg.cache()
    dsa.cache_append(dims, cache, lens, table, k.to(DEV), k.to(DEV), torch.ones(2, 64, dtype=torch.bfloat16, device=DEV),
                     offsets=off, rotation=dsa.make_rotation(_freq(128)), q=q.to(DEV), q_out=q_out, k_out=k_out)
    _reports(dsa.DSA_ERR_BAD_PAGE)
    pos = torch.tensor([16, 39])
    _close_rotated(q_out, _rotate(q.double(), pos, _freq(128), False), "bf16")
    _close_rotated(k_out, _rotate(k.double(), pos, _freq(128), False), "bf16")
    assert int((~torch.isnan(cache.k.float()).any(-1)).sum()) == 1


# ---------------------------------------------------------------- part of a batch
@pytest.mark.parametrize("rot", [0, 64])
@pytest.mark.parametrize("n", [9, 4000])
def test_append_of_part_of_a_batch(n, rot):
    """offsets[0] > 0: the second half of a batch's rows, out of the tokens of the whole batch.  Rows before offsets[0] are
    left alone like those behind the last, and are no error."""
    total = [n, 1, 2 * n, 3, n + 5, 0, 3 * n, 2]
    pg = Paged(total, 16, seed=120 + n)
    dims = dsa.make_dims(pg.cap, 2, 128, 8, 64, 8)
    lens, table = pg.args()
    off = torch.tensor([0] + total, dtype=torch.int32).cumsum(0).to(torch.int32).to(DEV)
    cat = lambda xs: torch.cat(xs).to(DEV)
    kw = {}
    if rot:
        kw = dict(rotation=dsa.make_rotation(_freq(rot)), k_out=torch.full((sum(total), 128), 7.0, dtype=torch.bfloat16, device=DEV))
    half, whole = pg.cache(), pg.cache()
    dsa.cache_append(dims, half, lens[4:], table[4:], cat(pg.K), cat(pg.V), cat(pg.KI), offsets=off[4:], **kw)
    dsa.check_device_error()
    if rot:
        assert torch.all(kw["k_out"][:off[4]] == 7) and not torch.any((kw["k_out"][off[4]:] == 7).all(-1))
    there = ~torch.isnan(half.k.float()).any(-1)
    assert int(there.sum()) == sum(total[4:])
    dsa.cache_append(dims, half, lens[:4], table[:4], cat(pg.K), cat(pg.V), cat(pg.KI), offsets=off[:5], **kw)
    dsa.cache_append(dims, whole, lens, table, cat(pg.K), cat(pg.V), cat(pg.KI), offsets=off, **kw)
    dsa.check_device_error()
    for x in ("k", "v", "kpool", "ktail"):
        a, b = getattr(half, x), getattr(whole, x)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)), x


@pytest.mark.parametrize("off,appended", [([0, 2, 5, 9], [0, 1]), ([0, 2, 5, 5], [0, 1]), ([9, 9, 9, 9], []), ([0, 0, 0, -1], []),
                                          ([3, 3, 3, 2], []), ([1, 3, 3, 5], [0, 2])])
def test_offsets_outside_the_tokens_are_reported(off, appended):
    """Rows that the offsets put behind the call's 5 tokens, or that descend, are skipped and reported, other rows appended;
    offsets within 0 .. 5 that leave tokens out are no error."""
    pg = Paged([8, 11, 6], 16, seed=130)
    dims = dsa.make_dims(pg.cap, 4, 128, 8, 64, 8)
    lens, table = pg.args()
    cache = pg.cache()
    k = torch.randn(5, 128, generator=pg.g).to(torch.bfloat16).to(DEV)
    dsa.cache_append(dims, cache, lens, table, k, k, torch.ones(5, 64, dtype=torch.bfloat16, device=DEV),
                     offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
    if 0 <= off[0] <= off[-1] <= 5:
        dsa.check_device_error()
    else:
        _reports(dsa.DSA_ERR_BAD_PAGE)
    want = torch.full_like(cache.k, float("nan"))
    for b in appended:
        n = off[b + 1] - off[b]
        pos = torch.arange(pg.lens_list[b] - n, pg.lens_list[b])
        at, r = pg.where(b, pos)
        want[at, r] = k[off[b]:off[b + 1]]
    for got in (cache.k, cache.v):
        assert torch.equal(got.nan_to_num(9.0), want.nan_to_num(9.0))


# ---------------------------------------------------------------- an append across a bad page
@pytest.mark.parametrize("rot", [0, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_across_a_bad_page_keeps_the_open_pool(dtype, rot):
    """A prompt piece begins inside a pool on a bad page and ends inside a pool on a good one: the good page's tokens are
    all kept, so that the pool they begin is completed by a later append as if nothing had happened."""
    pg = Paged([8, 30], 4, dtype=dtype, seed=115)
    dims = dsa.make_dims(pg.cap, 4, 128, 8, 64, 8, dtype=dtype)
    table = pg.table.clone()
    table[0, 0] = -1
    cache = pg.cache()
    rotation = dsa.make_rotation(_freq(rot)) if rot else None

    def put(a, z):
        cat = lambda xs: torch.cat([x[i:j] for x, i, j in zip(xs, a, z)]).to(DEV)
        off = torch.tensor([0, z[0] - a[0], z[0] - a[0] + z[1] - a[1]], dtype=torch.int32, device=DEV)
        dsa.cache_append(dims, cache, torch.tensor(z, dtype=torch.int32, device=DEV), table.to(DEV), cat(pg.K), cat(pg.V),
                         cat(pg.KI), offsets=off, rotation=rotation)
    put([2, 0], [6, 22])                     # row 0: tokens 2, 3 on the bad page, 4, 5 on the next
    _reports(dsa.DSA_ERR_BAD_PAGE)
    put([6, 22], [8, 30])
    dsa.check_device_error()
    kp = cache.kpool.cpu()
    assert torch.equal(kp[pg.table[0, 1].long(), 0], pg.pool_keys(0)[1])
    assert torch.equal(kp[pg.table[1, :7].long(), 0], pg.pool_keys(1)[:7])


# ---------------------------------------------------------------- pools on bad pages
@pytest.mark.parametrize("dtype,Hi,di", [("bf16", 8, 64), ("bf16", 3, 128), ("fp32", 4, 64), ("fp32", 8, 128)])
@pytest.mark.parametrize("n,k", [(400, 20), (4096, 60), (40000, 700)])
def test_pools_on_bad_pages_rank_last(dtype, Hi, di, n, k):
    """Weights of both signs, so that many scores lie below 0: no pool of a bad page is selected while k others are there;
    where they are not, the others are all selected.  Rows of a few, thousands and tens of thousands of tokens."""
    pg = Paged([n, n - 3, n], 16, di=di, dtype=dtype, seed=n + k + di).fill()
    dims = dsa.make_dims(pg.cap, 16, 128, Hi, di, k, dtype=dtype)
    lens, table = pg.args()
    cols = table.shape[1]
    gone = [torch.arange(cols) % 3 == 1, torch.zeros(cols, dtype=torch.bool), torch.arange(cols) >= 2]
    for b, m in enumerate(gone):
        table[b, m.to(DEV)] = pg.pages if b else -1
    q = torch.randint(-3, 4, (3, Hi, di), generator=pg.g).to(pg.dt)
    w = -torch.randint(1, 5, (3, Hi), generator=pg.g).float()
    w[:, 0] = 1.0
    idx = torch.full((3, k), -9, dtype=torch.int32, device=DEV)
    dsa.decode_indexer_topk(dims, pg.cache(), lens, table, q.to(DEV), w.to(DEV), idx, _junk_ws(dims, 3))
    _reports(dsa.DSA_ERR_BAD_PAGE)
    for b in range(3):
        P = pg.lens_list[b] // 4
        ok = ~gone[b][torch.arange(P) * 4 // 16]
        s = ((q[b].double() @ pg.pool_keys(b)[:P].double().T).clamp(min=0) * w[b].double()[:, None]).sum(0)
        s[~ok] = -math.inf
        best = torch.sort(s, descending=True, stable=True).indices[:k].sort().values
        assert torch.equal(idx[b].cpu().long(), best), b


# ---------------------------------------------------------------- drafts
@pytest.mark.parametrize("dtype,rot", [("bf16", 0), ("bf16", 64), ("fp32", 64)])
def test_draft_tokens_are_appended_together_and_verified_as_rows(dtype, rot):
    """Three sequences, drafts of 6, 1 and 5 tokens across pools and pages: one append with a row per sequence, then a row
    per draft token for the indexer and the attention, each of which sees its sequence up to itself.  Then a draft is cut
    back to a multiple of 4 and other tokens follow: the pool keys are those of the sequence as it went on."""
    Hq, k, page = 8, 9, 16
    base, draft = [61, 40, 127], [6, 1, 5]
    n = [a + m for a, m in zip(base, draft)]
    pg = Paged(n, page, dtype=dtype, seed=140 + rot, cap=144).fill(base)
    dims = dsa.make_dims(pg.cap, Hq, 128, 8, 64, k, dtype=dtype)
    table = pg.table.to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    T = sum(draft)
    q = torch.randn(T, Hq, 128, generator=pg.g).to(pg.dt)
    qi = torch.randint(-3, 4, (T, 8, 64), generator=pg.g).to(pg.dt)
    w = torch.randint(1, 5, (T, 8), generator=pg.g).float()
    cat = lambda xs, a=base, z=n: torch.cat([x[i:j] for x, i, j in zip(xs, a, z)]).to(DEV)
    qd, cache = q.to(DEV), pg.cache()
    kw = dict(rotation=dsa.make_rotation(_freq(rot)), q=qd, q_out=qd) if rot else {}
    dsa.cache_append(dims, cache, i32(n), table, cat(pg.K), cat(pg.V), cat(pg.KI), offsets=i32([0, 6, 7, 12]), **kw)
    seq = [b for b, m in enumerate(draft) for _ in range(m)]
    rows = i32([base[b] + j + 1 for b, m in enumerate(draft) for j in range(m)])
    each = table[torch.tensor(seq, device=DEV)].contiguous()
    ws, idx = _junk_ws(dims, T), torch.full((T, k), -9, dtype=torch.int32, device=DEV)
    o, lse = torch.empty_like(qd), torch.empty(T, Hq, device=DEV)
    dsa.decode_indexer_topk(dims, cache, rows, each, qi.to(DEV), w.to(DEV), idx, ws)
    dsa.decode_attn(dims, cache, rows, each, qd, o, lse, ws, idx=idx)
    dsa.check_device_error()
    if rot:     # the keys as they went into the cache
        for b in range(3):
            at, r = pg.where(b, torch.arange(n[b]))
            pg.K[b] = cache.k.cpu()[at, r]
    pg.lens_list, pg.K, pg.V, pg.KI = rows.tolist(), *([x[b] for b in seq] for x in (pg.K, pg.V, pg.KI))
    assert torch.equal(idx.cpu(), _ref_topk(pg, qi, w, k))
    _check_attn(pg, qd.cpu(), o, lse, 128 ** -0.5, idx.cpu())
    # sequence 0 keeps 64 of its tokens and goes on otherwise
    more = torch.randint(-3, 4, (5, 64), generator=pg.g).to(pg.dt)
    kv = torch.zeros(5, 128, dtype=pg.dt, device=DEV)
    dsa.cache_append(dims, cache, i32([69]), table[:1], kv, kv, more.to(DEV), offsets=i32([0, 5]))
    dsa.check_device_error()
    got = cache.kpool.cpu()[pg.table[0, 64 // page].long(), 0]
    assert torch.equal(got, more[:4].double().sum(0).to(pg.dt))
