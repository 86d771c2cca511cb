"""GPU parity of the paged decode operators against plain forms in 64 bits.

Every cache starts full of NaN: only what a sequence holds is ever written, so a kernel that reads past a
sequence's end, an unselected page or an empty slot shows it.

Tolerances (u = half a step of the type, relative: bf16 2^-8, fp32 2^-24).  A score is a sum of d products; in fp32
its error is at most ds = (d + 4) * 2^-23 * scale * sum |q k| (2^-23: a tensor core's adds may truncate).  A weight
exp(s - m) is then off by at most 2 ds + 2^-20 relative (the exponential's and the rescalings' own error), plus
2^-16 where it enters the second product as two bf16 terms, so with A = sum_j p_j |v_j| the output is off by at
most (4 ds + 2^-18 + n 2^-23) A (numerator and denominator; n keys added in fp32) plus its rounding u |o|; the lse
by 2 ds + 2^-20 + n 2^-23 + 2^-22 |lse|.
"""
import math

import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_sparse_dsa_gb300 import build
    build.build()
    dsa.library()


def _dt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


class Paged:
    """Sequences of the given lengths, contiguous on the host in 64 bits, and the same in a scattered, NaN-filled cache."""

    def __init__(self, lens, page, d=128, di=64, dtype="bf16", seed=0, cap=None, spare=3):
        g = self.g = torch.Generator().manual_seed(seed)
        self.dtype, self.page, self.dt = dtype, page, _dt(dtype)
        self.lens_list = list(lens)
        self.cap = cap or max(4, (max(lens) + 3) // 4 * 4)
        cols = -(-self.cap // page)
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        perm = torch.randperm(self.pages, generator=g).tolist()
        self.table = torch.full((len(lens), cols), -7, dtype=torch.int32)    # entries behind the last page: never read
        for b, n in enumerate(need):
            for c in range(n):
                self.table[b, c] = perm.pop()
        nan = lambda *s: torch.full(s, math.nan, dtype=self.dt)
        self.k_c, self.v_c = nan(self.pages, page, d), nan(self.pages, page, d)
        self.kp_c, self.kt_c = nan(self.pages, page // 4, di), nan(self.pages, 3, di)
        draw = lambda n, w: torch.randn(n, w, generator=g).to(self.dt)
        self.K, self.V = [draw(n, d) for n in lens], [draw(n, d) for n in lens]
        self.KI = [torch.randint(-3, 4, (n, di), generator=g).to(self.dt) for n in lens]

    def where(self, b, pos):
        return self.table[b, pos // self.page].long(), pos % self.page

    def fill(self, upto=None):
        """Write the sequences' first upto[b] tokens (default: all) into the cache."""
        for b, n in enumerate(self.lens_list if upto is None else upto):
            pos = torch.arange(n)
            pg, r = self.where(b, pos)
            self.k_c[pg, r], self.v_c[pg, r] = self.K[b][:n], self.V[b][:n]
            done = torch.arange(n // 4)
            pg, _ = self.where(b, 4 * done)
            self.kp_c[pg, done % (self.page // 4)] = self.pool_keys(b)[:n // 4]
            if n % 4:
                self.kt_c[self.table[b, (n - 1) // self.page].long(), :n % 4] = self.KI[b][n // 4 * 4:n]
        return self

    def pool_keys(self, b):
        n = len(self.KI[b]) // 4
        return self.KI[b][:4 * n].double().view(n, 4, self.KI[b].shape[1]).sum(1).to(self.dt)   # small integers: exact

    def cache(self):
        return dsa.PagedCache(k=self.k_c.to(DEV), v=self.v_c.to(DEV), kpool=self.kp_c.to(DEV), ktail=self.kt_c.to(DEV))

    def args(self):
        return torch.tensor(self.lens_list, dtype=torch.int32, device=DEV), self.table.to(DEV)

    def keys(self, b, idx=None):
        n = self.lens_list[b]
        if idx is None:
            return list(range(n))
        return [4 * p + j for p in idx[b].tolist() if 0 <= p < n // 4 for j in range(4)] + list(range(n // 4 * 4, n))


def _check_attn(pg, q, o, lse, scale, idx=None):
    d, u = q.shape[2], HALF[pg.dtype]
    o, lse = o.double().cpu(), lse.double().cpu()
    for b in range(q.shape[0]):
        rows = pg.keys(b, idx)
        if not rows:
            assert torch.all(o[b] == 0) and torch.all(lse[b] == -math.inf)
            continue
        k, v, qq = pg.K[b][rows].double(), pg.V[b][rows].double(), q[b].double()
        s = qq @ k.T * scale
        ref_l = torch.logsumexp(s, -1)
        p = (s - ref_l[:, None]).exp()
        ref = p @ v
        ds = (d + 4) * 2.0 ** -23 * scale * (qq.abs() @ k.abs().T).amax(-1)
        n = len(rows)
        tol = (4 * ds[:, None] + 2.0 ** -18 + n * 2.0 ** -23) * (p @ v.abs()) + u * ref.abs()
        if pg.dtype == "bf16":
            tol += 2.0 ** -16 * (p @ v.abs())
        assert torch.all((o[b] - ref).abs() <= tol), (b, ((o[b] - ref).abs() / tol).max())
        ltol = 2 * ds + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * ref_l.abs()
        assert torch.all((lse[b] - ref_l).abs() <= ltol), (b, ((lse[b] - ref_l).abs() / ltol).max())


def _attn(pg, Hq, d, k=8, idx=None, q_scale=1.0, stream=None):
    dims = dsa.make_dims(pg.cap, Hq, d, 8, 64, k, dtype=pg.dtype)
    B = len(pg.lens_list)
    q = (torch.randn(B, Hq, d, generator=pg.g) * q_scale).to(pg.dt)
    lens, table = pg.args()
    o = torch.full((B, Hq, d), 7.0, dtype=pg.dt, device=DEV)
    lse = torch.full((B, Hq), 7.0, device=DEV)
    dsa.decode_attn(dims, pg.cache(), lens, table, q.to(DEV), o, lse, _junk_ws(dims, B),
                    idx=None if idx is None else idx.to(DEV))
    return q, o, lse


def _junk_ws(dims, B):
    return torch.full((dsa.decode_workspace_bytes(dims, B),), 0xFF, dtype=torch.uint8, device=DEV)   # NaNs


LENS = [0, 1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 65, 130, 257, 1003]


# ---------------------------------------------------------------- dense attention
@pytest.mark.parametrize("dtype,Hq,d,page", [
    ("bf16", 16, 128, 64), ("bf16", 32, 128, 16), ("bf16", 16, 64, 4), ("bf16", 32, 64, 100), ("bf16", 1, 128, 12),
    ("bf16", 5, 64, 128), ("bf16", 17, 128, 64), ("bf16", 31, 64, 20),
    ("fp32", 8, 64, 16), ("fp32", 32, 128, 64), ("fp32", 1, 64, 4), ("fp32", 5, 128, 100)])
def test_dense_attention(dtype, Hq, d, page):
    pg = Paged(LENS, page, d=d, dtype=dtype, seed=Hq + d + page).fill()
    q, o, lse = _attn(pg, Hq, d)
    _check_attn(pg, q, o, lse, d ** -0.5)
    dsa.check_device_error()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[20011], [9001, 3, 0, 12289], [700] * 70, [1] * 600, [0] * 5,
                                  [1 + 7919 * b % 613 for b in range(700)]])
def test_dense_attention_batches(dtype, lens):
    """One long row, very uneven rows, more rows than resident CTAs (of one token each, and of uneven lengths, so that rows
    straddle the CTAs' ranges), only idle rows."""
    pg = Paged(lens, 64, d=64, dtype=dtype, seed=3).fill()
    q, o, lse = _attn(pg, 16, 64)
    _check_attn(pg, q, o, lse, 64 ** -0.5)
    dsa.check_device_error()


@pytest.mark.parametrize("dtype,Hq", [("bf16", 16), ("bf16", 32), ("fp32", 8), ("fp32", 20)])
@pytest.mark.parametrize("batch", [1, 17, 28, 45, 95, 150, 400, 700])
def test_dense_attention_short_rows(dtype, Hq, batch):
    """Whole caches of short rows in every number of CTAs per row, and more rows than fit at once."""
    lens = [(b * 7919 + 61) % 260 if b % 9 else 0 for b in range(batch)]
    lens[0] = 301
    pg = Paged(lens, 16, d=64, dtype=dtype, seed=batch + Hq).fill()
    q, o, lse = _attn(pg, Hq, 64)
    _check_attn(pg, q, o, lse, 64 ** -0.5)
    dsa.check_device_error()


@pytest.mark.parametrize("cap", [304, 60000])
def test_dense_attention_skips_and_reports_bad_rows(cap):
    """A bad page's tokens are missing, a row of bad length is idle, others are as without: for short rows and long ones."""
    pg = Paged([300, 170, 0, 65], 16, seed=4, cap=cap).fill()
    dims = dsa.make_dims(cap, 16, 128, 8, 64, 8)
    q = torch.randn(4, 16, 128, generator=pg.g).to(torch.bfloat16).to(DEV)
    lens, table = pg.args()

    def call(l, t):
        o, lse = torch.full_like(q, 7.0), torch.full((4, 16), 7.0, device=DEV)
        dsa.decode_attn(dims, pg.cache(), l, t, q, o, lse, _junk_ws(dims, 4))
        return o, lse

    o, lse = call(lens, table)
    _check_attn(pg, q.cpu(), o, lse, 128 ** -0.5)
    dsa.check_device_error()
    t = table.clone()
    t[0, 3], t[3, :] = pg.pages, -1
    o1, lse1 = call(lens, t)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error()
    assert e.value.status == dsa.DSA_ERR_BAD_PAGE
    assert torch.equal(o1[1], o[1]) and torch.all(o1[3] == 0) and torch.all(lse1[3] == -math.inf)
    assert not torch.equal(o1[0], o[0])
    pg.K[0], pg.V[0] = [torch.cat([x[:48], x[64:]]) for x in (pg.K[0], pg.V[0])]
    pg.lens_list = [284, 170, 0, 0]
    _check_attn(pg, q.cpu(), o1, lse1, 128 ** -0.5)
    l = lens.clone()
    l[0], l[1] = cap + 1, -2
    o2, lse2 = call(l, table)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error()
    assert e.value.status == dsa.DSA_ERR_BAD_PAGE
    assert torch.all(o2[:2] == 0) and torch.all(lse2[:2] == -math.inf) and torch.equal(o2[3], o[3])
    dsa.check_device_error()


def test_capacity_far_above_the_lengths():
    pg = Paged([5, 1000, 64], 16, cap=1 << 20).fill()
    q, o, lse = _attn(pg, 16, 128)
    _check_attn(pg, q, o, lse, 128 ** -0.5)
    dsa.check_device_error()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_scores(dtype):
    """Scores of some hundreds: the running maximum moves, earlier keys vanish."""
    pg = Paged([300, 77, 1024], 64, dtype=dtype, seed=9).fill()
    q, o, lse = _attn(pg, 16, 128, q_scale=60.0)
    _check_attn(pg, q, o, lse, 128 ** -0.5)


def test_infinite_and_nan_values_stay_in_their_rows():
    """A row whose keys hold NaN is NaN, a channel whose values hold infinity is not finite; other rows and channels are
    untouched."""
    pg = Paged([40, 50, 60], 16, seed=4)
    pg.K[0][3, 5] = math.nan
    pg.V[1][7, 2] = math.inf
    pg.fill()
    q, o, lse = _attn(pg, 16, 128)
    assert torch.isnan(o[0].float()).all() and torch.isnan(lse[0]).all()
    assert not torch.isfinite(o[1, :, 2].float()).any() and torch.isfinite(lse[1]).all()
    assert torch.isfinite(o[1, :, :2].float()).all() and torch.isfinite(o[1, :, 3:].float()).all()
    pg.lens_list, pg.K, pg.V = [60], pg.K[2:], pg.V[2:]
    _check_attn(pg, q[2:], o[2:], lse[2:], 128 ** -0.5)


# ---------------------------------------------------------------- selected pools
def _selection(pg, k, seed=1):
    g = torch.Generator().manual_seed(seed)
    idx = torch.full((len(pg.lens_list), k), -1, dtype=torch.int32)
    for b, n in enumerate(pg.lens_list):
        pick = torch.randperm(n // 4, generator=g)[:k].sort().values
        idx[b, :len(pick)] = pick.to(torch.int32)
    return idx


@pytest.mark.parametrize("dtype,Hq,d,page,k", [
    ("bf16", 16, 128, 64, 32), ("bf16", 32, 128, 16, 7), ("bf16", 16, 64, 4, 1), ("bf16", 3, 64, 100, 33),
    ("bf16", 32, 64, 20, 300), ("bf16", 20, 128, 128, 1024), ("fp32", 8, 64, 16, 64), ("fp32", 32, 128, 12, 5)])
def test_selected_attention(dtype, Hq, d, page, k):
    pg = Paged(LENS, page, d=d, dtype=dtype, seed=Hq + d + page + k).fill()
    idx = _selection(pg, k)
    q, o, lse = _attn(pg, Hq, d, k, idx)
    _check_attn(pg, q, o, lse, d ** -0.5, idx)
    dsa.check_device_error()


@pytest.mark.parametrize("dtype,Hq", [("bf16", 16), ("bf16", 32), ("fp32", 8)])
@pytest.mark.parametrize("batch", [1, 17, 28, 45, 60, 95, 150, 400, 700])
def test_selected_attention_batches(dtype, Hq, batch):
    """Every number of CTAs per row (16, 8 .. 1), and more rows than fit at once; some rows idle or too short to fill k."""
    lens = [(b * 7919 + 61) % 800 if b % 9 else 0 for b in range(batch)]
    lens[0] = 801
    pg = Paged(lens, 16, d=64, dtype=dtype, seed=batch).fill()
    idx = _selection(pg, 150)
    q, o, lse = _attn(pg, Hq, 64, 150, idx)
    _check_attn(pg, q, o, lse, 64 ** -0.5, idx)
    dsa.check_device_error()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_selection_in_any_form(dtype):
    """-1 anywhere, any order, nothing selected, a pool named twice (it counts twice), and the row's incomplete pool named
    (row 4's pool 100: it is not a complete one, so the entry is skipped and reported; its tokens are attended anyway)."""
    pg = Paged([257, 130, 66, 64, 403], 16, dtype=dtype, seed=6).fill()
    idx = torch.full((5, 9), -1, dtype=torch.int32)
    idx[0] = torch.tensor([-1, 63, -1, -1, 2, 0, -1, 40, -1])
    idx[2] = torch.tensor([5, 5, 1, -1, 5, -1, 0, 15, 2])
    idx[4] = torch.tensor([100, 99, 98, 97, 96, 95, 94, 93, 92])
    q, o, lse = _attn(pg, 16, 128, 9, idx)      # row 1: the partial pool only; row 3: no key at all
    _check_attn(pg, q, o, lse, 128 ** -0.5, idx)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error()
    assert e.value.status == dsa.DSA_ERR_BAD_INDEX


def test_bad_pools_pages_and_lengths_are_skipped_and_reported():
    pg = Paged([200, 200, 200, 200], 16, seed=8).fill()
    dims = dsa.make_dims(pg.cap, 16, 128, 8, 64, 10)
    idx = _selection(pg, 10)
    lens, table = pg.args()
    q = torch.randn(4, 16, 128, generator=pg.g).to(torch.bfloat16)
    ws, cache = _junk_ws(dims, 4), pg.cache()

    def call(i, l, t):
        o = torch.full((4, 16, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((4, 16), 7.0, device=DEV)
        dsa.decode_attn(dims, cache, l, t, q.to(DEV), o, lse, ws, idx=i)
        return o, lse

    bad = idx.clone()
    bad[1, 3], bad[2, 0] = 50, 1 << 30             # row 1 holds pools 0..49
    o, lse = call(bad.to(DEV), lens, table)
    _check_attn(pg, q, o, lse, 128 ** -0.5, bad)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error()
    assert e.value.status == dsa.DSA_ERR_BAD_INDEX
    for form in (idx.to(DEV), None):
        t = table.clone()
        t[3, :] = pg.pages                          # one past the last page, for every page of row 3
        t[1, 0] = -1
        o, lse = call(form, lens, t)
        with pytest.raises(dsa.DSAError) as e:
            dsa.check_device_error()
        assert e.value.status == dsa.DSA_ERR_BAD_PAGE
        assert torch.all(o[3] == 0) and torch.all(lse[3] == -math.inf)
        l = lens.clone()
        l[0], l[2] = -5, pg.cap + 1                 # both rows count as idle
        o2, lse2 = call(form, l, table)
        with pytest.raises(dsa.DSAError) as e:
            dsa.check_device_error()
        assert e.value.status == dsa.DSA_ERR_BAD_PAGE
        for b in (0, 2):
            assert torch.all(o2[b] == 0) and torch.all(lse2[b] == -math.inf)
        good, good_l = call(form, lens, table)
        assert torch.equal(o2[1], good[1]) and torch.equal(o[2], good[2]) and torch.equal(lse2[3], good_l[3])
    dsa.check_device_error()


# ---------------------------------------------------------------- indexer + top-k
def _ref_topk(pg, q, w, k):
    B = q.shape[0]
    idx = torch.full((B, k), -1, dtype=torch.int32)
    for b, n in enumerate(pg.lens_list):
        s = ((q[b].double() @ pg.pool_keys(b)[:n // 4].double().T).clamp(min=0) * w[b].double()[:, None]).sum(0)
        best = torch.sort(s + 0.0, descending=True, stable=True).indices[:k].sort().values
        idx[b, :len(best)] = best.to(torch.int32)
    return idx


def _topk(pg, Hi, di, k, lo=-3, w_lo=1):
    dims = dsa.make_dims(pg.cap, 16, 128, Hi, di, k, dtype=pg.dtype)
    B = len(pg.lens_list)
    q = torch.randint(lo, -lo + 1, (B, Hi, di), generator=pg.g).to(pg.dt)
    w = torch.randint(w_lo, 5 if w_lo > 0 else 2, (B, Hi), generator=pg.g).float()
    lens, table = pg.args()
    idx = torch.full((B, k), -9, dtype=torch.int32, device=DEV)
    dsa.decode_indexer_topk(dims, pg.cache(), lens, table, q.to(DEV), w.to(DEV), idx, _junk_ws(dims, B))
    return q, w, idx


@pytest.mark.parametrize("dtype,Hi,di,page,k", [
    ("bf16", 8, 64, 64, 16), ("bf16", 4, 128, 16, 5), ("bf16", 1, 64, 4, 1), ("bf16", 5, 128, 100, 250),
    ("bf16", 7, 64, 20, 512), ("fp32", 4, 64, 16, 64), ("fp32", 8, 128, 12, 3), ("fp32", 3, 128, 64, 1024)])
def test_indexer_topk(dtype, Hi, di, page, k):
    pg = Paged(LENS + [4001], page, di=di, dtype=dtype, seed=Hi + di + k).fill()
    q, w, idx = _topk(pg, Hi, di, k)
    assert torch.equal(idx.cpu(), _ref_topk(pg, q, w, k))
    dsa.check_device_error()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,k", [([90001], 512), ([70000, 50, 0, 30003], 1024), ([2000] * 200, 64), ([40000], 1),
                                    ([0, 0, 3], 8)])
def test_indexer_topk_batches(dtype, lens, k):
    """Long rows with thousands of ties (inputs in -1..1, weights of both signs), few and many rows, no pool at all."""
    pg = Paged(lens, 64, dtype=dtype, seed=k).fill()
    q, w, idx = _topk(pg, 8, 64, k, lo=-1, w_lo=-1)
    assert torch.equal(idx.cpu(), _ref_topk(pg, q, w, k))
    dsa.check_device_error()


def test_indexer_topk_all_scores_equal():
    """Every score 0 (or -0): the first k pools."""
    pg = Paged([50003, 17], 64, seed=2).fill()
    dims = dsa.make_dims(pg.cap, 16, 128, 8, 64, 512)
    lens, table = pg.args()
    idx = torch.empty(2, 512, dtype=torch.int32, device=DEV)
    for w0 in (0.0, -0.0):
        w = torch.full((2, 8), w0, device=DEV)
        q = torch.ones(2, 8, 64, dtype=torch.bfloat16, device=DEV)
        dsa.decode_indexer_topk(dims, pg.cache(), lens, table, q, w, idx, _junk_ws(dims, 2))
        assert torch.equal(idx[0].cpu(), torch.arange(512, dtype=torch.int32))
        assert idx[1].tolist() == [0, 1, 2, 3] + [-1] * 508


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_indexer_topk_many_wide_rows(dtype):
    """The wide indexer (di = 128) at a size that gives every warp a full block of pools."""
    pg = Paged([9000 + 37 * b for b in range(30)], 64, di=128, dtype=dtype, seed=77).fill()
    q, w, idx = _topk(pg, 8, 128, 300)
    assert torch.equal(idx.cpu(), _ref_topk(pg, q, w, 300))
    dsa.check_device_error()


@pytest.mark.parametrize("Hi,di", [(1, 64), (3, 128), (4, 64), (4, 128), (5, 64)])
def test_indexer_topk_many_rows_of_few_heads(Hi, di):
    """fp32 with at most and just above 4 heads, at a size that gives every warp a full block of pools."""
    pg = Paged([9000 + 37 * b for b in range(38)], 20, di=di, dtype="fp32", seed=di + Hi).fill()
    q, w, idx = _topk(pg, Hi, di, 70)
    assert torch.equal(idx.cpu(), _ref_topk(pg, q, w, 70))
    dsa.check_device_error()


@pytest.mark.parametrize("batch", [2, 15, 18, 19, 37, 77, 153])
def test_indexer_topk_cluster_sizes(batch):
    """Rows beyond the exact limit, in batches around those at which the clusters change: alone on the SMs, side by side,
    smaller, one CTA a row.  The candidates crowd into one CTA's slice in every third row."""
    g = torch.Generator().manual_seed(batch)
    values = []
    for b in range(batch):
        v = torch.rand(8300 + 61 * (b % 9), generator=g)
        if b % 3 == 0:
            v[4100:4900] += 2.0
        values.append(v)
    _given_scores(values, 300)


def _given_scores(values, k, sign=1.0):
    """Rows of an fp32 layer whose scores are exactly sign * values [B][n] (each >= 0): one indexer head that reads one
    channel."""
    B = len(values)
    lens = [4 * len(v) for v in values]
    cap = max(lens)
    cols = cap // 64 + 1
    dims = dsa.make_dims(cap, 16, 128, 1, 64, k, dtype="fp32")
    table = torch.arange(B * cols, dtype=torch.int32).view(B, cols)[:, :-(-cap // 64)].contiguous()
    kpool = torch.zeros(B * cols, 16, 64)
    for b, v in enumerate(values):
        flat = torch.zeros(cols * 16)
        flat[:len(v)] = v
        kpool[b * cols:(b + 1) * cols, :, 0] = flat.view(cols, 16)
    q = torch.zeros(B, 1, 64)
    q[:, 0, 0] = 1.0
    idx = torch.full((B, k), -9, dtype=torch.int32, device=DEV)
    dsa.decode_indexer_topk(dims, dsa.PagedCache(kpool=kpool.to(DEV)), torch.tensor(lens, dtype=torch.int32, device=DEV),
                            table.to(DEV), q.to(DEV), torch.full((B, 1), sign, device=DEV), idx, _junk_ws(dims, B))
    for b, v in enumerate(values):
        best = torch.sort(sign * v, descending=True, stable=True).indices[:k].sort().values
        want = torch.full((k,), -1, dtype=torch.int32)
        want[:len(best)] = best.to(torch.int32)
        assert torch.equal(idx[b].cpu(), want), b
    dsa.check_device_error()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("n,k", [(4095, 512), (4096, 512), (4097, 512), (4097, 1024), (20000, 1), (70000, 1024),
                                 (70000, 512)])
def test_topk_of_awkward_scores(n, k, sign):
    """Scores that rise or fall along the row, that sit in one stretch of it or at every 61st pool only (which evenly spaced
    samples misjudge), that tie in bulk just above or below the k-th, that span all magnitudes: always the exact selection."""
    g = torch.Generator().manual_seed(n + k)
    r = torch.rand(n, generator=g)
    ramp = torch.arange(n, dtype=torch.float32)
    stretch, comb, ties, few = r.clone(), r.clone(), torch.full((n,), 3.0), torch.full((n,), 3.0)
    stretch[n // 3:n // 3 + 2 * k] += 5.0
    comb[::61] += 7.0
    ties[torch.randperm(n, generator=g)[:k // 2]] = 4.0
    ties[torch.randperm(n, generator=g)[:n // 3]] = 1.0
    few[torch.randperm(n, generator=g)[:min(n, 2 * k)]] = 9.0
    wide = torch.exp(100.0 * (r - 0.5))
    near = 1.0 + torch.randint(0, 50, (n,), generator=g).float() * 2.0 ** -23
    _given_scores([r, ramp, ramp.flip(0), stretch, comb, ties, few, wide, near], k, sign)


def test_topk_of_one_row_of_awkward_scores():
    """The same kinds for one row on a cluster of 16 CTAs."""
    g = torch.Generator().manual_seed(8)
    n, k = 262144, 1024
    r = torch.rand(n, generator=g)
    comb, stretch, most = r.clone(), r.clone(), r.clone()
    comb[5::64] += 3.0          # 4096 pools, away from every sample
    stretch[200000:200000 + 5000] += 3.0
    most[:200000] = 2.0
    for v in (r, torch.arange(n, dtype=torch.float32), comb, stretch, most, torch.full((n,), 1.5)):
        _given_scores([v], k)


def test_topk_with_nan_and_infinite_scores_ends():
    """A NaN score has no rank, but the call ends, with pools of the row only, each at most once; infinities rank normally."""
    for n in (3000, 50000):
        v = torch.rand(n, generator=torch.Generator().manual_seed(3))
        v[7::n // 9] = math.inf
        _given_scores([v], 64)
        for bad in (v.clone(), torch.full((n,), math.nan)):
            bad[::2] = math.nan
            dims = dsa.make_dims(4 * n, 16, 128, 1, 64, 64, dtype="fp32")
            cols = -(-4 * n // 64)
            kpool = torch.zeros(cols, 16, 64)
            kpool.view(-1, 64)[:n, 0] = bad
            q = torch.zeros(1, 1, 64)
            q[0, 0, 0] = 1.0
            for w in (1.0, -1.0, math.nan):     # max(0, NaN) is 0 in the indexer: a NaN weight makes every score NaN
                idx = torch.full((1, 64), -9, dtype=torch.int32, device=DEV)
                dsa.decode_indexer_topk(dims, dsa.PagedCache(kpool=kpool.to(DEV)),
                                        torch.tensor([4 * n], dtype=torch.int32, device=DEV),
                                        torch.arange(cols, dtype=torch.int32, device=DEV)[None], q.to(DEV),
                                        torch.full((1, 1), w, device=DEV), idx, _junk_ws(dims, 1))
                got = idx[0].tolist()
                assert len(set(got)) == 64 and min(got) >= 0 and max(got) < n and got == sorted(got)
    dsa.check_device_error()


def test_indexer_topk_of_real_scores():
    """N(0,1) inputs: every row's selection is a top-k of the 64-bit scores up to their fp32 error."""
    pg = Paged([30001, 2053], 64, seed=12)
    pg.KI = [torch.randn(n, 64, generator=pg.g).to(torch.bfloat16) for n in pg.lens_list]
    pool = [x[:len(x) // 4 * 4].float().view(-1, 4, 64) for x in pg.KI]
    pool = [(((x[:, 0] + x[:, 1]) + x[:, 2]) + x[:, 3]).to(torch.bfloat16) for x in pool]
    pg.pool_keys = lambda b: pool[b]
    pg.fill()
    dims = dsa.make_dims(pg.cap, 16, 128, 8, 64, 256)
    lens, table = pg.args()
    q, w = torch.randn(2, 8, 64, generator=pg.g).to(torch.bfloat16), torch.rand(2, 8, generator=pg.g)
    idx = torch.empty(2, 256, dtype=torch.int32, device=DEV)
    dsa.decode_indexer_topk(dims, pg.cache(), lens, table, q.to(DEV), w.to(DEV), idx, _junk_ws(dims, 2))
    for b in range(2):
        dots = q[b].double() @ pool[b].double().T
        s = (dots.clamp(min=0) * w[b].double()[:, None]).sum(0)
        # 64 products and 8 heads in fp32
        err = ((64 + 12) * 2.0 ** -23 * (q[b].double().abs() @ pool[b].double().abs().T) * w[b].double()[:, None]).sum(0)
        got = idx[b].long().cpu()
        assert len(set(got.tolist())) == 256 and torch.equal(got, got.sort().values)
        out = torch.ones(len(s), dtype=torch.bool)
        out[got] = False
        assert (s + err)[got].min() >= (s - err)[out].max()
    dsa.check_device_error()


def test_indexer_topk_bad_pages_and_lengths():
    pg = Paged([400, 400, 400], 16, seed=5).fill()
    dims = dsa.make_dims(pg.cap, 16, 128, 8, 64, 20)
    lens, table = pg.args()
    q = torch.randint(-3, 4, (3, 8, 64), generator=pg.g).to(torch.bfloat16)
    w = torch.randint(1, 5, (3, 8), generator=pg.g).float()
    idx = torch.empty(3, 20, dtype=torch.int32, device=DEV)
    t, l = table.clone(), lens.clone()
    t[0, 3] = pg.pages
    l[2] = -1
    dsa.decode_indexer_topk(dims, pg.cache(), l, t, q.to(DEV), w.to(DEV), idx, _junk_ws(dims, 3))
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error()
    assert e.value.status == dsa.DSA_ERR_BAD_PAGE
    assert torch.equal(idx[1].cpu(), _ref_topk(pg, q, w, 20)[1])
    assert torch.all(idx[2] == -1)
    assert idx[0].min() >= 0 and idx[0].max() < 100


# ---------------------------------------------------------------- append
def _freq(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _rotate(x, pos, freq, interleaved):
    """x [n, ..., d] in 64 bits at positions pos [n]."""
    n = 2 * len(freq)
    a = pos.double()[:, None] * freq
    a = a.view(len(pos), *([1] * (x.dim() - 2)), len(freq))
    i = torch.arange(len(freq))
    re, im = (2 * i, 2 * i + 1) if interleaved else (i, i + n // 2)
    y = x.clone()
    y[..., re] = x[..., re] * a.cos() - x[..., im] * a.sin()
    y[..., im] = x[..., re] * a.sin() + x[..., im] * a.cos()
    return y


def _close_rotated(got, ref, dtype):
    """One rounding, and products with a sine and cosine off by 2^-21 (the angle's 2^-24 of at most half a turn, twice)."""
    got, ref = got.double().cpu(), ref.double()
    tol = HALF[dtype] * ref.abs() + 2.0 ** -20 * ref.abs().amax(-1, keepdim=True) * math.sqrt(2.0)
    assert torch.all((got - ref).abs() <= tol)


@pytest.mark.parametrize("dtype,Hq,d,di,page,rot,inter", [
    ("bf16", 16, 128, 64, 64, 0, False), ("bf16", 16, 128, 64, 16, 64, False), ("bf16", 5, 64, 128, 4, 64, True),
    ("bf16", 32, 128, 128, 100, 128, True), ("bf16", 1, 128, 64, 20, 16, False), ("bf16", 7, 64, 64, 12, 48, False),
    ("fp32", 8, 64, 64, 16, 64, False), ("fp32", 3, 128, 128, 4, 32, True), ("fp32", 2, 128, 64, 64, 0, False),
    ("fp32", 32, 128, 64, 12, 128, False)])
@pytest.mark.parametrize("far", [0, 1 << 20])
def test_append_in_ragged_pieces(dtype, Hq, d, di, page, rot, inter, far):
    """Sequences appended in uneven pieces (some empty, some of one token, some across several pages and pools), rows
    behind the last piece left alone; the cache equals the sequences, NaN where nothing was written.  far: positions
    behind a million tokens that are not in the cache (their table entries are never read)."""
    far = far // page // 4 * 4 * page if far else 0
    if far and page < 16:
        pytest.skip("a block table of that many tiny pages")
    total = [37, 0, 130, 64, 7]
    pg = Paged(total, page, d=d, di=di, dtype=dtype, seed=rot + page)
    if far:
        front = torch.full((len(total), far // page), -7, dtype=torch.int32)
        pg.table, pg.cap = torch.cat([front, pg.table], 1), pg.cap + far
    dims = dsa.make_dims(pg.cap, Hq, d, 8, di, 8, dtype=dtype)
    cache = pg.cache()
    table = pg.table.to(DEV)
    rotation = dsa.make_rotation(_freq(rot), interleaved=inter) if rot else None
    done = [0] * len(total)
    gq = torch.Generator().manual_seed(99)
    pieces = [[1, 0, 2, 4, 3], [2, 0, 1, 0, 0], [0] * 5, [5, 0, 60, 3, 1], [29, 0, 3, 57, 3], [0, 0, 64, 0, 0]]
    for piece in pieces:
        src = [slice(done[b], done[b] + n) for b, n in enumerate(piece)]
        done = [x + n for x, n in zip(done, piece)]
        T = sum(piece)
        pad = 3
        cat = lambda xs: torch.cat([x[s] for x, s in zip(xs, src)] + [torch.full((pad, xs[0].shape[1]), 7.0).to(pg.dt)])
        off = torch.tensor([0] + piece, dtype=torch.int32).cumsum(0).to(torch.int32)
        lens = torch.tensor([x + far if total[b] else 0 for b, x in enumerate(done)], dtype=torch.int32)
        kw = {}
        if rot:
            q = torch.randn(T + pad, Hq, d, generator=gq).to(pg.dt)
            kw = dict(rotation=rotation, q=q.to(DEV), q_out=torch.full((T + pad, Hq, d), 7.0, dtype=pg.dt, device=DEV),
                      k_out=torch.full((T + pad, d), 7.0, dtype=pg.dt, device=DEV))
        kn, vn, kin = cat(pg.K), cat(pg.V), cat(pg.KI)
        dsa.cache_append(dims, cache, lens.to(DEV), table, kn.to(DEV), vn.to(DEV), kin.to(DEV), offsets=off.to(DEV), **kw)
        if rot:
            pos = torch.cat([torch.arange(s.start, s.stop) for s in src]) + far
            if T:
                _close_rotated(kw["q_out"][:T], _rotate(q[:T].double(), pos, _freq(rot), inter), dtype)
                _close_rotated(kw["k_out"][:T], _rotate(kn[:T].double(), pos, _freq(rot), inter), dtype)
            assert torch.all(kw["q_out"][T:] == 7) and torch.all(kw["k_out"][T:] == 7)
    dsa.check_device_error()
    assert done == total
    seen_k, seen_p = torch.zeros(pg.pages, page, dtype=torch.bool), torch.zeros(pg.pages, page // 4, dtype=torch.bool)
    K, V, KP, KT = cache.k.cpu(), cache.v.cpu(), cache.kpool.cpu(), cache.ktail.cpu()
    for b, n in enumerate(total):
        if not n:
            continue
        at = far // page
        pos = torch.arange(n)
        w, r = pg.table[b, at + pos // page].long(), pos % page
        seen_k[w, r] = True
        assert torch.equal(V[w, r], pg.V[b])
        if rot:
            _close_rotated(K[w, r], _rotate(pg.K[b].double(), pos + far, _freq(rot), inter), dtype)
        else:
            assert torch.equal(K[w, r], pg.K[b])
        p = torch.arange(n // 4)
        w = pg.table[b, at + 4 * p // page].long()
        seen_p[w, p % (page // 4)] = True
        assert torch.equal(KP[w, p % (page // 4)], pg.pool_keys(b))
        if n % 4:
            assert torch.equal(KT[pg.table[b, at + (n - 1) // page].long(), :n % 4], pg.KI[b][n // 4 * 4:])
    assert torch.isnan(K[~seen_k]).all() and torch.isnan(V[~seen_k]).all() and torch.isnan(KP[~seen_p]).all()


@pytest.mark.parametrize("dtype,d,di,page", [("bf16", 128, 64, 64), ("bf16", 64, 128, 12), ("fp32", 128, 128, 16),
                                             ("fp32", 64, 64, 100)])
def test_append_long_prompts(dtype, d, di, page):
    """Prompts of more than 20000 tokens in all, behind starts of every remainder modulo 4, in two calls."""
    total = [9001, 1, 0, 6002, 3, 5003, 4000, 2]
    first = [1, 0, 0, 2, 1, 1003, 8, 1]
    pg = Paged(total, page, d=d, di=di, dtype=dtype, seed=d + di + page)
    dims = dsa.make_dims(pg.cap, 4, d, 8, di, 8, dtype=dtype)
    cache, table = pg.cache(), pg.table.to(DEV)
    for a, z in (([0] * 8, first), (first, total)):
        cat = lambda xs: torch.cat([x[i:j] for x, i, j in zip(xs, a, z)] + [torch.full((5, xs[0].shape[1]), 7.0).to(pg.dt)])
        off = torch.tensor([0] + [j - i for i, j in zip(a, z)], dtype=torch.int32).cumsum(0).to(torch.int32)
        dsa.cache_append(dims, cache, torch.tensor(z, dtype=torch.int32, device=DEV), table, cat(pg.K).to(DEV), cat(pg.V).to(DEV),
                         cat(pg.KI).to(DEV), offsets=off.to(DEV))
    dsa.check_device_error()
    want = Paged(total, page, d=d, di=di, dtype=dtype, seed=d + di + page).fill()
    for got, ref in ((cache.k, want.k_c), (cache.v, want.v_c), (cache.kpool, want.kp_c)):
        got, ref = got.cpu(), ref
        assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(got.nan_to_num(), ref.nan_to_num())
    for b, n in enumerate(total):
        if n % 4:
            assert torch.equal(cache.ktail.cpu()[pg.table[b, (n - 1) // page].long(), :n % 4], pg.KI[b][n // 4 * 4:])


def test_cache_beyond_32_bit_offsets():
    """A cache of 20 million tokens: the rows' pages lie beyond element 2^31 of K and V (byte 2^32), and everything agrees
    with the same rows in a small cache."""
    page, pages = 64, 320000
    small = Paged([900, 333], page, seed=90)
    dims = dsa.make_dims(small.cap, 16, 128, 8, 64, 20)
    shift = pages - small.pages
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)
    big = dsa.PagedCache(k=e(pages, page, 128), v=e(pages, page, 128), kpool=e(pages, page // 4, 64), ktail=e(pages, 3, 64))
    lens, table = small.args()
    cat = lambda xs: torch.cat(xs).to(DEV)
    q = torch.randn(2, 16, 128, generator=small.g).to(torch.bfloat16).to(DEV)
    qi = torch.randint(-3, 4, (2, 8, 64), generator=small.g).to(torch.bfloat16).to(DEV)
    w = torch.rand(2, 8, generator=small.g).to(DEV)
    res = []
    for cache, t in ((small.cache(), table), (big, table + shift)):
        dsa.cache_append(dims, cache, lens, t, cat(small.K), cat(small.V), cat(small.KI),
                         offsets=torch.tensor([0, 900, 1233], dtype=torch.int32, device=DEV))
        ws, idx = _junk_ws(dims, 2), torch.empty(2, 20, dtype=torch.int32, device=DEV)
        o, lse = (torch.empty_like(q), torch.empty_like(q)), (torch.empty(2, 16, device=DEV), torch.empty(2, 16, device=DEV))
        dsa.decode_indexer_topk(dims, cache, lens, t, qi, w, idx, ws)
        dsa.decode_attn(dims, cache, lens, t, q, o[0], lse[0], ws, idx=idx)
        dsa.decode_attn(dims, cache, lens, t, q, o[1], lse[1], ws)
        res.append((idx, *o, *lse))
    dsa.check_device_error()
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_append_pool_keys_round_as_pool_keys_does():
    """Real-valued keys: pool keys formed across appends are dsa.pool_keys' bit for bit."""
    n, page = 403, 16
    pg = Paged([n], page, di=128, seed=21)
    ki = (torch.randn(n, 128, generator=pg.g) * 3).to(torch.bfloat16)
    dims = dsa.make_dims(pg.cap, 16, 128, 8, 128, 8)
    cache, table, at = pg.cache(), pg.table.to(DEV), 0
    for m in (1, 2, 5, 1, 1, 1, 1, 300, 6, 85):
        lens = torch.tensor([at + m], dtype=torch.int32, device=DEV)
        off = torch.tensor([0, m], dtype=torch.int32, device=DEV)
        dsa.cache_append(dims, cache, lens, table, pg.K[0][at:at + m].to(DEV), pg.V[0][at:at + m].to(DEV),
                         ki[at:at + m].to(DEV), offsets=off)
        at += m
    assert at == n
    want = torch.empty(n // 4, 128, dtype=torch.bfloat16, device=DEV)
    dsa.pool_keys(dsa.make_dims(n // 4 * 4, 16, 128, 8, 128, 8), ki[:n // 4 * 4].to(DEV), want)
    p = torch.arange(n // 4)
    got = cache.kpool.cpu()[pg.table[0, 4 * p // page].long(), p % (page // 4)]
    assert torch.equal(got, want.cpu())
    dsa.check_device_error()


def test_append_in_place_rotation_and_idle_rows():
    """q_out = q and k_out = k; without offsets, idle rows append nothing and their q is left alone."""
    pg = Paged([9, 0, 4, 130], 16, seed=31).fill()
    dims = dsa.make_dims(pg.cap, 16, 128, 8, 64, 8)
    lens, table = pg.args()
    rot = dsa.make_rotation(_freq(64))
    k, v = (torch.randn(4, 128, generator=pg.g).to(torch.bfloat16) for _ in range(2))
    ki = torch.randint(-3, 4, (4, 64), generator=pg.g).to(torch.bfloat16)
    q = torch.randn(4, 16, 128, generator=pg.g).to(torch.bfloat16)
    kd, qd, cache = k.to(DEV), q.to(DEV), pg.cache()
    dsa.cache_append(dims, cache, lens, table, kd, v.to(DEV), ki.to(DEV), rotation=rot, q=qd, q_out=qd, k_out=kd)
    pos = lens.cpu().long() - 1
    for b in (0, 2, 3):
        _close_rotated(qd[b:b + 1], _rotate(q[b:b + 1].double(), pos[b:b + 1], _freq(64), False), "bf16")
        _close_rotated(kd[b:b + 1], _rotate(k[b:b + 1].double(), pos[b:b + 1], _freq(64), False), "bf16")
        w, r = pg.where(b, pos[b])
        assert torch.equal(cache.k[w, r], kd[b]) and torch.equal(cache.v[w, r].cpu(), v[b])
    assert torch.equal(qd[1].cpu(), q[1]) and torch.equal(kd[1].cpu(), k[1])
    dsa.check_device_error()


def test_append_skips_and_reports_bad_rows():
    pg = Paged([9, 20, 4, 130, 8], 16, seed=33)
    dims = dsa.make_dims(pg.cap, 16, 128, 8, 64, 8)
    k = torch.randn(5, 128, generator=pg.g).to(torch.bfloat16).to(DEV)
    ki = torch.ones(5, 64, dtype=torch.bfloat16, device=DEV)
    lens, table = pg.args()
    l, t = lens.clone(), table.clone()
    l[0], l[3], t[1, 1] = pg.cap + 1, -2, pg.pages
    cache = pg.cache()
    dsa.cache_append(dims, cache, l, t, k, k, ki)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_device_error()
    assert e.value.status == dsa.DSA_ERR_BAD_PAGE
    written = ~torch.isnan(cache.k.float()).any(-1)
    assert int(written.sum()) == 2          # rows 2 and 4
    for off in ([-1, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 9], [0, 12, 12, 12, 12, 12]):
        cache = pg.cache()
        dsa.cache_append(dims, cache, lens, table, k, k, ki, offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
        with pytest.raises(dsa.DSAError) as e:
            dsa.check_device_error()
        assert e.value.status == dsa.DSA_ERR_BAD_PAGE


# ---------------------------------------------------------------- the calls together
@pytest.mark.parametrize("dtype,Hq,rot", [("bf16", 16, 0), ("bf16", 32, 64), ("fp32", 8, 0)])
def test_decoding_continues_the_layer(dtype, Hq, rot):
    """Two prompts enter the cache in chunks, then tokens are decoded one by one; the selections equal those of dsa.layer_fwd
    on the whole sequences and the outputs meet the same exact values."""
    d, di, Hi, k, page, L = 128, 64, 8, 20, 16, 240
    prompt = [121, 57]
    n = [L, L - 64]
    pg = Paged(n, page, d=d, di=di, dtype=dtype, seed=Hq + rot, cap=L)
    g = pg.g
    Q = [torch.randn(m, Hq, d, generator=g).to(pg.dt) for m in n]
    QI = [torch.randint(-3, 4, (m, Hi, di), generator=g).to(pg.dt) for m in n]
    W = [torch.randint(1, 5, (m, Hi), generator=g).float() for m in n]
    dims = dsa.make_dims(L, Hq, d, Hi, di, k, dtype=dtype)
    rotation = dsa.make_rotation(_freq(rot)) if rot else None
    cache, table, ws = pg.cache(), pg.table.to(DEV), _junk_ws(dims, 2)
    done = [0, 0]
    KR, QR = [[], []], [[], []]
    for cut in ([50, 57], prompt):
        off = torch.tensor([0, cut[0] - done[0], cut[0] - done[0] + cut[1] - done[1]], dtype=torch.int32)
        cat = lambda xs: torch.cat([x[a:z] for x, a, z in zip(xs, done, cut)]).to(DEV)
        kw = {}
        if rot:
            q = cat(Q)
            kw = dict(rotation=rotation, q=q, q_out=q, k_out=torch.empty(q.shape[0], d, dtype=pg.dt, device=DEV))
        dsa.cache_append(dims, cache, torch.tensor(cut, dtype=torch.int32, device=DEV), table, cat(pg.K), cat(pg.V),
                         cat(pg.KI), offsets=off.to(DEV), **kw)
        if rot:
            for b in range(2):
                s = slice(int(off[b]), int(off[b + 1]))
                KR[b].append(kw["k_out"][s].cpu())
                QR[b].append(kw["q_out"][s].cpu())
        done = list(cut)
    # what layer_fwd sees: the keys and queries as rotated (and rounded) once
    if rot:
        pos = [torch.arange(p, m) for p, m in zip(prompt, n)]
        for b in range(2):
            KR[b].append(_rotate(pg.K[b][prompt[b]:].double(), pos[b], _freq(rot), False).to(pg.dt))
            QR[b].append(_rotate(Q[b][prompt[b]:].double(), pos[b], _freq(rot), False).to(pg.dt))
        kr, qr = [torch.cat(x) for x in KR], [torch.cat(x) for x in QR]
    else:
        kr, qr = pg.K, Q
    want_idx = []
    for b in range(2):
        dl = dsa.make_dims(n[b], Hq, d, Hi, di, k, dtype=dtype)
        bufs = dsa.alloc_forward_buffers(dl)
        dsa.layer_fwd(dl, qr[b].to(DEV), kr[b].to(DEV), pg.V[b].to(DEV), QI[b].to(DEV), pg.KI[b].to(DEV), W[b].to(DEV), bufs.o,
                      bufs.lse, bufs.idx, bufs.kpool, bufs.ws)
        want_idx.append(bufs.idx.cpu())
    ref = Paged.__new__(Paged)
    ref.dtype, ref.K, ref.V = dtype, kr, pg.V
    o, lse = torch.empty(2, Hq, d, dtype=pg.dt, device=DEV), torch.empty(2, Hq, device=DEV)
    idx = torch.empty(2, k, dtype=torch.int32, device=DEV)
    for step in range(max(m - p for m, p in zip(n, prompt))):
        live = [p + step < m for p, m in zip(prompt, n)]
        at = [min(p + step, m - 1) for p, m in zip(prompt, n)]
        lens = torch.tensor([a + 1 if x else 0 for a, x in zip(at, live)], dtype=torch.int32, device=DEV)
        row = lambda xs: torch.stack([x[a] for x, a in zip(xs, at)]).to(DEV)
        dsa.decode_step(dims, cache, lens, table, row(Q), row(pg.K), row(pg.V), row(QI), row(pg.KI), row(W), o, lse, idx, ws,
                        rotation=rotation)
        for b in range(2):
            if not live[b]:
                assert torch.all(idx[b] == -1) and torch.all(o[b] == 0)
                continue
            assert torch.equal(idx[b].cpu(), want_idx[b][at[b]])
        ref.lens_list = lens.tolist()
        if rot:   # the step's own rotations may round the last bit otherwise: compare against what the cache holds
            ref.K = [torch.cat([cache.k.cpu()[pg.table[b].long()].flatten(0, 1)[:n[b]]]) for b in range(2)]
            q_now = torch.stack([x[a] for x, a in zip(qr, at)])
            _check_attn_loose(ref, q_now, o, lse, d ** -0.5, idx.cpu(), dtype)
        else:
            _check_attn(ref, row(Q).cpu(), o, lse, d ** -0.5, idx.cpu())
    dsa.check_device_error()


def _check_attn_loose(pg, q, o, lse, scale, idx, dtype):
    """As _check_attn, for a query whose rotation may have rounded the other way: one step of the type per channel moves a
    score by at most 2 u scale sum |q k|, and a weight by twice that."""
    for b in range(q.shape[0]):
        rows = pg.keys(b, idx)
        if not rows:
            continue
        k, v, qq = pg.K[b][rows].double(), pg.V[b][rows].double(), q[b].double()
        s = qq @ k.T * scale
        l = torch.logsumexp(s, -1)
        p = (s - l[:, None]).exp()
        ds = 2.01 * HALF[dtype] * scale * (qq.abs() @ k.abs().T).amax(-1)
        tol = (4 * ds[:, None] + 2.0 ** -14) * (p @ v.abs()) + HALF[dtype] * (p @ v).abs()
        assert torch.all((o[b].double().cpu() - p @ v).abs() <= tol)
        assert torch.all((lse[b].double().cpu() - l).abs() <= 2 * ds + 2.0 ** -14)


def test_cutting_back_to_a_pool_boundary():
    """Rejected draft tokens: the length goes back to a multiple of 4 and the tokens after it are appended again."""
    pg = Paged([41], 16, seed=40)
    dims = dsa.make_dims(pg.cap, 16, 128, 8, 64, 8)
    cache, table = pg.cache(), pg.table.to(DEV)

    def put(a, z, ki):
        dsa.cache_append(dims, cache, torch.tensor([z], dtype=torch.int32, device=DEV), table, pg.K[0][a:z].to(DEV),
                         pg.V[0][a:z].to(DEV), ki[a:z].to(DEV), offsets=torch.tensor([0, z - a], dtype=torch.int32, device=DEV))
    wrong = torch.full_like(pg.KI[0], 100.0)
    put(0, 30, pg.KI[0])
    put(30, 39, wrong)
    put(28, 33, pg.KI[0])
    put(33, 41, pg.KI[0])
    p = torch.arange(10)
    assert torch.equal(cache.kpool.cpu()[pg.table[0, 4 * p // 16].long(), p % 4], pg.pool_keys(0))
    dsa.check_device_error()


def test_graph_replay_streams_and_reproducibility():
    """A captured step replays with other lengths and tables; two captured graphs with workspaces of their own run side by
    side on two streams; the results equal the eager ones bit for bit."""
    pg = Paged([700, 33, 0, 1029], 16, seed=50, cap=2048).fill()
    B, Hq, d, k = 4, 16, 128, 24
    dims = dsa.make_dims(pg.cap, Hq, d, 8, 64, k)
    lens, table = pg.args()
    lens0 = lens.clone()
    q = torch.randn(B, Hq, d, generator=pg.g).to(torch.bfloat16).to(DEV)
    qi = torch.randint(-3, 4, (B, 8, 64), generator=pg.g).to(torch.bfloat16).to(DEV)
    w = torch.rand(B, 8, generator=pg.g).to(DEV)
    cache = pg.cache()

    def outs():
        return (torch.empty(B, Hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(B, Hq, device=DEV),
                torch.empty(B, k, dtype=torch.int32, device=DEV), _junk_ws(dims, B))

    def run(o, lse, idx, ws, dense):
        dsa.decode_indexer_topk(dims, cache, lens, table, qi, w, idx, ws)
        dsa.decode_attn(dims, cache, lens, table, q, o, lse, ws, idx=None if dense else idx)

    sets = [outs(), outs()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    for i in range(2):
        run(*sets[i], dense=i == 1)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            run(*sets[i], dense=i == 1)
        graphs.append(gr)
    for trial in range(3):
        lens.copy_(lens0 if trial == 0 else (lens0 // (trial + 1)).to(torch.int32))
        torch.cuda.synchronize()
        for _ in range(5):
            for gr, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    gr.replay()
        torch.cuda.synchronize()
        for i in range(2):
            e = outs()
            run(*e, dense=i == 1)
            for a, c in zip(sets[i][:3], e[:3]):
                assert torch.equal(a, c)
        pg.lens_list = lens.tolist()
        _check_attn(pg, q.cpu(), sets[0][0], sets[0][1], d ** -0.5, sets[0][2].cpu())
        _check_attn(pg, q.cpu(), sets[1][0], sets[1][1], d ** -0.5)
    dsa.check_device_error()


def test_calls_wait_for_what_comes_before_them():
    """Kernels may become resident before their predecessors end; what they read and overwrite is still ordered: inputs that
    a kernel just before the call writes, outputs that a kernel just after it reads, one workspace for all calls, appends
    that the next call reads; the same with the device held up between calls gives the same bits."""
    def run(held):
        pg = Paged([400, 77, 1201, 9], 16, seed=51, cap=1400).fill()
        B, Hq, d, k = 4, 16, 128, 24
        dims = dsa.make_dims(pg.cap, Hq, d, 8, 64, k)
        cols = -(-pg.cap // 16)
        lens, _ = pg.args()
        spare = torch.arange(pg.pages, pg.pages + B * cols, dtype=torch.int32).view(B, cols)
        table = torch.where(pg.table >= 0, pg.table, spare).to(DEV)
        grow = lambda t: torch.cat([t, torch.zeros(B * cols, *t.shape[1:], dtype=t.dtype)]).to(DEV)
        cache = dsa.PagedCache(k=grow(pg.k_c), v=grow(pg.v_c), kpool=grow(pg.kp_c), ktail=grow(pg.kt_c))
        g = torch.Generator(device=DEV).manual_seed(5)
        rn = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
        ws, rot = _junk_ws(dims, B), dsa.make_rotation(_freq(64))
        o, o2 = rn(B, Hq, d), rn(B, Hq, d)
        lse, idx = torch.zeros(B, Hq, device=DEV), torch.zeros(B, k, dtype=torch.int32, device=DEV)
        q, kk, v, qi, ki, w = rn(B, Hq, d), rn(B, d), rn(B, d), rn(B, 8, 64), rn(B, 64), torch.rand(B, 8, generator=g, device=DEV)
        seen = []
        wait = torch.cuda.synchronize if held else lambda: None
        for step in range(40):
            lens.add_(1)
            wait()
            q.mul_(0.75).add_(o, alpha=0.25)
            wait()
            dsa.decode_step(dims, cache, lens, table, q, kk, v, qi, ki, w, o, lse, idx, ws, rotation=rot)
            wait()
            dsa.decode_attn(dims, cache, lens, table, o, o2, lse, ws)
            wait()
            kk.copy_(o2[:, step % Hq])
            seen.append((o.clone(), o2.clone(), lse.clone(), idx.clone()))
            wait()
        dsa.check_device_error()
        return seen
    for a, b in zip(run(False), run(True)):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_capture_across_streams():
    """A graph whose calls depend on other streams' work: what one stream computes, another stream's calls read."""
    pg = Paged([700, 33, 0, 1029], 16, seed=52).fill()
    B, Hq, d, k = 4, 16, 128, 24
    dims = dsa.make_dims(pg.cap, Hq, d, 8, 64, k)
    lens, table = pg.args()
    cache, ws, ws2 = pg.cache(), _junk_ws(dims, B), _junk_ws(dims, B)
    src = torch.randn(B, Hq, d, generator=pg.g).to(DEV)
    q = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device=DEV)
    qi = torch.randint(-3, 4, (B, 8, 64), generator=pg.g).to(torch.bfloat16).to(DEV)
    w = torch.rand(B, 8, generator=pg.g).to(DEV)
    out = [(torch.zeros_like(q), torch.zeros(B, Hq, device=DEV)) for _ in range(2)]
    idx = torch.zeros(B, k, dtype=torch.int32, device=DEV)
    total = torch.zeros(B, Hq, d, device=DEV)

    def work(main, side):
        q.copy_(src)
        ready = torch.cuda.Event()
        ready.record(main)
        with torch.cuda.stream(side):
            side.wait_event(ready)
            dsa.decode_attn(dims, cache, lens, table, q, *out[1], ws2)
            done = torch.cuda.Event()
            done.record(side)
        dsa.decode_indexer_topk(dims, cache, lens, table, qi, w, idx, ws)
        dsa.decode_attn(dims, cache, lens, table, q, *out[0], ws, idx=idx)
        main.wait_event(done)
        total.copy_(out[0][0].float() + out[1][0].float())

    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        work(main, side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        work(main, side)
    for trial in range(3):
        src.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        got = total.clone(), idx.clone(), out[1][1].clone()
        with torch.cuda.stream(main):
            work(main, side)
        torch.cuda.synchronize()
        assert torch.equal(got[0], total) and torch.equal(got[1], idx) and torch.equal(got[2], out[1][1])
        _check_attn(pg, q.cpu(), *out[1], d ** -0.5)
        _check_attn(pg, q.cpu(), *out[0], d ** -0.5, idx.cpu())
    dsa.check_device_error()


def test_rows_may_share_pages():
    """Three rows of one sequence at growing lengths (a draft being verified), over one block-table row each."""
    pg = Paged([301], 16, seed=60).fill()
    pg.lens_list, pg.table = [299, 300, 301], pg.table.repeat(3, 1)
    pg.K, pg.V, pg.KI = pg.K * 3, pg.V * 3, pg.KI * 3
    q, o, lse = _attn(pg, 16, 128)
    _check_attn(pg, q, o, lse, 128 ** -0.5)
    qi, w, idx = _topk(pg, 8, 64, 10)
    assert torch.equal(idx.cpu(), _ref_topk(pg, qi, w, 10))


def test_binding_refuses_what_it_cannot_pass_on():
    pg = Paged([100, 60], 16, seed=70).fill()
    dims = dsa.make_dims(pg.cap, 16, 128, 8, 64, 8)
    lens, table = pg.args()
    cache, ws = pg.cache(), _junk_ws(dims, 2)
    q = torch.zeros(2, 16, 128, dtype=torch.bfloat16, device=DEV)
    o, lse = torch.zeros_like(q), torch.zeros(2, 16, device=DEV)
    good = dict(dims=dims, cache=cache, lens=lens, block_table=table, q=q, o=o, lse=lse, ws=ws)
    dsa.decode_attn(**good)
    for bad in (dict(lens=lens.long()), dict(lens=lens.cpu()), dict(block_table=table[:, :-1]), dict(block_table=table.T),
                dict(q=q.float()), dict(q=q[:1]), dict(q=q.transpose(1, 2)), dict(o=o[:, :8]), dict(lse=lse.double()),
                dict(q=torch.zeros(2, 32, 128, dtype=torch.bfloat16, device=DEV)[:, ::2]), dict(idx=torch.zeros(2, 8, device=DEV)),
                dict(idx=torch.zeros(2, 9, dtype=torch.int32, device=DEV)), dict(ws=ws[::2]),
                dict(dims=dsa.make_dims(pg.cap, 16, 64, 8, 64, 8)), dict(dims=dsa.make_dims(pg.cap, 16, 128, 8, 64, 8, dtype="fp32"))):
        with pytest.raises(ValueError):
            dsa.decode_attn(**{**good, **bad})
    with pytest.raises(dsa.DSAError) as e:
        dsa.decode_attn(**{**good, "ws": None})
    assert e.value.status == dsa.DSA_ERR_WORKSPACE
    with pytest.raises(dsa.DSAError) as e:
        dsa.decode_attn(**{**good, "q": torch.zeros(2 * 16 * 128 + 8, dtype=torch.bfloat16, device=DEV)[4:-4].view(2, 16, 128)})
    assert e.value.status == dsa.DSA_ERR_INVALID_ARG      # 8 bytes off a 16-byte boundary
    dsa.check_device_error()
