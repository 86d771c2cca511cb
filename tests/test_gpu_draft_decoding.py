"""Draft trees as a decoder uses them: heads normalised and rotated to their places in the tree, pools selected for every
node, the trees attended to, an accepted path committed to pages that were reserved for it; sequences forked, released and
compacted on the way.  The sequences' own contiguous copies in 64 bits say what every node has to see.  The steps of one test
are calls, those of the other replays of one captured graph.  Tolerances: those of test_gpu_decode."""
import math
import os
import random
import subprocess
import sys

import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from test_gpu_decode import DEV, HALF, _built, _check_attn, _dt, _freq, _junk_ws  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Decoder:
    B, N, PAGE, D, DI, HI = 3, 7, 16, 128, 64, 8

    def __init__(self, dtype, Hq, k, seed, pages=60, L=512):
        self.dtype, self.Hq, self.k, self.dt, self.L = dtype, Hq, k, _dt(dtype), L
        self.g, self.r = torch.Generator().manual_seed(seed), random.Random(seed)
        self.dims = dsa.make_dims(L, Hq, self.D, self.HI, self.DI, k, dtype=dtype)
        self.cache = dsa.alloc_paged_cache(self.dims, pages, self.PAGE)
        for x in (self.cache.k, self.cache.v, self.cache.kpool, self.cache.ktail):
            x.fill_(math.nan)
        self.refs = _i32([0] * pages)
        B, T, cols = self.B, self.B * self.N, -(-L // self.PAGE)
        self.lens, self.new_lens, self.table = _i32([0] * B), _i32([0] * B), _i32([[-1] * cols] * B)
        self.missing = _i32([0])
        self.rot = dsa.make_rotation(_freq(64))
        self.qw, self.kw = (1 + 0.2 * torch.randn(self.D, generator=self.g)).to(DEV), (1 + 0.2 * torch.randn(self.D, generator=self.g)).to(DEV)
        e = lambda *s, dt=self.dt: torch.zeros(*s, dtype=dt, device=DEV)  # noqa: E731
        self.q, self.kk, self.v, self.ki, self.qi = e(T, Hq, self.D), e(T, self.D), e(T, self.D), e(T, self.DI), e(T, self.HI, self.DI)
        self.w = e(T, self.HI, dt=torch.float32)
        self.qr, self.kr = torch.zeros_like(self.q), torch.zeros_like(self.kk)
        self.o, self.lse, self.idx = torch.zeros_like(self.q), e(T, Hq, dt=torch.float32), e(T, k, dt=torch.int32)
        self.parents, self.depth, self.accepted = e(T, dt=torch.int32), e(T, dt=torch.int32), e(B, dt=torch.int32)
        self.offsets, self.row = _i32([self.N * b for b in range(B + 1)]), torch.arange(T, device=DEV) // self.N
        self.ws, self.pws = dsa.alloc_tree_workspace(self.dims, B, T), dsa.alloc_page_workspace(self.dims, self.cache, B)
        self.iws = _junk_ws(self.dims, T)
        self.K, self.V, self.KI = ([torch.zeros(0, n, dtype=torch.float64) for _ in range(B)] for n in (self.D, self.D, self.DI))

    def prompt(self, lens):
        n = sum(lens)
        k, v, ki = (torch.randn(n, self.D, generator=self.g).to(self.dt), torch.randn(n, self.D, generator=self.g).to(self.dt),
                    torch.randint(-3, 4, (n, self.DI), generator=self.g).to(self.dt))
        kd = k.to(DEV)
        dsa.qk_norm_rotate(self.dims, None, kd, None, kd, 1e-6, k_weight=self.kw, rotation=self.rot,
                           positions=_i32([i for m in lens for i in range(m)]))
        new = _i32(lens)
        dsa.cache_reserve(self.dims, self.cache, self.refs, self.lens, new, self.table, self.missing, self.pws)
        dsa.cache_append(self.dims, self.cache, new, self.table, kd, v.to(DEV), ki.to(DEV),
                         offsets=_i32([sum(lens[:b]) for b in range(self.B + 1)]))
        self.lens.copy_(new)
        k, at = kd.double().cpu(), 0
        for b, m in enumerate(lens):
            self.K[b], self.V[b], self.KI[b] = k[at:at + m], v[at:at + m].double(), ki[at:at + m].double()
            at += m
        assert self.missing.item() == 0

    def draw(self):
        """New drafts into the step's buffers; returns the accepted nodes and the trees."""
        g = self.g
        up = [[self.r.randint(max(-1, i - 3), i - 1) for i in range(self.N)] for _ in range(self.B)]
        deep = []
        for row in up:
            d = []
            for p in row:
                d.append(1 if p < 0 else d[p] + 1)
            deep.append(d)
        acc = [self.r.randint(-1, self.N - 1) for _ in range(self.B)]
        for x in (self.q, self.kk, self.v):
            x.copy_(torch.randn(x.shape, generator=g))
        self.ki.copy_(torch.randint(-3, 4, self.ki.shape, generator=g))
        self.qi.copy_(torch.randint(-3, 4, self.qi.shape, generator=g))
        self.w.copy_(torch.randint(1, 5, self.w.shape, generator=g))
        self.parents.copy_(_i32([p for row in up for p in row]))
        self.depth.copy_(_i32([d for row in deep for d in row]))
        self.accepted.copy_(_i32(acc))
        grow = [deep[b][a] if a >= 0 else 0 for b, a in enumerate(acc)]
        self.grow = _i32(grow) if not hasattr(self, "grow") else self.grow.copy_(_i32(grow))
        return up, acc

    def step(self):
        lens = self.lens[self.row]
        dsa.qk_norm_rotate(self.dims, self.q, self.kk, self.qr, self.kr, 1e-6, q_weight=self.qw, k_weight=self.kw,
                           rotation=self.rot, positions=lens + self.depth - 1)
        dsa.decode_indexer_topk(self.dims, self.cache, lens, self.table[self.row], self.qi, self.w, self.idx, self.iws)
        dsa.decode_tree_attn(self.dims, self.cache, self.lens, self.table, self.offsets, self.parents, self.qr, self.kr, self.v,
                             self.o, self.lse, self.ws, idx=self.idx)
        torch.add(self.lens, self.grow, out=self.new_lens)
        dsa.cache_reserve(self.dims, self.cache, self.refs, self.lens, self.new_lens, self.table, self.missing, self.pws)
        dsa.cache_commit(self.dims, self.cache, self.lens, self.table, self.offsets, self.parents, self.accepted, self.kr, self.v,
                         self.ki, self.lens)

    def check(self, up, acc):
        """What the last step computed, and what it added."""
        dsa.check_device_error()
        assert self.missing.item() == 0
        qr, kr, v, ki = (x.double().cpu() for x in (self.qr, self.kr, self.v, self.ki))
        qi, w, idx = self.qi.double().cpu(), self.w.double().cpu(), self.idx.cpu()
        o, lse, scale = self.o.double().cpu(), self.lse.double().cpu(), self.dims.scale
        for b in range(self.B):
            n = len(self.K[b])
            pools = self.KI[b][:n // 4 * 4].view(-1, 4, self.DI).sum(1)
            for i in range(self.N):
                t = b * self.N + i
                s = ((qi[t] @ pools.T).clamp(min=0) * w[t][:, None]).sum(0)
                best = sorted(range(len(s)), key=lambda p: (-s[p].item(), p))[:self.k]
                assert idx[t].tolist() == sorted(best) + [-1] * (self.k - len(best))
                line, j = [], i
                while j >= 0:
                    line.insert(0, b * self.N + j)
                    j = up[b][j]
                at = [4 * p + j for p in sorted(best) for j in range(4)] + list(range(n // 4 * 4, n))
                k, vv = torch.cat([self.K[b][at], kr[line]]), torch.cat([self.V[b][at], v[line]])
                z = qr[t] @ k.T * scale
                ref_l = torch.logsumexp(z, -1)
                p = (z - ref_l[:, None]).exp()
                ref = p @ vv
                ds = (self.D + 4) * 2.0 ** -23 * scale * (qr[t].abs() @ k.abs().T).amax(-1)
                tol = (4 * ds[:, None] + 2.0 ** -18 + len(k) * 2.0 ** -23) * (p @ vv.abs()) + HALF[self.dtype] * ref.abs()
                if self.dtype == "bf16":
                    tol += 2.0 ** -16 * (p @ vv.abs())
                assert torch.all((o[t] - ref).abs() <= tol)
                assert torch.all((lse[t] - ref_l).abs() <= 2 * ds + 2.0 ** -20 + len(k) * 2.0 ** -23 + 2.0 ** -22 * ref_l.abs())
                if i == acc[b]:
                    taken = line
            if acc[b] >= 0:
                self.K[b], self.V[b] = torch.cat([self.K[b], kr[taken]]), torch.cat([self.V[b], v[taken]])
                self.KI[b] = torch.cat([self.KI[b], ki[taken]])
        assert self.lens.tolist() == [len(x) for x in self.K]

    def check_pages(self):
        """The counts are the tables', and every sequence lies in its pages as its own copy has it."""
        names = {}
        for p in self.table.flatten().tolist():
            if p >= 0:
                names[p] = names.get(p, 0) + 1
        assert {p: c for p, c in enumerate(self.refs.tolist()) if c} == names
        kc, vc, kp, kt = (x.double().cpu() for x in (self.cache.k, self.cache.v, self.cache.kpool, self.cache.ktail))
        for b in range(self.B):
            n = len(self.K[b])
            pos, done = torch.arange(n), torch.arange(n // 4)
            row = self.table[b].cpu().long()
            assert torch.equal(kc[row[pos // self.PAGE], pos % self.PAGE], self.K[b])
            assert torch.equal(vc[row[pos // self.PAGE], pos % self.PAGE], self.V[b])
            assert torch.equal(kp[row[4 * done // self.PAGE], done % (self.PAGE // 4)],
                               self.KI[b][:n // 4 * 4].view(-1, 4, self.DI).sum(1).to(self.dt).double())
            if n % 4:
                assert torch.equal(kt[row[(n - 1) // self.PAGE], :n % 4], self.KI[b][n // 4 * 4:])

    def fork(self, parents):
        lens, table = torch.zeros_like(self.lens), torch.zeros_like(self.table)
        dsa.cache_fork(self.dims, self.cache, self.refs, self.lens, self.table, _i32(parents), lens, table)
        dsa.cache_release(self.dims, self.cache, self.refs, self.lens, self.table)
        self.lens.copy_(lens)
        self.table.copy_(table)
        self.K, self.V, self.KI = ([x[p].clone() for p in parents] for x in (self.K, self.V, self.KI))

    def compact(self):
        remap, used = torch.zeros_like(self.refs), _i32([0])
        dsa.cache_compact(self.dims, self.cache, self.refs, self.lens, self.table, remap, used, self.pws)
        dsa.check_device_error()
        assert int((self.refs[:used.item()] > 0).sum()) == used.item() and not torch.any(self.refs[used.item():])


@pytest.mark.parametrize("dtype,Hq,k", [("bf16", 16, 9), ("bf16", 32, 64), ("fp32", 8, 9)])
def test_decoding_with_draft_trees(dtype, Hq, k):
    d = Decoder(dtype, Hq, k, seed=Hq + k)
    d.prompt([61, 0, 130])
    for i in range(10):
        if i == 3:
            d.fork([0, 0, 2])      # the empty row becomes a branch of the first
        if i == 5:
            d.compact()
        if i == 7:
            d.fork([2, 1, 2])
        up, acc = d.draw()
        d.step()
        d.check(up, acc)
        d.check_pages()
    # the whole cache, by the call that takes one token a row
    q = torch.randn(3, Hq, d.D, generator=d.g).to(d.dt)
    o, lse = torch.zeros(3, Hq, d.D, dtype=d.dt, device=DEV), torch.zeros(3, Hq, device=DEV)
    dsa.decode_attn(d.dims, d.cache, d.lens, d.table, q.to(DEV), o, lse, _junk_ws(d.dims, 3))

    class View:
        K, V, keys = d.K, d.V, staticmethod(lambda b, idx=None: list(range(len(d.K[b]))))
    View.dtype = dtype
    _check_attn(View, q, o, lse, d.dims.scale)


@pytest.mark.parametrize("lens", [[61, 23, 130], [64, 3, 95]])
def test_rows_cut_back_grow_again(lens):
    """A row goes back to the end of a pool, to a place within its open pool, or to a page's end: the pages behind are given back,
    and the pools completed later are those of the tokens that are there."""
    d = Decoder("bf16", 16, 9, seed=sum(lens))
    d.prompt(lens)
    for i in range(3):
        up, acc = d.draw()
        d.step()
        d.check(up, acc)
        n = [len(x) for x in d.K]
        keep = [max(0, n[0] // 4 * 4 - 8 * i), n[1] // 4 * 4 + n[1] % 4 // 2, n[2] // 16 * 16]
        dsa.cache_release(d.dims, d.cache, d.refs, d.lens, d.table, keep=_i32(keep))
        d.lens.copy_(_i32(keep))
        d.K, d.V, d.KI = ([x[:m] for x, m in zip(y, keep)] for y in (d.K, d.V, d.KI))
        d.check_pages()
    up, acc = d.draw()
    d.step()
    d.check(up, acc)
    d.check_pages()


def test_a_captured_step_decodes():
    """One graph of a whole step, replayed with other drafts, lengths and pages; forks and compaction between replays."""
    d = Decoder("bf16", 16, 9, seed=5)
    d.prompt([20, 33, 4])
    up, acc = d.draw()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.step()
    torch.cuda.current_stream().wait_stream(side)
    d.check(up, acc)
    up, acc = d.draw()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.step()
    for i in range(8):
        if i:
            up, acc = d.draw()
        if i == 3:
            d.fork([1, 1, 0])
        if i == 5:
            d.compact()
        d.ws.fill_(0xFF)
        d.pws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        d.check(up, acc)
        d.check_pages()


def test_the_first_call_of_a_process_may_be_captured():
    """Nothing that a call sets up the first time stands in the way of a capture."""
    code = """
import torch, long_context_sparse_dsa_gb300 as dsa
i32 = dict(dtype=torch.int32, device="cuda")
for dtype, cap in (("bf16", 64), ("bf16", 65536), ("fp32", 64)):
    dt = dict(dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    dims = dsa.make_dims(cap, 16, 128, 8, 64, 8, dtype=dtype)
    cache = dsa.alloc_paged_cache(dims, 8, 16)
    for x in (cache.k, cache.v, cache.kpool, cache.ktail):
        x.normal_()
    refs, missing, remap = torch.zeros(8, **i32), torch.zeros(1, **i32), torch.zeros(8, **i32)
    lens, new, zero = torch.full((2,), 30, **i32), torch.full((2,), 36, **i32), torch.zeros(2, **i32)
    table = torch.full((2, cap // 16), -1, **i32)
    offsets, accepted = torch.tensor([0, 6, 12], **i32), torch.tensor([5, 2], **i32)
    q, k, v, ki = torch.randn(12, 16, 128, **dt), torch.randn(12, 128, **dt), torch.randn(12, 128, **dt), torch.randn(12, 64, **dt)
    dq, dk, w = torch.randn(12, 16, 128, device="cuda"), torch.randn(12, 128, device="cuda"), torch.zeros(128, device="cuda")
    qn, kn, o, lse = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty(12, 16, device="cuda")
    gq, gk, out = torch.empty_like(dq), torch.empty_like(dk), torch.zeros_like(lens)
    ws, pws = dsa.alloc_tree_workspace(dims, 2, 12), dsa.alloc_page_workspace(dims, cache, 2)
    nws = torch.empty(dsa.qk_norm_bwd_workspace_bytes(dims, 12), dtype=torch.uint8, device="cuda")
    kept = [x.clone() for x in (refs, table, cache.k, cache.v, cache.kpool, cache.ktail)]

    def step():
        dsa.qk_norm_rotate(dims, q, k, qn, kn, 1e-6)
        dsa.qk_norm_rotate_bwd(dims, q, k, dq, dk, gq, gk, 1e-6, nws, dq_weight=w)
        dsa.cache_reserve(dims, cache, refs, zero, new, table, missing, pws)
        dsa.decode_tree_attn(dims, cache, lens, table, offsets, None, qn, kn, v, o, lse, ws)
        dsa.cache_commit(dims, cache, lens, table, offsets, None, accepted, kn, v, ki, out)
        dsa.cache_release(dims, cache, refs, new, table, keep=out)
        dsa.cache_compact(dims, cache, refs, out, table, remap, missing, pws)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = []
    for go in (graph.replay, step):
        for x, y in zip((refs, table, cache.k, cache.v, cache.kpool, cache.ktail), kept):
            x.copy_(y)
        go()
        torch.cuda.synchronize()
        dsa.check_device_error()
        seen.append([x.clone() for x in (o, lse, gq, gk, w, out, refs, table, cache.k, cache.kpool, missing)])
    assert all(torch.equal(x, y) for x, y in zip(*seen)), [torch.equal(x, y) for x, y in zip(*seen)]
    assert out.tolist() == [36, 33] and missing.item() == 6 and bool(torch.isfinite(o).all())
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr
