"""Room reserved for the deepest drafts before the accepted path is known, as include/dsa_pages.h says to: reserve, commit of a
shorter path, release of the rest with the reserved length, with forks and compaction between.  No page is lost, none named by
two rows that write to it, and every sequence stays what it is.  Steps and their checks: test_gpu_draft_decoding."""
import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from test_gpu_decode import DEV, _built  # noqa: F401
from test_gpu_draft_decoding import Decoder, _i32

pytestmark = pytest.mark.gpu


class Roomy(Decoder):
    """A decoder that reserves for all of its nodes."""
    PAGE = 4   # room of several pages

    def before(self):
        """What does not need the accepted paths."""
        lens = self.lens[self.row]
        dsa.qk_norm_rotate(self.dims, self.q, self.kk, self.qr, self.kr, 1e-6, q_weight=self.qw, k_weight=self.kw,
                           rotation=self.rot, positions=lens + self.depth - 1)
        torch.add(self.lens, self.N, out=self.new_lens)
        dsa.cache_reserve(self.dims, self.cache, self.refs, self.lens, self.new_lens, self.table, self.missing, self.pws)
        dsa.decode_indexer_topk(self.dims, self.cache, lens, self.table[self.row], self.qi, self.w, self.idx, self.iws)
        dsa.decode_tree_attn(self.dims, self.cache, self.lens, self.table, self.offsets, self.parents, self.qr, self.kr, self.v,
                             self.o, self.lse, self.ws, idx=self.idx)

    def after(self):
        dsa.cache_commit(self.dims, self.cache, self.lens, self.table, self.offsets, self.parents, self.accepted, self.kr, self.v,
                         self.ki, self.lens)
        dsa.cache_release(self.dims, self.cache, self.refs, self.new_lens, self.table, keep=self.lens)

    def compact_with_room(self):
        remap, used = torch.zeros_like(self.refs), _i32([0])
        dsa.cache_compact(self.dims, self.cache, self.refs, self.new_lens, self.table, remap, used, self.pws)
        dsa.check_device_error()
        held = sorted({p for p in self.table.flatten().tolist() if p >= 0})
        assert held == list(range(used.item()))


@pytest.mark.parametrize("dtype,Hq", [("bf16", 16), ("fp32", 8)])
def test_unused_room_is_given_back(dtype, Hq):
    d = Roomy(dtype, Hq, 9, seed=17, pages=120, L=256)
    d.prompt([61, 0, 30])
    short = 0
    for i in range(16):
        if i in (4, 9):
            d.fork([0, 0, 2] if i == 4 else [2, 1, 2])
        up, acc = d.draw()
        short += sum(d.grow.tolist()) < 3 * d.N
        d.before()
        if i % 3 == 1:
            d.compact_with_room()      # pages of the room move too, before anything is written to them
        d.after()
        d.check(up, acc)
        d.check_pages()
        assert torch.equal((d.table >= 0).sum(1, dtype=torch.int32), (d.lens + d.PAGE - 1) // d.PAGE)
    assert short > 8
    dsa.cache_release(d.dims, d.cache, d.refs, d.lens, d.table)
    assert not torch.any(d.refs)       # nothing was lost


def test_unused_room_in_a_captured_step():
    d = Roomy("bf16", 16, 9, seed=18, pages=100, L=256)
    d.prompt([20, 33, 4])
    up, acc = d.draw()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.before()
        d.after()
    torch.cuda.current_stream().wait_stream(side)
    d.check(up, acc)
    d.check_pages()
    d.draw()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.before()
        d.after()
    for i in range(8):
        up, acc = d.draw()
        if i == 4:
            d.fork([1, 1, 0])
        graph.replay()
        torch.cuda.synchronize()
        d.check(up, acc)
        d.check_pages()
    dsa.cache_release(d.dims, d.cache, d.refs, d.lens, d.table)
    assert not torch.any(d.refs)
