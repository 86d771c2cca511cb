"""Reserving pages for rows whose open page is nobody's.  Everything is exact (test_gpu_pages)."""
import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa
from test_gpu_decode import _built  # noqa: F401
from test_gpu_decode_contract import _reports
from test_gpu_pages import World, _i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [3, 600])
def test_reserve_refuses_an_open_page_that_is_free(rows):
    """A row whose next token goes to a page that refs counts for nobody: the page may be given away in the same call, so the row
    asks for nothing and is reported; the others are served."""
    w = World(3 * rows, 16, 64, seed=6)
    table, refs = [[b, -1, -1, -1] for b in range(rows)], [1] * rows + [0] * (2 * rows)
    refs[1] = 0                                  # row 1's page
    if rows > 500:
        refs[rows - 2] = -1
    lens, new, dev, missing = [5] * rows, [17 + 16 * (b % 2) for b in range(rows)], _i32(table), _i32([-1])
    w.refs.copy_(_i32(refs))
    dsa.cache_reserve(w.dims, w.cache, w.refs, _i32(lens), _i32(new), dev, missing, w.ws(rows))
    _reports(dsa.DSA_ERR_BAD_PAGE)
    free = [p for p, c in enumerate(refs) if c == 0]
    for b in range(rows):
        if refs[b] > 0:
            for c in range(1, w.held(new[b])):
                table[b][c] = free.pop(0)
    for row in table:
        for p in row[1:]:
            if p >= 0:
                refs[p] = 1
    assert missing.item() == 0 and dev.tolist() == table and w.refs.tolist() == refs
    assert table[0][1] == 1
    for x, y in w.copy.items():
        assert torch.equal(getattr(w.cache, x), y)
