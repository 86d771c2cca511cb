"""A Rotation hands a pointer and a length to the kernels: it takes only tensors that hold what they will read."""
import pytest
import torch

import long_context_sparse_dsa_gb300 as dsa


@pytest.mark.parametrize("turns", [
    torch.zeros(32, dtype=torch.int32),              # half the bytes
    torch.zeros(32, dtype=torch.float64),
    torch.zeros(64, dtype=torch.int64)[::2],         # every other one
    torch.zeros(4, 8, dtype=torch.int64),
    torch.zeros(0, dtype=torch.int64),
    torch.zeros(7, dtype=torch.int64),
    [1] * 8])
def test_rotation_refuses_other_tensors(turns):
    with pytest.raises(ValueError):
        dsa.Rotation(turns, False)


def test_rotation_takes_turns():
    turns = torch.arange(16, dtype=torch.int64)
    r = dsa.Rotation(turns, True)
    assert r.dim == 32 and r.turns is turns and r._c.turns == turns.data_ptr() and r._c.interleaved == 1
