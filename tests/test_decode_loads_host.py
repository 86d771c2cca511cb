"""The paged decode kernels become resident while the kernel before them on the stream may still write what they read
(decode.cuh).  The non-coherent load path is for data that nobody writes during a kernel's life, so none of their sources may
ask for it: not by name, and not by a pointer to const that the compiler is told nothing else writes to."""
import glob
import os
import re

import pytest

from long_context_sparse_dsa_gb300 import build as dsa_build

FILES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(dsa_build.CSRC, "decode*.cu*")))


def _code(name):
    with open(os.path.join(dsa_build.CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", FILES)
def test_no_non_coherent_loads(name):
    code = _code(name)
    for word in ("__ldg", "__restrict__", "ld.global.nc", "ld_nc", "tex1D"):
        assert word not in code, word


def test_the_files_are_these():
    assert {"decode_append.cu", "decode_attn.cu", "decode_scores.cu", "decode_topk.cu", "decode.cuh"} <= set(FILES)
    # kernels of this kind are launched by these files only
    for f in glob.glob(os.path.join(dsa_build.CSRC, "*.cu")):
        if os.path.basename(f) not in FILES:
            assert "launch_chained" not in _code(os.path.basename(f)), f
