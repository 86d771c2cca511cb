"""Registers that the selected-pool attention kernels spill: what the compiler says, no GPU needed.  Moving a line of the kernel
changed it once, and 32 fp32 heads of 64 took 7% longer."""
import os
import re
import subprocess

from long_context_sparse_dsa_gb300 import build as dsa_build


def test_selected_rows_spill_no_more_than_they_did(tmp_path):
    cmd = [dsa_build._nvcc(), *dsa_build.ARCH, *dsa_build.FLAGS, "-Xptxas", "-v", "-c", os.path.join(dsa_build.CSRC, "decode_attn.cu"),
           "-o", str(tmp_path / "x.o")]
    said = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    spills = {}
    for name, stores in re.findall(r"entry function '(\w+)'.*?(\d+) bytes spill stores", said, re.S):
        if "decode_attn_rows_kernel" in name and "ELb1EEE" in name:   # selected pools
            spills[name] = int(stores)
    assert len(spills) == 10
    for name, n in spills.items():
        assert n <= (20 if "IfLi64ELi32E" in name else 0), (name, n)
