"""Microscaled KV cache, on the CPU: what its sources, binding and MXCache's
bookkeeping promise at the ends of their contracts."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sub_bit_vector_b200", "csrc")


def test_no_read_only_loads_in_kernels_that_start_early():
    """The read-only path (__ldg, ld.global.nc, __restrict__ pointers that the
    compiler may turn into it) is for data that nothing writes while the kernel
    lives.  These kernels may be resident before the one that writes their
    inputs has ended."""
    files = sorted(glob.glob(os.path.join(CSRC, "mx*.cu*")))
    assert len(files) == 5
    for f in files:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(f).read(), flags=re.S)
        assert "griddepcontrol.wait" in code or "mx_begin()" in code or f.endswith("mx_attn.cuh")
        for word in ("__ldg(", ".nc", "__restrict__", "ldg("):
            assert word not in code, (os.path.basename(f), word)
