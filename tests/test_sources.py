"""What the kernels' sources may not hold (no GPU)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_deterministic_bf16_gb300", "csrc")


def test_no_load_goes_to_several_ctas():
    """The same library serves programs on one GPU and on several, so no bulk or
    tensor load is multicast over a cluster.  (A commit's arrivals may be.)"""
    files = [f for p in ("*.cu", "*.cuh", "*.h", "*.cpp") for f in glob.glob(os.path.join(CSRC, p))]
    assert files
    for f in files:
        with open(f) as s:
            joined = re.sub(r'"\s*"', "", s.read())   # neighbouring string literals are one
        found = re.findall(r"cp\.async[^\"\n]*multicast[^\"\n]*", joined)
        assert not found, (os.path.basename(f), found)
