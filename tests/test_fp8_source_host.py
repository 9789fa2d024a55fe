"""Read-only loads in the kernels that overlap the launch before them, without a GPU."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_routed_non_b200", "csrc")
FILES = sorted(os.path.basename(p) for pat in ("fp8*.cuh", "fp8_gemm*.cu", "norm.cu") for p in glob.glob(os.path.join(CSRC, pat)))


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_load_of_what_the_launch_before_may_write(name):
    """Each of these kernels starts while the launch before it runs, and all they read may come from
    it: the read-only path asks for memory that does not change while the kernel runs."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    found = re.findall(r"[^\n]*(?:__ldg\s*\(|ld\.global\.nc)[^\n]*", code)
    assert not found, found


def test_the_combine_reads_y_by_plain_loads():
    """It overlaps the product that writes y and its exponents (the metadata's tables are finished by then)."""
    with open(os.path.join(CSRC, "combine.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "ld.global.nc" not in code and not re.search(r"__ldg\s*\(\s*(y|scol|y_scale)", code)
