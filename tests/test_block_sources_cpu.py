"""Rules that the sources of the operators around the experts keep and no result shows reliably."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "serving_topk_permute_gb300", "csrc")


def code_of(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", ["linear.cu", "norm.cu", "router.cu", "quant.cuh"])
def test_nothing_is_loaded_through_the_read_only_path(name):
    """These kernels start while the kernel before them in the stream may still write their inputs; __ldg
    and ld.global.nc want data that stays as it is for the kernel's whole life."""
    assert not re.search(r"__ldg\b|ld\.global(\.\w+)*\.nc|__ldlu\b", code_of(name))
