"""The rules of the sources around the experts, for the score router, the sandwich norm and the 4-bit projection."""
import os
import re

import pytest

from test_block_sources_cpu import CSRC, code_of

SOURCES = ["score_router.cu", "sandwich.cu", "int4.cu", "router.cuh", "rows.cuh", "pipeline.cuh"]


@pytest.mark.parametrize("name", SOURCES)
def test_nothing_is_loaded_through_the_read_only_path(name):
    """These kernels start while the kernel before them in the stream may still write their inputs."""
    assert not re.search(r"__ldg\b|ld\.global(\.\w+)*\.nc|__ldlu\b", code_of(name))


@pytest.mark.parametrize("name", SOURCES)
def test_no_wait_is_unbounded(name):
    """A wait on a barrier goes through the bounded ones: no loop of its own over the tests of a phase."""
    text = code_of(name)
    assert "__trap" not in text and not re.search(r"\bassert\s*\(", text)
    assert not re.search(r"while\s*\(\s*!?\s*mbar_(try|test)_wait", text)


@pytest.mark.parametrize("name", [n for n in SOURCES if n.endswith(".cu")])
def test_a_dependent_launch_waits_before_it_reads(name):
    """Each kernel of a file is launched as a dependent one, so each waits for the kernel before it."""
    text = code_of(name)
    bodies = re.split(r"__global__", text)[1:]
    assert bodies
    for b in bodies:
        head = b.index("{")
        assert "grid_dep_wait()" in b[head:], b[:head]


def test_sources_are_there():
    assert all(os.path.exists(os.path.join(CSRC, n)) for n in SOURCES)
