"""Kernels that start while the one before them ends (launch_overlapped in layer.cuh) must
not read by way of the read-only cache, which is for memory that no one writes while the
kernel runs: the kernel before may still be writing their operands. No GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "selective_state_space_17_b200", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def overlapped():
    return sorted(f for f in os.listdir(CSRC) if f.endswith(".cu") and "launch_overlapped(" in code(f))


def test_the_sources_are_found():
    assert overlapped() == ["conv.cu", "linear.cu", "norm.cu"]


@pytest.mark.parametrize("name", overlapped() + ["layer.cuh", "sm100_mma.cuh"])
def test_overlapped_kernels_read_with_plain_loads(name):
    """No read-only load, nor io<T>::load, which is one; nor a promise of no aliases that
    would let the compiler make one."""
    found = re.findall(r"__ldg\w*\s*\(|\.nc\b|ld\.global\.nc|\bio<\w+>::load|__restrict__", code(name))
    assert not found, found
