"""Kernels that are set up while the one before them still runs (csrc/launch.cuh) may not read through the read-only
path: it wants memory that nothing writes while the kernel lives, and the compiler may move such a load ahead of the
wait.  Shown on the source, since a reordered load need not show in a run."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_bit_block_amax_b200", "csrc")


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def files():
    """The units that launch early, and the headers that only they include."""
    units = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and "launch_early(" in code(f)]
    others = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and f not in units]
    includes = lambda fs: {h for f in fs for h in re.findall(r'#include "(\w+\.cuh)"', code(f))}
    return units + sorted(includes(units) - includes(others) - {"launch.cuh"})


def test_there_are_early_kernels():
    assert {"few.cu", "gemm.cu", "layer.cu", "segments.cuh"} <= set(files())


@pytest.mark.parametrize("name", files())
def test_early_kernels_read_with_ordinary_loads(name):
    for pattern in (r"\b__ldg\s*\(", r"\bldg_stream\s*\(", r"ld\.global(\.\w+)*\.nc", r"__restrict__"):
        hits = [line.strip() for line in code(name).splitlines() if re.search(pattern, line)]
        assert not hits, f"{name}: {hits}"


@pytest.mark.parametrize("name", [f for f in files() if f.endswith(".cu")])
def test_no_access_before_the_wait(name):
    """Up to the wait an early kernel touches no memory that its parameters point to: pointers of the parameter struct
    and pointer parameters first appear behind it."""
    for kernel in re.finditer(r"__global__.*?\n}\n", code(name), flags=re.S):
        body = kernel.group(0)
        if "wait_for_stream()" not in body:
            continue
        head = body[body.index("{"):body.index("wait_for_stream()")]
        assert not re.search(r"p\.(sf\w*|\w*_gs|offsets|counts|bias|residual|pre|c|c_amax|dy|z|dz|sums|amax|maxima|ids|hist|"
                             r"row_copy|copy_row|src|other|dst|weights|dweights)\b", head), body[:120]
