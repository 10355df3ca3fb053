"""Kernels that are launched as programmatic dependents use no load that may be moved to before their
wait for the previous kernel: the read-only ones, which the assembler moves."""
import glob
import os
import re

import pytest

from dense_fp32_gemm_09_gb300 import build

# Files whose kernels with such loads are launched after the previous kernel has ended.
PLAIN = {"sgemm_api.cu": ("pack_rows_kernel", "transpose_kernel"), "sgemm_tf32x3.cu": ("split_kernel",)}
READ_ONLY = re.compile(r"__ldg\s*\(|\bld\.global\.nc\b|const\s+\w+\s*\*\s*__restrict__")


def code(path):
    """Without comments and the names in messages."""
    return re.sub(r'//[^\n]*|"\w+_kernel[^"\n]*"', "", open(path).read())


def sources():
    return sorted(f for kind in ("*.cu", "*.cuh", "*.h") for f in glob.glob(os.path.join(build.CSRC, kind)))


@pytest.mark.parametrize("path", sources(), ids=os.path.basename)
def test_no_read_only_loads(path):
    if os.path.basename(path) not in PLAIN:
        assert not READ_ONLY.findall(code(path))


@pytest.mark.parametrize("name,kernel", [(n, k) for n, ks in PLAIN.items() for k in ks])
def test_the_others_are_launched_plainly(name, kernel):
    text = code(os.path.join(build.CSRC, name))
    uses = re.findall(rf"\b{kernel}\b\s*(<<<|\()?", text)
    assert uses.count("(") == 1 and set(uses) == {"(", "<<<"}      # its definition, and launches
