"""The C library needs nvcc only: what else is missing costs the binding, not the build."""
import os
import subprocess
import sys

import pytest

from conftest import REPO
from dense_fp32_gemm_09_gb300 import build

WITHOUT_TORCH = """
import sys, warnings
sys.path.insert(0, sys.argv[1])
sys.modules["torch"] = None
warnings.simplefilter("error" if sys.argv[2] == "strict" else "ignore")
"""


def run(code, how="ignore"):
    return subprocess.run([sys.executable, "-c", WITHOUT_TORCH + code, REPO, how],
                          capture_output=True, text=True, timeout=300)


def test_builds_without_torch(lib):
    r = run("from dense_fp32_gemm_09_gb300 import build, load\n"
            "assert build.build() == build.LIB_PATH\nassert load().sgemm_num_kernels() > 0\n")
    assert r.returncode == 0, r.stderr
    r = run("from dense_fp32_gemm_09_gb300 import build\nbuild.build()\n", "strict")
    assert r.returncode != 0 and "UserWarning: the binding of the 4-bit" in r.stderr


def test_a_compiler_that_fails_costs_the_binding_only(lib, monkeypatch, tmp_path):
    monkeypatch.setenv("CXX", "false")
    monkeypatch.setattr(build, "fast_path", lambda: str(tmp_path / "_fast_calls.so"))
    with pytest.warns(UserWarning, match="not built"):
        assert build.build() == build.LIB_PATH
    with pytest.raises(RuntimeError, match="fast_calls"):
        build.build_binding()


def test_the_binding_is_that_of_the_installed_torch(lib):
    import torch
    name = os.path.basename(build.fast_path())
    assert torch.__version__ in name and f"cpython-{sys.version_info[0]}{sys.version_info[1]}" in name
    assert os.path.exists(build.fast_path())


def test_everything_can_be_imported_without_torch():
    r = run("from dense_fp32_gemm_09_gb300 import *\nassert callable(sgemm_query_config)\n"
            "import dense_fp32_gemm_09_gb300 as sg\n"
            "assert 'sgemm' in sg.__all__ and 'mx4_matmul' not in sg.__all__\n")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([sys.executable, "-c", "import sys; sys.path.insert(0, sys.argv[1])\n"
                        "from dense_fp32_gemm_09_gb300 import *\nassert mx4_matmul and norm_after\n",
                        REPO], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
