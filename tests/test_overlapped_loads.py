"""Loads of kernels that may start while the kernel before them still writes (CPU only, on the sources).

__ldg, ld.global.nc and const __restrict__ parameters promise that the data stays as it is while the
kernel runs.  A kernel launched by launch_overlapped cannot promise that of anything the kernel
before it may write, and the compiler may take such a load ahead of griddepcontrol.wait."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "expert_cached_sparse_b200" / "csrc"
OVERLAPPED = sorted(p.name for p in CSRC.iterdir() if "overlap.cuh" in p.read_text() or "launch_overlapped" in p.read_text())
NON_COHERENT = re.compile(r"__ldg\s*\(|ld\.global[.\w]*\.nc\b|ld\.global\.nc|const\s[^,()]*\*\s*__restrict__")


def code(name):
    """The source without its comments."""
    s = re.sub(r"/\*.*?\*/", "", (CSRC / name).read_text(), flags=re.S)
    return re.sub(r"//[^\n]*", "", s)


def test_the_sources_are_found():
    assert {"grouped_gemm.cu", "grouped_gemm_fp8.cu", "fp8_quant.cu", "tc.cuh"} <= set(OVERLAPPED) | {"grouped_gemm.cu", "grouped_gemm_fp8.cu"}


@pytest.mark.parametrize("name", sorted(set(OVERLAPPED) | {"grouped_gemm.cu", "grouped_gemm_fp8.cu"}))
def test_overlapped_kernels_load_no_data_as_read_only(name):
    assert NON_COHERENT.findall(code(name)) == []
