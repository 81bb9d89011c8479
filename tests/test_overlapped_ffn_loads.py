"""The grouped FFN's first kernels may start while the kernel before the call still writes the rows and the
routing (CPU only, on the sources): they too read those with plain loads through plain pointers."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "expert_cached_sparse_b200" / "csrc"


def code(name):
    s = re.sub(r"/\*.*?\*/", "", (CSRC / name).read_text(), flags=re.S)
    return re.sub(r"//[^\n]*", "", s)


@pytest.mark.parametrize("name,kernel", [("ffn.cu", "ffn_prep_kernel"), ("ffn_fp4.cu", "fp4_plan_kernel"), ("ffn_fp4.cu", "fp4_terms_kernel")])
def test_kernels_that_read_the_calls_inputs(name, kernel):
    parts = [p for p in re.split(r"(?=\b__global__\b)", code(name)) if p.startswith("__global__")]
    body = [p for p in parts if re.search(rf"\b{kernel}\s*\(", p.split("{")[0])]
    assert len(body) == 1
    text = body[0].split("\n}\n")[0]
    assert "pdl_wait()" in text
    assert not re.findall(r"__ldg\s*\(|\.nc\b|const\s[^,()]*\*\s*__restrict__", text)


def test_rows_of_activations():
    s = code("ffn_fp4.cu")
    start = s.index("void load8(")
    assert "__ldg" not in s[start:s.index("\n}\n", start)]
