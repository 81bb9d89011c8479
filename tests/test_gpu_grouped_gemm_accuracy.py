"""How far float32 results are off on normal inputs (2-norm against 64 bits), at an inner size where sums
kept in one accumulator would show: the tensor core truncates as it adds, and 16384 terms in one accumulator
are off by 1.9e-5 (2.1e-6 where a cluster splits the sum).  Partial sums of 256 inner indices (weight
gradients: 512 rows) are 16 (32) additions of 16 products, off by 2^-22 of a running sum at most, whose
truncations point against the sum; the header's figures, 2.4e-7 to 2.7e-7 and 4.8e-7, are what that leaves.
The bounds here are twice those."""
import pytest
import torch

from expert_cached_sparse_b200 import api as A

pytestmark = pytest.mark.gpu

BF, F32, F64, F8, DEV = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn, "cuda"
K = 16384


def case(rows, width):
    g = torch.Generator(device=DEV)
    g.manual_seed(60)
    x, w = (torch.randn(n, K, generator=g, device=DEV).to(BF) for n in (rows, width))
    return x, w, torch.tensor([0, rows], dtype=torch.int32, device=DEV)


def err(got, ref):
    return float((got.to(F64) - ref).norm() / ref.norm())


@pytest.mark.parametrize("rows,width", [(64, 256), (320, 1280)], ids=["few", "pairs"])
def test_row_products(rows, width):
    x, w, off = case(rows, width)
    ref = x.to(F64) @ w.to(F64).t()
    y = torch.empty(rows, width, device=DEV)
    A.moe_grouped_gemm(x, w[None], off, y)
    assert err(y, ref) < 5.4e-7
    A.moe_grouped_gemm_dx(x, w.t().contiguous()[None], off, y)
    assert err(y, ref) < 5.4e-7


@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient(accumulate):
    x, w, _ = case(136, 392)
    dw = torch.zeros(1, 136, 392, device=DEV)
    A.moe_grouped_gemm_dw(x.t().contiguous(), w.t().contiguous(), torch.tensor([0, K], dtype=torch.int32, device=DEV), dw,
                          accumulate=accumulate)
    assert err(dw[0], x.to(F64) @ w.to(F64).t()) < 9.6e-7


@pytest.mark.parametrize("rows,width", [(64, 256), (320, 1280)], ids=["few", "many"])
def test_e4m3_product(rows, width):
    x, w, off = case(rows, width)
    xq, wq = x.to(F8), w.to(F8)
    y = torch.empty(rows, width, device=DEV)
    A.moe_grouped_gemm_fp8(xq, torch.ones(K // 128, rows, device=DEV), wq[None],
                           torch.ones(1, width // 128, K // 128, device=DEV), off, y)
    assert err(y, xq.to(F32).to(F64) @ wq.to(F32).to(F64).t()) < 2e-7
