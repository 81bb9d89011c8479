"""Sums over long inner sizes.  The tensor core truncates as it adds, so a sum of terms of one sign comes
out too small by an amount that grows with the number of additions in one accumulator.  Row and column
factors spread the results over a binade, so that bf16 roundings average out over n results and what is
left of the mean relative error is the sums' own.

Bound on that mean: an accumulator takes at most 8192 inner indices, 512 additions of 16 products, each
off by at most 2^-22 of a running sum that is half the final one on average, 512 * 2^-23 = 2^-14.  The sums
of these partial sums, 128 at 2^20 (of float32 outputs 4096 or fewer, with partial sums so much shorter),
round to nearest, with either sign: below 2^-19.  bf16 rounding is off by at most 2^-8 relative, with
standard deviation below 2^-8 / sqrt(3), five times which over sqrt(n) bounds its mean."""
import pytest
import torch

from expert_cached_sparse_b200 import api as A

pytestmark = pytest.mark.gpu

BF, F32, F64, DEV = torch.bfloat16, torch.float32, torch.float64, "cuda"
LONG = 1 << 20


def positive(g, scaled, summed):
    """[scaled][summed] values of one sign, each of the `scaled` ones with a factor of its own."""
    t = torch.empty(scaled, summed, dtype=BF, device=DEV)
    step = max(1, (64 << 20) // summed)
    for i in range(0, scaled, step):
        n = min(step, scaled - i)
        f = torch.rand(n, 1, generator=g, device=DEV).exp2_()
        t[i:i + n] = torch.rand(n, summed, generator=g, device=DEV).add_(0.5).mul_(f).to(BF)
    return t


def product64(a, b):
    """a b^T in 64 bits, a few rows of b at a time."""
    a = a.to(F64)
    step = max(1, (256 << 20) // b.shape[1])
    return torch.cat([a @ b[i:i + step].to(F64).t() for i in range(0, b.shape[0], step)], 1)


def check(got, ref):
    rel = (got.to(F64) - ref) / ref
    half = {BF: 2.0 ** -8, F32: 2.0 ** -24}[got.dtype]
    bound = 2.0 ** -14 + 2.0 ** -19 + 5 * half / 3 ** 0.5 / ref.numel() ** 0.5
    assert abs(float(rel.mean())) <= bound, (float(rel.mean()), bound)
    assert float(rel.abs().max()) <= half * 1.001 + 2 * (2.0 ** -14 + 2.0 ** -19)


def offsets(*ends):
    return torch.tensor([0, *ends], dtype=torch.int32, device=DEV)


# 32-row tiles split over a cluster, the same unsplit (more tiles), and pairs of CTAs
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,width", [(64, 256), (320, 1280)], ids=["few", "pairs"])
def test_forward(rows, width, dt):
    g = torch.Generator(device=DEV)
    g.manual_seed(50)
    x, w = positive(g, rows, LONG), positive(g, width, LONG)
    y = torch.empty(rows, width, dtype=dt, device=DEV)
    A.moe_grouped_gemm(x, w[None], offsets(rows), y)
    check(y, product64(x, w))
    assert A.moe_get_device_error() == 0


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,width", [(64, 256), (320, 1280)], ids=["few", "pairs"])
def test_rows_gradient(rows, width, dt):
    g = torch.Generator(device=DEV)
    g.manual_seed(51)
    dy, wt = positive(g, rows, LONG), positive(g, width, LONG)
    w = wt.t().contiguous()
    dx = torch.empty(rows, width, dtype=dt, device=DEV)
    A.moe_grouped_gemm_dx(dy, w[None], offsets(rows), dx)
    check(dx, product64(dy, wt))
    assert A.moe_get_device_error() == 0


def test_forward_of_many_experts_with_few_rows():
    """32-row tiles without a split."""
    g = torch.Generator(device=DEV)
    g.manual_seed(52)
    E, K, N = 16, 1 << 18, 1280
    x = positive(g, 16 * E, K)
    w = positive(g, E * N, K).view(E, N, K)
    y = torch.empty(16 * E, N, dtype=BF, device=DEV)
    A.moe_grouped_gemm(x, w, offsets(*range(16, 16 * E + 1, 16)), y)
    check(y, torch.cat([product64(x[16 * e:16 * e + 16], w[e]) for e in range(E)]))


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_weight_gradient(dt, accumulate):
    """One expert of 2^20 rows between an empty one and a small one."""
    g = torch.Generator(device=DEV)
    g.manual_seed(53)
    N, K, small = 136, 392, 300
    dyt, xt = positive(g, N, LONG + small), positive(g, K, LONG + small)
    dy, x = dyt.t().contiguous(), xt.t().contiguous()
    base = 1000 * torch.rand(3, N, K, generator=g, device=DEV)
    dw = base.to(dt)
    first = dw.to(F64)
    A.moe_grouped_gemm_dw(dy, x, offsets(0, LONG, LONG + small), dw, accumulate=accumulate)
    for e, rows in ((1, slice(0, LONG)), (2, slice(LONG, LONG + small))):
        ref = product64(dyt[:, rows], xt[:, rows])
        check(dw[e], ref + first[e] if accumulate else ref)
    assert torch.equal(dw[0].to(F64), first[0]) if accumulate else not bool(dw[0].any())
    assert A.moe_get_device_error() == 0
