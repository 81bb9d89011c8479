"""Row products on pairs of CTAs: what the second CTA copies and reads is handed to the first one's MMAs
in order, whatever else the GPU does, and however the rows fall on the pair's two halves.  Inputs are
small integers, so every result has one value."""
import pytest
import torch

from expert_cached_sparse_b200 import api as A

pytestmark = pytest.mark.gpu

BF, F32, F64, DEV = torch.bfloat16, torch.float32, torch.float64, "cuda"


def ints(shape, g):
    return torch.randint(-3, 4, shape, generator=g, device=DEV).to(F32).to(BF)


def setup(counts, K, N, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    E, rows = len(counts), sum(counts)
    off = torch.tensor([sum(counts[:e]) for e in range(E + 1)], dtype=torch.int32, device=DEV)
    x, w, dy = ints((rows, K), g), ints((E, N, K), g), ints((rows, N), g)
    y, dx = torch.empty(rows, N, dtype=F64, device=DEV), torch.empty(rows, K, dtype=F64, device=DEV)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        y[a:b] = x[a:b].to(F64) @ w[e].to(F64).t()
        dx[a:b] = dy[a:b].to(F64) @ w[e].to(F64)
    return off, x, w, dy, y, dx


# blocks of one row to 256: the second CTA has no columns, few, all but one, all; K and N off every step
@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("counts", [[1, 16, 17, 600], [31, 32, 33, 48, 49, 640], [255, 256, 257, 129], [1300]],
                         ids=["few", "halves", "whole", "one"])
def test_every_split_of_the_columns(counts, dt):
    K, N = 840, 1096
    off, x, w, dy, y64, dx64 = setup(counts, K, N, 40)
    y, dx = torch.full((x.shape[0], N), 7.0, dtype=dt, device=DEV), torch.full((x.shape[0], K), 7.0, dtype=dt, device=DEV)
    A.moe_grouped_gemm(x, w, off, y)
    A.moe_grouped_gemm_dx(dy, w, off, dx)
    assert torch.equal(y, y64.to(dt)) and torch.equal(dx, dx64.to(dt))
    assert A.moe_get_device_error() == 0


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_repeated_beside_other_work(dt):
    """The hand-overs' timing varies: 40 calls beside copies on another stream that take the memory's bandwidth."""
    off, x, w, dy, y64, dx64 = setup([700, 0, 300, 24, 1000], 1032, 2056, 41)
    y = [torch.empty(x.shape[0], 2056, dtype=dt, device=DEV) for _ in range(4)]
    dx = [torch.empty(x.shape[0], 1032, dtype=dt, device=DEV) for _ in range(4)]
    want_y, want_dx = y64.to(dt), dx64.to(dt)
    a = torch.empty(128 << 20, dtype=torch.uint8, device=DEV)
    b = torch.empty_like(a)
    torch.cuda.synchronize()
    other, st = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(other):
            for _ in range(3):
                b.copy_(a)
        with torch.cuda.stream(st):
            for t in y + dx:
                t.fill_(7)
            for i in range(4):
                A.moe_grouped_gemm(x, w, off, y[i], stream=st)
                A.moe_grouped_gemm_dx(dy, w, off, dx[i], stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(t, want_y) for t in y) and all(torch.equal(t, want_dx) for t in dx)
    assert A.moe_get_device_error() == 0
