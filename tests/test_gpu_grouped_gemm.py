"""Expert matrix products, their gradients and the FP8 forms on the GPU.

Most checks are exact.  Inputs that are small integers (and scales that are
powers of two) make every product and every partial sum an integer below 2^24
times one power of two, so the fp32 result has one value whatever the order of
the sums, and float32 outputs must equal the 64-bit reference bit for bit;
bf16 outputs must equal its rounding.  Normal inputs are held to bounds
derived where they are used.
"""
import pathlib
import subprocess
import sys

import numpy as np
import pytest
import torch

from expert_cached_sparse_b200 import _lib as L
from expert_cached_sparse_b200 import api as A

pytestmark = pytest.mark.gpu

BF, F32, F64, F8 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
DEV = "cuda"

# rows per expert: empty experts first, last and in between, one row, both sides of every tile edge
COUNTS = {
    "one": [1],
    "single16": [0, 0, 16],
    "edges": [0, 1, 15, 16, 17, 0, 31, 33, 0],
    "tiles": [63, 64, 65, 0, 127, 128, 129],
    "big": [255, 0, 256, 257, 3],
    "long": [700, 1],
    "many": [(7 * e) % 4 for e in range(300)],
}
SIZES = [(8, 8), (16, 64), (64, 128), (72, 136), (128, 120), (264, 1000), (1000, 264), (512, 512)]
CASES = [(c, s) for c in COUNTS for s in SIZES if c in ("edges", "tiles") or s in ((72, 136), (264, 1000), (512, 512))]
IDS = [f"{c}-{i}x{o}" for c, (i, o) in CASES]


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def ints(shape, g, m=3, dtype=BF):
    return torch.randint(-m, m + 1, shape, generator=g, device=DEV).to(F32).to(dtype)


def offsets_of(counts, first=0):
    return torch.tensor([first] + [first + int(c) for c in np.cumsum(counts)], dtype=torch.int32, device=DEV)


def ranges(offsets, rows):
    o = offsets.tolist()
    return [(a, b) if 0 <= a <= b <= rows else (0, 0) for a, b in zip(o[:-1], o[1:])]


def ref_fwd(x, w, off):
    y = torch.zeros(x.shape[0], w.shape[1], dtype=F64, device=DEV)
    for e, (a, b) in enumerate(ranges(off, x.shape[0])):
        if b > a:
            y[a:b] = x[a:b].to(F64) @ w[e].to(F64).t()
    return y


def ref_dx(dy, w, off):
    return ref_fwd(dy, w.transpose(1, 2), off)


def ref_dw(dy, x, off):
    return torch.stack([dy[a:b].to(F64).t() @ x[a:b].to(F64) for a, b in ranges(off, x.shape[0])])


def spread(s, n, k):
    i, j = torch.arange(n, device=DEV) // 128, torch.arange(k, device=DEV) // 128
    return s[..., i, :][..., j]


def ref_fp8(xq, xs, wq, ws, off):
    rows, K = xq.shape
    x = xq.to(F32).to(F64) * xs.to(F64).t()[:, torch.arange(K, device=DEV) // 128]
    return ref_fwd(x, wq.to(F32).to(F64) * spread(ws.to(F64), wq.shape[1], K), off)


def pow2(shape, g):
    return torch.randint(-1, 2, shape, generator=g, device=DEV).to(F32).exp2()


def fp8_inputs(E, rows, K, N, g):
    return (ints((rows, K), g, dtype=F8), pow2(((K + 127) // 128, rows), g), ints((E, N, K), g, dtype=F8),
            pow2((E, (N + 127) // 128, (K + 127) // 128), g))


@pytest.mark.parametrize("name,size", CASES, ids=IDS)
@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_forward_exact(name, size, dt):
    counts, (K, N) = COUNTS[name], size
    g, rows, E = gen(1), sum(counts), len(counts)
    off = offsets_of(counts)
    x, w = ints((rows, K), g), ints((E, N, K), g)
    y = torch.full((rows, N), 7.0, dtype=dt, device=DEV)
    A.moe_grouped_gemm(x, w, off, y)
    assert torch.equal(y, ref_fwd(x, w, off).to(dt))


@pytest.mark.parametrize("name,size", CASES, ids=IDS)
@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_gradients_exact(name, size, dt):
    counts, (K, N) = COUNTS[name], size
    g, rows, E = gen(2), sum(counts), len(counts)
    off = offsets_of(counts)
    x, w, dy = ints((rows, K), g), ints((E, N, K), g), ints((rows, N), g)
    dx = torch.full((rows, K), 7.0, dtype=dt, device=DEV)
    A.moe_grouped_gemm_dx(dy, w, off, dx)
    assert torch.equal(dx, ref_dx(dy, w, off).to(dt))
    dw = torch.full((E, N, K), 7.0, dtype=dt, device=DEV)
    A.moe_grouped_gemm_dw(dy, x, off, dw)
    want = ref_dw(dy, x, off)
    assert torch.equal(dw, want.to(dt))
    # accumulating adds in fp32 to what is there and leaves experts without rows alone
    base = ints((E, N, K), g).to(dt)
    acc = base.clone()
    A.moe_grouped_gemm_dw(dy, x, off, acc, accumulate=True)
    assert torch.equal(acc, (base.to(F64) + want).to(dt))


@pytest.mark.parametrize("name,size", CASES, ids=IDS)
@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_fp8_exact(name, size, dt):
    counts, (K, N) = COUNTS[name], size
    K = (K + 15) // 16 * 16
    g, rows, E = gen(3), sum(counts), len(counts)
    off = offsets_of(counts)
    args = fp8_inputs(E, rows, K, N, g)
    y = torch.full((rows, N), 7.0, dtype=dt, device=DEV)
    A.moe_grouped_gemm_fp8(*args, off, y)
    assert torch.equal(y, ref_fp8(*args, off).to(dt))


@pytest.mark.parametrize("K", [2048, 4096])
def test_long_inner_sizes(K):
    """One to a few rows over long inner sizes, and one expert only."""
    g = gen(4)
    for counts in ([1], [0, 2, 0, 1], [1] * 8, [130]):
        off, rows, E, N = offsets_of(counts), sum(counts), len(counts), 384
        x, w, dy = ints((rows, K), g), ints((E, N, K), g), ints((rows, N), g)
        y = torch.empty(rows, N, dtype=F32, device=DEV)
        A.moe_grouped_gemm(x, w, off, y)
        assert torch.equal(y.double(), ref_fwd(x, w, off))
        dx = torch.empty(rows, K, dtype=F32, device=DEV)
        A.moe_grouped_gemm_dx(dy, w, off, dx)
        assert torch.equal(dx.double(), ref_dx(dy, w, off))
        wt = ints((E, K, N), g)   # long outer size of the weights: dx sums over it
        dyk, dxn = ints((rows, K), g), torch.empty(rows, N, dtype=F32, device=DEV)
        A.moe_grouped_gemm_dx(dyk, wt, off, dxn)
        assert torch.equal(dxn.double(), ref_dx(dyk, wt, off))
        a = fp8_inputs(E, rows, K, N, g)
        A.moe_grouped_gemm_fp8(*a, off, y)
        assert torch.equal(y.double(), ref_fp8(*a, off))


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_many_rows_over_long_inner_sizes(dt):
    """Tiles of many rows (pairs of CTAs) whose inner sizes take several partial sums and several rounds
    of the stages, off every tile edge."""
    counts, K, N = [600, 0, 257, 3], 1552, 1160
    g, rows, E = gen(15), sum(counts), len(counts)
    off = offsets_of(counts)
    x, w, dy = ints((rows, K), g), ints((E, N, K), g), ints((rows, N), g)
    y, dx = torch.empty(rows, N, dtype=dt, device=DEV), torch.empty(rows, K, dtype=dt, device=DEV)
    A.moe_grouped_gemm(x, w, off, y)
    assert torch.equal(y, ref_fwd(x, w, off).to(dt))
    A.moe_grouped_gemm_dx(dy, w, off, dx)
    assert torch.equal(dx, ref_dx(dy, w, off).to(dt))
    a = fp8_inputs(E, rows, K, N, g)
    A.moe_grouped_gemm_fp8(*a, off, y)
    assert torch.equal(y, ref_fp8(*a, off).to(dt))


def test_overlapping_ranges_end():
    """Ranges that share rows make more tiles than a call of these sizes can need.  What the shared rows
    get is one of the experts' products (here the same for all), and the call ends."""
    rows, E, K, N = 4, 9, 2048, 128
    g = gen(16)
    off = torch.tensor([0, 4] * 5, dtype=torch.int32, device=DEV)[: E + 1]     # (0,4) (4,0) (0,4) ...
    x, w = ints((rows, K), g), ints((1, N, K), g).expand(E, N, K).contiguous()
    y = torch.empty(rows, N, dtype=F32, device=DEV)
    A.moe_grouped_gemm(x, w, off, y)
    assert torch.equal(y.double(), x.double() @ w[0].double().t())
    a = list(fp8_inputs(1, rows, K, N, g))
    a[2], a[3] = a[2].expand(E, N, K).contiguous(), a[3].expand(E, 1, 16).contiguous()
    A.moe_grouped_gemm_fp8(*a, off, y)
    assert torch.equal(y.double(), ref_fp8(a[0], a[1], a[2][:1], a[3][:1], offsets_of([rows])))
    assert A.moe_get_device_error() == 0


def _norm_bound(K, S, ref, dt):
    """Elementwise bound for normal inputs: the output's rounding (half a step) plus the fp32 sums.
    A sum of K exact products in any order and grouping, every addition off by at most one unit in
    the last place (2^-23, truncation included) of a partial sum that S = sum |terms| bounds."""
    half = {F32: 2.0 ** -24, BF: 2.0 ** -8}[dt]
    return half * ref.abs() + (K + 8) * 2.0 ** -23 * S * (1 + half)


def test_normal_inputs_within_the_rounding_bound():
    counts, K, N = [5, 0, 300, 64], 1032, 520
    g, rows, E = gen(5), sum(counts), len(counts)
    off = offsets_of(counts)
    x = torch.randn(rows, K, generator=g, device=DEV).to(BF)
    w = (0.02 * torch.randn(E, N, K, generator=g, device=DEV)).to(BF)
    dy = torch.randn(rows, N, generator=g, device=DEV).to(BF)
    for dt in (F32, BF):
        y, dx, dw = (torch.empty(s, dtype=dt, device=DEV) for s in ((rows, N), (rows, K), (E, N, K)))
        A.moe_grouped_gemm(x, w, off, y)
        A.moe_grouped_gemm_dx(dy, w, off, dx)
        A.moe_grouped_gemm_dw(dy, x, off, dw)
        for got, f, a, b, terms in ((y, ref_fwd, x, w, K), (dx, ref_dx, dy, w, N), (dw, ref_dw, dy, x, max(counts))):
            ref, S = f(a, b, off), f(a.abs(), b.abs(), off)
            assert bool(((got.double() - ref).abs() <= _norm_bound(terms, S, ref, dt)).all())
            # random signs: the sums' own error stays far below that bound, 2-norm well under 1e-5
            if dt == F32:
                assert float((got.double() - ref).norm() / ref.norm()) < 1e-5


def test_fp8_arbitrary_scales_within_the_rounding_bound():
    """Scales of any magnitude and sign: (xs ws) rounded once, one product and one sum per block."""
    counts, K, N = [5, 0, 300, 64], 1040, 520
    g, rows, E = gen(6), sum(counts), len(counts)
    off = offsets_of(counts)
    xq = torch.randn(rows, K, generator=g, device=DEV).mul(50).to(F8)
    wq = torch.randn(E, N, K, generator=g, device=DEV).mul(50).to(F8)
    xs = torch.randn(9, rows, generator=g, device=DEV)
    ws = torch.randn(E, 5, 9, generator=g, device=DEV) * 1e-4
    ref = ref_fp8(xq, xs, wq, ws, off)
    S = ref_fp8(xq.to(F32).abs().to(F8), xs.abs(), wq.to(F32).abs().to(F8), ws.abs(), off)
    for dt in (F32, BF):
        y = torch.empty(rows, N, dtype=dt, device=DEV)
        A.moe_grouped_gemm_fp8(xq, xs, wq, ws, off, y)
        assert bool(((y.double() - ref).abs() <= _norm_bound(K + 4, S, ref, dt)).all())


def test_gradients_are_the_forward_products_differences():
    """The product is linear, so a difference of two forward calls is a derivative, exact on integers:
    <dy, F(x + d, w) - F(x, w)> = <dx, d> and <dy, F(x, w + d) - F(x, w)> = <dW, d>."""
    counts, K, N = [3, 0, 40, 1], 136, 72
    g, rows, E = gen(7), sum(counts), len(counts)
    off = offsets_of(counts)
    x, w, dy, d, dw_ = (ints(s, g, 2) for s in ((rows, K), (E, N, K), (rows, N), (rows, K), (E, N, K)))

    def F(x, w):
        y = torch.empty(rows, N, dtype=F32, device=DEV)
        A.moe_grouped_gemm(x, w, off, y)
        return y.double()

    dx = torch.empty(rows, K, dtype=F32, device=DEV)
    gw = torch.empty(E, N, K, dtype=F32, device=DEV)
    A.moe_grouped_gemm_dx(dy, w, off, dx)
    A.moe_grouped_gemm_dw(dy, x, off, gw)
    assert float((dy.double() * (F(x + d, w) - F(x, w))).sum()) == float((dx.double() * d.double()).sum())
    assert float((dy.double() * (F(x, w + dw_) - F(x, w))).sum()) == float((gw.double() * dw_.double()).sum())


@pytest.mark.parametrize("K,N", [(72, 136), (256, 512)])
def test_rows_nobody_owns_are_neither_read_nor_written(K, N):
    """Rows before the first and behind the last expert hold NaN: outputs there keep a sentinel, and
    nothing of them reaches a result."""
    counts, before, behind = [17, 0, 130, 5], 3, 9
    g, E = gen(8), len(counts)
    rows = before + sum(counts) + behind
    off = offsets_of(counts, before)
    own = slice(before, rows - behind)
    x, w, dy = ints((rows, K), g), ints((E, N, K), g), ints((rows, N), g)
    y0, dx0, dw0 = ref_fwd(x, w, off), ref_dx(dy, w, off), ref_dw(dy, x, off)
    for t in (x, dy):
        t[:before] = float("nan")
        t[rows - behind:] = float("inf")
    y, dx = torch.full((rows, N), 7.0, dtype=F32, device=DEV), torch.full((rows, K), 7.0, dtype=F32, device=DEV)
    dw = torch.empty(E, N, K, dtype=F32, device=DEV)
    A.moe_grouped_gemm(x, w, off, y)
    A.moe_grouped_gemm_dx(dy, w, off, dx)
    A.moe_grouped_gemm_dw(dy, x, off, dw)
    for got, ref in ((y, y0), (dx, dx0)):
        assert torch.equal(got[own].double(), ref[own])
        assert bool((got[:before] == 7).all() and (got[rows - behind:] == 7).all())
    assert torch.equal(dw.double(), dw0)
    K16 = (K + 15) // 16 * 16
    a = fp8_inputs(E, rows, K16, N, g)
    ref = ref_fp8(*a, off)
    a[1][:, :before] = float("nan")
    a[1][:, rows - behind:] = float("inf")
    y = torch.full((rows, N), 7.0, dtype=F32, device=DEV)
    A.moe_grouped_gemm_fp8(*a, off, y)
    assert torch.equal(y[own].double(), ref[own])
    assert bool((y[:before] == 7).all() and (y[rows - behind:] == 7).all())


def test_one_experts_nan_stays_its_own():
    """NaN and infinity in one expert's rows or weights leave the other experts' results exact, also
    where a tile's rows or a step of the sum over rows crosses into the neighbour."""
    counts, K, N = [19, 21, 50], 200, 136
    g, rows, E = gen(9), sum(counts), len(counts)
    off = offsets_of(counts)
    x, w, dy = ints((rows, K), g), ints((E, N, K), g), ints((rows, N), g)
    y0, dx0, dw0 = ref_fwd(x, w, off), ref_dx(dy, w, off), ref_dw(dy, x, off)
    x[19:40], dy[19:40], w[1] = float("nan"), float("inf"), float("nan")
    y, dx = torch.empty(rows, N, dtype=F32, device=DEV), torch.empty(rows, K, dtype=F32, device=DEV)
    dw = torch.empty(E, N, K, dtype=F32, device=DEV)
    A.moe_grouped_gemm(x, w, off, y)
    A.moe_grouped_gemm_dx(dy, w, off, dx)
    A.moe_grouped_gemm_dw(dy, x, off, dw)
    for got, ref in ((y, y0), (dx, dx0)):
        assert torch.equal(got[:19].double(), ref[:19]) and torch.equal(got[40:].double(), ref[40:])
        assert bool(torch.isnan(got[19:40]).all())
    assert torch.equal(dw[0].double(), dw0[0]) and torch.equal(dw[2].double(), dw0[2])
    assert bool(torch.isnan(dw[1]).all())


def test_bad_ranges_count_as_empty():
    K, N, rows = 72, 136, 64
    g = gen(10)
    off = torch.tensor([0, 10, 5, 30, 200, 64, -4, 64], dtype=torch.int32, device=DEV)
    E = off.numel() - 1     # (0,10) ok, (10,5) down, (5,30) ok, (30,200) (200,64) outside, (64,-4) down, (-4,64) outside
    off[2] = 10             # (10,10) empty, (10,30) ok: no two experts share a row
    x, w, dy = ints((rows, K), g), ints((E, N, K), g), ints((rows, N), g)
    y, dx = torch.full((rows, N), 7.0, dtype=F32, device=DEV), torch.full((rows, K), 7.0, dtype=F32, device=DEV)
    dw = torch.full((E, N, K), 7.0, dtype=F32, device=DEV)
    A.moe_grouped_gemm(x, w, off, y)
    A.moe_grouped_gemm_dx(dy, w, off, dx)
    A.moe_grouped_gemm_dw(dy, x, off, dw)
    assert torch.equal(y[:30].double(), ref_fwd(x, w, off)[:30]) and bool((y[30:] == 7).all())
    assert torch.equal(dx[:30].double(), ref_dx(dy, w, off)[:30]) and bool((dx[30:] == 7).all())
    assert torch.equal(dw.double(), ref_dw(dy, x, off))


def test_column_slices_of_wider_matrices():
    """gate | up halves in place: inputs and outputs with a leading dimension, columns around untouched."""
    counts, K, N = [33, 0, 100], 136, 264
    g, rows, E = gen(11), sum(counts), len(counts)
    off = offsets_of(counts)
    xw, dyw = ints((rows, 2 * K), g), ints((rows, N + 24), g)
    x, dy, w = xw[:, K:], dyw[:, 8:8 + N], ints((E, N, K), g)
    for dt in (F32, BF):
        yw, dxw = torch.full((rows, N + 16), 7.0, dtype=dt, device=DEV), torch.full((rows, 2 * K), 7.0, dtype=dt, device=DEV)
        A.moe_grouped_gemm(x, w, off, yw[:, 8:8 + N])
        A.moe_grouped_gemm_dx(dy, w, off, dxw[:, K:])
        assert torch.equal(yw[:, 8:8 + N], ref_fwd(x, w, off).to(dt))
        assert bool((yw[:, :8] == 7).all() and (yw[:, 8 + N:] == 7).all())
        assert torch.equal(dxw[:, K:], ref_dx(dy, w, off).to(dt)) and bool((dxw[:, :K] == 7).all())
    dw = torch.empty(E, N, K, dtype=F32, device=DEV)
    A.moe_grouped_gemm_dw(dy, x, off, dw)
    assert torch.equal(dw.double(), ref_dw(dy, x, off))
    a = list(fp8_inputs(E, rows, 144, N, g))
    wide = ints((rows, 304), g, dtype=F8)
    wide[:, 160:] = a[0]
    a[0] = wide[:, 160:]
    yw = torch.full((rows, N + 16), 7.0, dtype=BF, device=DEV)
    A.moe_grouped_gemm_fp8(*a, off, yw[:, 8:8 + N])
    assert torch.equal(yw[:, 8:8 + N], ref_fp8(*a, off).to(BF))
    assert bool((yw[:, :8] == 7).all() and (yw[:, 8 + N:] == 7).all())


def test_one_rows_stride_does_not_count():
    g = gen(18)
    x, w = ints((3, 75), g)[:1, :72], ints((1, 136, 72), g)
    y = torch.zeros(3, 139, dtype=F32, device=DEV)
    A.moe_grouped_gemm(x, w, offsets_of([1]), y[:1, :136])
    assert torch.equal(y[:1, :136].double(), ref_fwd(x, w, offsets_of([1]))) and not bool(y[1:].any() or y[:, 136:].any())


def test_misaligned_slices_are_refused():
    x, w, y = (torch.zeros(s, dtype=BF, device=DEV) for s in ((8, 72), (1, 64, 64), (8, 64)))
    off = offsets_of([8])
    for args in ((x[:, 4:68], w, off, y), (x[:, :64].contiguous(), w, off, torch.zeros(8, 68, dtype=BF, device=DEV)[:, :64])):
        with pytest.raises(A.MoeError) as e:
            A.moe_grouped_gemm(*args)
        assert e.value.code == L.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient_without_rows(accumulate):
    dw = torch.full((3, 64, 72), 7.0, dtype=BF, device=DEV)
    A.moe_grouped_gemm_dw(torch.empty(0, 64, dtype=BF, device=DEV), torch.empty(0, 72, dtype=BF, device=DEV),
                          offsets_of([0, 0, 0]), dw, accumulate=accumulate)
    assert bool((dw == (7 if accumulate else 0)).all())


def test_same_bits_every_call_and_across_streams():
    counts, K, N = [1, 0, 300, 40], 520, 1000
    g, rows, E = gen(12), sum(counts), len(counts)
    off = offsets_of(counts)
    x, w, dy = (torch.randn(s, generator=g, device=DEV).to(BF) for s in ((rows, K), (E, N, K), (rows, N)))
    q = [torch.randn(s, generator=g, device=DEV).to(F8) for s in ((rows, 528), (E, N, 528))]
    xs, ws = torch.rand(5, rows, generator=g, device=DEV), torch.rand(E, 8, 5, generator=g, device=DEV)
    torch.cuda.synchronize()

    def call(stream):
        with torch.cuda.stream(stream):
            y, dx, y8 = (torch.zeros(rows, n, dtype=F32, device=DEV) for n in (N, K, N))
            dw = torch.zeros(E, N, K, dtype=F32, device=DEV)
            A.moe_grouped_gemm(x, w, off, y, stream=stream)
            A.moe_grouped_gemm_dx(dy, w, off, dx, stream=stream)
            A.moe_grouped_gemm_dw(dy, x, off, dw, stream=stream)
            A.moe_grouped_gemm_fp8(q[0], xs, q[1], ws, off, y8, stream=stream)
        return y, dx, dw, y8

    streams = [torch.cuda.Stream() for _ in range(3)]
    runs = [call(s) for s in streams for _ in range(2)]     # overlapping on the GPU
    torch.cuda.synchronize()
    for r in runs[1:]:
        for a, b in zip(runs[0], r):
            assert torch.equal(a, b)


def test_captured_call_follows_new_offsets_and_data():
    K, N, E, rows = 264, 392, 4, 200
    g = gen(13)
    off = offsets_of([50, 50, 50, 50])
    x, w, dy = ints((rows, K), g), ints((E, N, K), g), ints((rows, N), g)
    y, dx = torch.empty(rows, N, dtype=F32, device=DEV), torch.empty(rows, K, dtype=F32, device=DEV)
    dw = torch.empty(E, N, K, dtype=F32, device=DEV)
    f = list(fp8_inputs(E, rows, 272, N, g))
    y8 = torch.empty(rows, N, dtype=F32, device=DEV)
    xf = torch.randn(rows, 272, generator=g, device=DEV)
    q, s = torch.empty(rows, 272, dtype=F8, device=DEV), torch.empty(3, rows, dtype=F32, device=DEV)

    def calls(stream):
        A.moe_grouped_gemm(x, w, off, y, stream=stream)
        A.moe_grouped_gemm_dx(dy, w, off, dx, stream=stream)
        A.moe_grouped_gemm_dw(dy, x, off, dw, stream=stream)
        A.moe_grouped_gemm_fp8(*f, off, y8, stream=stream)
        A.moe_fp8_quantize_act(xf, q, s, stream=stream)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(torch.cuda.current_stream())
    for k, counts in enumerate(([50, 50, 50, 50], [200, 0, 0, 0], [0, 3, 130, 67], [0, 0, 0, 0])):
        off.copy_(offsets_of(counts))
        x.copy_(ints((rows, K), g))
        for t in (y, dx, y8, dw):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        n = sum(counts)
        assert torch.equal(y[:n].double(), ref_fwd(x, w, off)[:n]) and bool((y[n:] == 7).all())
        assert torch.equal(dx[:n].double(), ref_dx(dy, w, off)[:n])
        assert torch.equal(dw.double(), ref_dw(dy, x, off))
        assert torch.equal(y8[:n].double(), ref_fp8(*f, off)[:n])
        assert torch.equal(q.to(F32), _codes(xf)[0].to(F32))


def test_calls_back_to_back_wait_for_each_other():
    """Kernels may start while the one before them ends: every call of a chain still reads what the calls
    before it wrote, and writes what they no longer read, on a stream and in a graph."""
    E, K, N, rows = 5, 256, 384, 90
    g = gen(19)
    off = offsets_of([20, 0, 33, 1, 36])
    w1, w2 = (ints((E, a, b), g, 1) for a, b in ((N, K), (K, N)))
    q1, q2 = torch.empty(E, N, K, dtype=F8, device=DEV), torch.empty(E, N, K, dtype=F8, device=DEV)
    s1 = torch.empty(E, N // 128, K // 128, device=DEV)
    s2 = torch.empty_like(s1)
    x0 = torch.randn(rows, K, generator=g, device=DEV).to(BF)
    x, y = torch.empty_like(x0), torch.empty(rows, N, dtype=BF, device=DEV)
    q, s = torch.empty(rows, K, dtype=F8, device=DEV), torch.empty(K // 128, rows, device=DEV)
    y8, dw = torch.empty(rows, N, device=DEV), torch.empty(E, N, K, device=DEV)
    ids = torch.zeros(rows, K, device=DEV)

    def chain(pause):
        st = torch.cuda.current_stream()
        x.copy_(x0)
        for i in range(12):
            for f in (lambda: A.moe_grouped_gemm(x, w1, off, y, stream=st),
                      lambda: A.moe_grouped_gemm(y, w2, off, x, stream=st),
                      lambda: x.mul_(1 / 256),
                      lambda: A.moe_grouped_gemm_dw(y, x, off, dw, accumulate=i > 0, stream=st),
                      lambda: A.moe_fp8_quantize_act(x, q, s, stream=st),
                      lambda: A.moe_fp8_quantize_weight(dw, q1 if i % 2 else q2, s1 if i % 2 else s2, stream=st),
                      lambda: A.moe_grouped_gemm_fp8(q, s, q1 if i % 2 else q2, s1 if i % 2 else s2, off, y8, stream=st),
                      lambda: ids.add_(y8[:, :K])):
                f()
                if pause:
                    torch.cuda.synchronize()

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (x, y, dw, y8, ids, s, s1, s2, q.to(F32), q1.to(F32), q2.to(F32))]

    chain(True)
    want = results()
    assert all(bool(torch.isfinite(t).all()) for t in want) and bool(want[3].any())
    ids.zero_()
    chain(False)
    assert all(torch.equal(a, b) for a, b in zip(results(), want))
    ids.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(False)
    for _ in range(3):
        ids.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))


def test_first_call_of_a_process_may_be_a_captured_one():
    """Nothing a first call sets up (limits, symbols) is refused while a stream is being captured."""
    code = """
import torch
from expert_cached_sparse_b200 import api as A
d, bf, f8 = "cuda", torch.bfloat16, torch.float8_e4m3fn
for counts in ([1, 2], [300, 20]):
    rows, K, N = sum(counts), 128, 256
    off = torch.tensor([0, counts[0], rows], dtype=torch.int32, device=d)
    x, w, dy = (torch.ones(s, device=d).to(bf) for s in ((rows, K), (2, N, K), (rows, N)))
    q, wq = (torch.empty(s, dtype=f8, device=d) for s in ((rows, K), (2, N, K)))
    s, ws = torch.empty(1, rows, device=d), torch.empty(2, 2, 1, device=d)
    outs = []
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = torch.cuda.current_stream()
        for t in (torch.float32, bf):
            y, y8, dx, dw = (torch.empty(s, dtype=t, device=d) for s in ((rows, N), (rows, N), (rows, K), (2, N, K)))
            A.moe_grouped_gemm(x, w, off, y, stream=st)
            A.moe_grouped_gemm_dx(dy, w, off, dx, stream=st)
            A.moe_grouped_gemm_dw(dy, x, off, dw, stream=st)
            A.moe_fp8_quantize_act(x, q, s, stream=st)
            A.moe_fp8_quantize_weight(w, wq, ws, stream=st)
            A.moe_grouped_gemm_fp8(q, s, wq, ws, off, y8, stream=st)
            outs += [(y, K), (dx, N), (y8, K), (dw[0], counts[0]), (dw[1], counts[1])]
    for o, _ in outs:
        o.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    for i, (o, v) in enumerate(outs):
        want = torch.full((), v, device=d).to(o.dtype).float()
        assert bool(((o.float() - want).abs() <= 1e-6 * v).all()), (i, v, o.flatten()[:4])
print("done")
"""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                         cwd=pathlib.Path(__file__).resolve().parents[1])
    assert out.returncode == 0 and "done" in out.stdout, out.stderr[-2000:]


@pytest.mark.parametrize("rows", [500, 70000])
def test_as_many_experts_as_allowed(rows):
    """4096 experts: the tables take most of what the stages leave."""
    E, K, N = 4096, 80, 136
    g = gen(17)
    cut = torch.sort(torch.randint(0, rows + 1, (E - 1,), generator=g, device=DEV))[0]
    off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), rows)]).to(torch.int32)
    x, w, dy = ints((rows, K), g, 1), ints((E, N, K), g, 1), ints((rows, N), g, 1)
    own = torch.repeat_interleave(torch.arange(E, device=DEV), off.diff().long())
    step = 5000

    def rowwise(a, m):   # rows with their own matrix
        return torch.cat([torch.einsum("rk,rnk->rn", a[i:i + step].to(F32), m[own[i:i + step]].to(F32))
                                        for i in range(0, rows, step)])

    y, dx = torch.empty(rows, N, dtype=F32, device=DEV), torch.empty(rows, K, dtype=F32, device=DEV)
    A.moe_grouped_gemm(x, w, off, y)
    assert torch.equal(y, rowwise(x, w))
    A.moe_grouped_gemm_dx(dy, w, off, dx)
    assert torch.equal(dx, rowwise(dy, w.transpose(1, 2)))
    dw, want = (torch.zeros(E, N, K, dtype=F32, device=DEV) for _ in range(2))
    A.moe_grouped_gemm_dw(dy, x, off, dw)
    for i in range(0, rows, step):
        want.index_add_(0, own[i:i + step], dy[i:i + step].to(F32)[:, :, None] * x[i:i + step].to(F32)[:, None, :])
    assert torch.equal(dw, want)
    a = fp8_inputs(E, rows, K, N, g)
    A.moe_grouped_gemm_fp8(*a, off, y)
    want = rowwise(a[0].to(F32), a[2].to(F32)) * a[1][0][:, None] * a[3][own, :, 0].repeat_interleave(128, 1)[:, :N]
    assert torch.equal(y, want)


def test_offsets_past_32_bits():
    """Rows and weights whose element offsets pass 2^31 and 2^32."""
    g = gen(14)
    K, N, ld, rows = 64, 72, 65536, 66000               # rows x ld = 4.3e9 elements
    store = torch.empty(rows * ld, dtype=BF, device=DEV)
    x = store.as_strided((rows, K), (ld, 1))
    x.copy_(ints((rows, K), g))
    counts = [rows - 300, 0, 300]
    off, w = offsets_of(counts), ints((3, N, K), g)
    y = store.as_strided((rows, N), (ld, 1), 1024)        # the output in other columns of the same rows
    A.moe_grouped_gemm(x, w, off, y)
    assert torch.equal(y, ref_fwd(x, w, off).to(BF))
    dw = torch.empty(3, N, K, dtype=F32, device=DEV)
    dy = ints((rows, N), g, 1)
    y.copy_(dy)
    A.moe_grouped_gemm_dw(y, x, off, dw)
    assert torch.equal(dw.double(), ref_dw(dy, x, off))
    dx = store.as_strided((rows, K), (ld, 1), 2048)
    A.moe_grouped_gemm_dx(y, w, off, dx)
    assert torch.equal(dx, ref_dx(dy, w, off).to(BF))
    del store, x, y, dx
    torch.cuda.empty_cache()
    E, K, N = 260, 4096, 4096                            # 4.4e9 weight elements
    counts = [0] * E
    counts[3], counts[130], counts[E - 1] = 2, 1, 3
    off, rows = offsets_of(counts), 6
    w = torch.empty(E, N, K, dtype=BF, device=DEV)
    for e in (3, 130, E - 1):
        w[e] = ints((N, K), g)
    x, y = ints((rows, K), g), torch.empty(rows, N, dtype=F32, device=DEV)
    A.moe_grouped_gemm(x, w, off, y)
    assert torch.equal(y.double(), ref_fwd(x, w, off))
    dx = torch.empty(rows, K, dtype=F32, device=DEV)
    A.moe_grouped_gemm_dx(x, w, off, dx)
    assert torch.equal(dx.double(), ref_dx(x, w, off))
    A.moe_grouped_gemm_dw(x, x, off, w)                   # bf16 gradients over the same store
    last = x[3:].to(F64)
    assert torch.equal(w[E - 1], (last.t() @ last).to(BF)) and not bool(w[4:130].any())


# ------------------------------------------------------------------ quantisation
def _codes(v):
    """Codes [rows][cols] and scales [blocks][rows] of float32 rows, fp32 arithmetic on the CPU."""
    v = v.detach().float().cpu()
    r, K = v.shape
    kb = (K + 127) // 128
    p = torch.nn.functional.pad(v, (0, kb * 128 - K)).view(r, kb, 128)
    m = torch.nan_to_num(p, nan=0.0, posinf=float("inf"), neginf=float("-inf")).abs().amax(2)
    s = torch.where(m < 2.0 ** -100, torch.ones_like(m), m / 448.0)
    q = (p / s[:, :, None]).view(r, kb * 128)[:, :K].to(F8)
    return q.to(DEV), s.t().contiguous().to(DEV)


def same_codes(a, b):
    """Equal values; a NaN equals a NaN whatever its sign."""
    a, b = a.to(F32), b.to(F32)
    return bool((torch.isnan(a) == torch.isnan(b)).all()) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 4096), (3, 136), (16, 128), (17, 1000), (301, 2048), (5, 264)])
def test_quantize_rows_bit_exact(dt, rows, cols):
    g = gen(20)
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x *= torch.randint(-20, 20, (rows, 1), generator=g, device=DEV).to(F32).exp2()
    x = x.to(dt)
    q, s = torch.empty(rows, cols, dtype=F8, device=DEV), torch.empty((cols + 127) // 128, rows, device=DEV)
    A.moe_fp8_quantize_act(x, q, s)
    qr, sr = _codes(x)
    assert torch.equal(s, sr) and same_codes(q, qr)


def test_quantize_special_values():
    x = torch.zeros(8, 256, device=DEV)
    x[1, :128] = 2.0 ** -101                    # below the smallest block: scale 1, zeros
    x[2, :128] = 2.0 ** -99
    x[3, 5], x[3, 6] = float("nan"), 3.0
    x[4, 7], x[4, 8] = float("inf"), 3.0
    x[5, 200] = -float("inf")
    x[6] = 3.0e38
    x[7, 0], x[7, 1] = -448.0, 1.0 / 1024       # ties and subnormal codes at scale 1
    q, s = torch.empty(8, 256, dtype=F8, device=DEV), torch.empty(2, 8, device=DEV)
    A.moe_fp8_quantize_act(x, q, s)
    qr, sr = _codes(x)
    assert torch.equal(s, sr) and same_codes(q, qr)
    assert float(s[0, 0]) == 1 and float(s[0, 1]) == 1 and not bool(q[:2].to(F32).any())
    v = q.to(F32) * s.t().repeat_interleave(128, 1)
    assert bool(torch.isnan(v[3, 5])) and abs(float(v[3, 6]) - 3) < 1e-6 and bool(torch.isnan(v[4, :128]).all())
    assert not bool(torch.isnan(v[4, 128:]).any()) and bool(torch.isnan(v[5, 128:]).all())


@pytest.mark.parametrize("exponent", [-98, 0, 120])
def test_quantize_divides_exactly_for_every_significand(exponent):
    """Block maxima of all 2^23 significands, the other values on and one step beside the midpoints of two
    codes, where a quotient off by its last bit changes the code.  (A quotient rounded to 53 bits and then
    to 24 is the one rounded to 24 at once, as 53 >= 2 * 24 + 2.)"""
    n = 1 << 21
    mid = torch.tensor([2.0 ** -10, 1.0625, 17.0, 232.0, 432.0], dtype=F64, device=DEV)
    step = torch.tensor([-1, 0, 1], dtype=torch.int32, device=DEV)
    q, s = torch.empty(n, 16, dtype=F8, device=DEV), torch.empty(1, n, device=DEV)
    for first in range(0, 1 << 23, n):
        m = torch.ldexp(1 + torch.arange(first, first + n, device=DEV).to(F64) / (1 << 23),
                        torch.tensor(exponent, device=DEV)).to(F32)
        sr = (m.to(F64) / 448).to(F32)
        near = (sr.to(F64)[:, None] * mid).to(F32).view(torch.int32)
        x = torch.cat([m[:, None], (near[:, :, None] + step).view(n, 15).view(F32)], 1)
        A.moe_fp8_quantize_act(x, q, s)
        assert torch.equal(s[0], sr)
        assert torch.equal(q.to(F32), (x.to(F64) / sr.to(F64)[:, None]).to(F32).to(F8).to(F32))


def test_quantize_slices_and_untouched_columns():
    g = gen(21)
    wide = torch.randn(33, 600, generator=g, device=DEV).to(BF)
    x = wide[:, 8:280]
    qw = torch.full((33, 400), 2.0, device=DEV).to(F8)
    s = torch.empty(3, 33, device=DEV)
    A.moe_fp8_quantize_act(x, qw[:, 16:288], s)
    qr, sr = _codes(x)
    assert torch.equal(s, sr) and same_codes(qw[:, 16:288], qr)
    assert bool((qw[:, :16].to(F32) == 2).all() and (qw[:, 288:].to(F32) == 2).all())


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 8), (40, 768), (7, 200)])
def test_quantize_swiglu(dt, rows, cols):
    """silu(gate) * up in fp32 with 2^x within 2^-22, its argument -gate log2(e) off by 1.5 |gate| 2^-24
    (constant and product), the reciprocal within 2^-23, the sum and two products within 2^-24 each: h is
    within (4 + 1.5 |gate| + 2 + 3) 2^-24 = (9 + 1.5 |gate|) 2^-24 relative, second order below one more;
    the scale follows the largest h within that and its division's 2^-24, and the code is the nearest one."""
    g = gen(22)
    x = (3 * torch.randn(rows, 2 * cols, generator=g, device=DEV)).to(dt)
    q, s = torch.empty(rows, cols, dtype=F8, device=DEV), torch.empty((cols + 127) // 128, rows, device=DEV)
    A.moe_fp8_quantize_act(x, q, s, swiglu=True)
    d = x.double()
    h = d[:, :cols] * torch.sigmoid(d[:, :cols]) * d[:, cols:]
    kb = s.shape[0]
    m = torch.nn.functional.pad(h, (0, kb * 128 - cols)).view(rows, kb, 128).abs().amax(2)
    sd = s.t().double()
    rel = (11 + 1.5 * float(d[:, :cols].abs().max())) * 2.0 ** -24
    assert bool(((sd - m / 448).abs() <= rel * (m / 448)).all())
    sx = sd[:, torch.arange(cols, device=DEV) // 128]
    half = torch.maximum(h.abs() * 2.0 ** -4, sx * 2.0 ** -10)    # half a step of e4m3, normal or subnormal
    assert bool(((q.to(F32).double() * sx - h).abs() <= half * (1 + 2.0 ** -15) + rel * h.abs()).all())


def test_quantize_swiglu_far_gates():
    """exp overflow on one side, underflow on the other: silu goes to 0 and to the gate itself."""
    x = torch.zeros(1, 256, device=DEV)
    x[0, :4] = torch.tensor([-200.0, 200.0, -1e30, 1e30])
    x[0, 128:] = 1e-3
    q, s = torch.empty(1, 128, dtype=F8, device=DEV), torch.empty(1, 1, device=DEV)
    A.moe_fp8_quantize_act(x, q, s, swiglu=True)
    v = q.to(F32)[0] * s[0, 0]
    assert bool(torch.isfinite(v).all()) and abs(float(v[3]) / 1e27 - 1) < 1e-6 and not bool(v[:3].any() or v[4:].any())


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("E,N,K", [(1, 1, 8), (3, 128, 128), (2, 130, 264), (1, 1000, 72), (5, 256, 512)])
def test_quantize_weights_bit_exact(dt, E, N, K):
    g = gen(23)
    w = (0.02 * torch.randn(E, N, K, generator=g, device=DEV)).to(dt)
    w[0, :, : min(K, 128)] = 0
    q, s = torch.empty(E, N, K, dtype=F8, device=DEV), torch.empty(E, (N + 127) // 128, (K + 127) // 128, device=DEV)
    A.moe_fp8_quantize_weight(w, q, s)
    c = w.float().cpu()
    for e in range(E):
        for i in range(s.shape[1]):
            for j in range(s.shape[2]):
                b = c[e, 128 * i:128 * i + 128, 128 * j:128 * j + 128]
                m = b.abs().max()
                sc = m / 448.0 if m >= 2.0 ** -100 else torch.tensor(1.0)
                assert float(s[e, i, j]) == float(sc)
                assert same_codes(q[e, 128 * i:128 * i + 128, 128 * j:128 * j + 128].cpu(), (b / sc).to(F8))


# ------------------------------------------------------------------ together
def _route(n, E, k, H, g):
    idx = torch.rand(n, E, generator=g, device=DEV).topk(k, 1).indices.int().contiguous()
    x = torch.randn(n, H, generator=g, device=DEV).to(BF)
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    row_of, assign_of = (torch.empty(n * k, dtype=torch.int32, device=DEV) for _ in range(2))
    xp = torch.empty(n * k, H, dtype=BF, device=DEV)
    ws = torch.empty(A.moe_permute_workspace_bytes(n, E, k), dtype=torch.uint8, device=DEV)
    A.moe_permute(idx, n, E, k, x, H, off, row_of, assign_of, xp, ws)
    tw = torch.softmax(torch.randn(n, k, generator=g, device=DEV), 1)
    return x, idx, off, row_of, assign_of, xp, tw


@pytest.mark.parametrize("n", [1, 37])
def test_a_layer_of_products_matches_the_fused_ffn_and_its_gradients(n):
    """permute -> products -> SwiGLU -> product -> combine against the packed BF16 expert FFN and 64 bits,
    then the whole layer backward against autograd in 64 bits."""
    E, k, H, F = 8, 2, 256, 192
    g = gen(30)
    x, idx, off, row_of, assign_of, xp, tw = _route(n, E, k, H, g)
    w13 = (0.05 * torch.randn(E, 2 * F, H, generator=g, device=DEV)).to(BF)
    w2 = (0.05 * torch.randn(E, H, F, generator=g, device=DEV)).to(BF)
    rows = n * k
    gu = torch.empty(rows, 2 * F, dtype=F32, device=DEV)
    A.moe_grouped_gemm(xp, w13, off, gu)
    h = (torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]).to(BF)
    y = torch.empty(rows, H, dtype=BF, device=DEV)
    A.moe_grouped_gemm(h, w2, off, y)
    out = torch.empty(n, H, dtype=BF, device=DEV)
    A.moe_combine(y, row_of, tw, n, k, H, out)

    # 64 bits, with gradients
    X, W13, W2 = (t.double().requires_grad_() for t in (x, w13, w2))
    O = torch.zeros(n, H, dtype=F64, device=DEV)
    for j in range(k):
        e = idx[:, j].long()
        a = torch.einsum("toh,th->to", W13[e], X)
        hh = torch.nn.functional.silu(a[:, :F]) * a[:, F:]
        O = O + tw[:, j:j + 1].double() * torch.einsum("thf,tf->th", W2[e], hh)
    # h, y and out rounded to bf16 (half a step, 2^-8, each) on the way: three roundings
    assert float((out.double() - O).norm() / O.norm()) < 3 * 2.0 ** -8

    # the packed path on the same experts
    shape = A.make_shape(1, E, H, F, k, A.W_BF16)
    class Ew:
        w13_scales = w2_scales = None
        tensor_scales = np.zeros(2, np.float32)
    pool = []
    for e in range(E):
        ew = Ew()
        ew.w13 = w13[e].cpu().view(torch.int16).numpy().view(np.uint16)
        ew.w2 = w2[e].cpu().view(torch.int16).numpy().view(np.uint16)
        pool.append(A.moe_pack_expert(shape, ew))
    pool = torch.from_numpy(np.concatenate(pool)).to(DEV)
    y2 = torch.empty_like(y)
    wsf = torch.empty(A.moe_ffn_workspace_bytes(shape, rows), dtype=torch.uint8, device=DEV)
    A.moe_grouped_ffn(shape, pool, E, torch.arange(E, dtype=torch.int32, device=DEV), off, xp, rows, y2, wsf)
    assert float((y.double() - y2.double()).norm() / y.double().norm()) < 2 * 2.0 ** -8

    # backward: d out -> d y (rows) -> d h, dW2 -> d gate|up -> dW13, d x
    dout = torch.randn(n, H, generator=g, device=DEV).to(BF)
    O.backward(dout.double())
    tok = assign_of.long() // k
    wr = tw.flatten()[assign_of.long()]
    dy = (wr[:, None] * dout[tok].float()).to(BF)
    dh = torch.empty(rows, F, dtype=F32, device=DEV)
    A.moe_grouped_gemm_dx(dy, w2, off, dh)
    dw2 = torch.empty(E, H, F, dtype=F32, device=DEV)
    A.moe_grouped_gemm_dw(dy, h, off, dw2)
    gate, up = gu[:, :F], gu[:, F:]
    sg = torch.sigmoid(gate)
    dgu = torch.cat([dh * up * sg * (1 + gate * (1 - sg)), dh * gate * sg], 1).to(BF)
    dxp = torch.empty(rows, H, dtype=F32, device=DEV)
    A.moe_grouped_gemm_dx(dgu, w13, off, dxp)
    dw13 = torch.zeros(E, 2 * F, H, dtype=F32, device=DEV)
    for _ in range(2):                                     # two halves of a batch would add up alike
        A.moe_grouped_gemm_dw(dgu, xp, off, dw13, accumulate=True)
    dx = torch.zeros(n, H, device=DEV).index_add_(0, tok, dxp)
    # roundings on each path: dy, h (dW2); dy, dgu (dx, dW13): two of 2^-8 each
    for got, ref in ((dw2, W2.grad), (dw13 / 2, W13.grad), (dx, X.grad)):
        assert float((got.double() - ref).norm() / ref.norm()) < 2 * 2.0 ** -8


def test_an_fp8_layer_together():
    """quantise -> product -> SwiGLU and quantise -> product -> combine, against 64 bits on the same codes."""
    E, k, H, F, n = 8, 2, 400, 272, 45
    g = gen(31)
    x, idx, off, row_of, assign_of, xp, tw = _route(n, E, k, H, g)
    w13 = (0.05 * torch.randn(E, 2 * F, H, generator=g, device=DEV)).to(BF)
    w2 = (0.05 * torch.randn(E, H, F, generator=g, device=DEV)).to(BF)
    rows = n * k

    def qw(w):
        q = torch.empty(w.shape, dtype=F8, device=DEV)
        s = torch.empty(E, (w.shape[1] + 127) // 128, (w.shape[2] + 127) // 128, device=DEV)
        A.moe_fp8_quantize_weight(w, q, s)
        return q, s

    (q13, s13), (q2, s2) = qw(w13), qw(w2)
    xq, xs = torch.empty(rows, H, dtype=F8, device=DEV), torch.empty((H + 127) // 128, rows, device=DEV)
    A.moe_fp8_quantize_act(xp, xq, xs)
    gu = torch.empty(rows, 2 * F, dtype=F32, device=DEV)
    A.moe_grouped_gemm_fp8(xq, xs, q13, s13, off, gu)
    hq, hs = torch.empty(rows, F, dtype=F8, device=DEV), torch.empty((F + 127) // 128, rows, device=DEV)
    A.moe_fp8_quantize_act(gu, hq, hs, swiglu=True)
    y = torch.empty(rows, H, dtype=BF, device=DEV)
    A.moe_grouped_gemm_fp8(hq, hs, q2, s2, off, y)
    out = torch.empty(n, H, dtype=BF, device=DEV)
    A.moe_combine(y, row_of, tw, n, k, H, out)
    gu64 = ref_fp8(xq, xs, q13, s13, off)
    assert float((gu.double() - gu64).norm() / gu64.norm()) < 1e-5
    y64 = ref_fp8(hq, hs, q2, s2, off)
    assert float((y.double() - y64).norm() / y64.norm()) < 2.0 ** -8
    # the whole against the unquantised experts: four quantisations, each off by at most 2^-4 relative per element
    e = torch.searchsorted(off[1:].long(), torch.arange(rows, device=DEV), right=True)
    a = torch.einsum("toh,th->to", w13.double()[e], xp.double())
    hh = torch.nn.functional.silu(a[:, :F]) * a[:, F:]
    yy = torch.einsum("thf,tf->th", w2.double()[e], hh)
    ref = torch.zeros(n, H, dtype=F64, device=DEV).index_add_(0, assign_of.long() // k,
                                                              tw.flatten()[assign_of.long()][:, None].double() * yy)
    assert float((out.double() - ref).norm() / ref.norm()) < 4 * 2.0 ** -4


def test_products_behind_the_fused_ffn_wait_for_it_and_are_profiled():
    """A product and a quantiser launched right behind the fused FFN (whose kernels let the next one start
    early) read all that it wrote.  (Rows are normalised once a turn: the FFN squares their size.)"""
    E, k, H, F, n = 8, 2, 256, 192, 64
    g = gen(31)
    _, _, off, _, _, xp, _ = _route(n, E, k, H, g)
    rows = n * k
    shape = A.make_shape(1, E, H, F, k, A.W_BF16)

    class Ew:
        w13_scales = w2_scales = None
        tensor_scales = np.zeros(2, np.float32)

    pool = []
    for e in range(E):
        ew = Ew()
        for name, s in (("w13", (2 * F, H)), ("w2", (H, F))):
            w = (0.3 * torch.randn(s, generator=g, device=DEV)).to(BF)
            setattr(ew, name, w.cpu().view(torch.int16).numpy().view(np.uint16))
        pool.append(A.moe_pack_expert(shape, ew))
    pool = torch.from_numpy(np.concatenate(pool)).to(DEV)
    w = (0.1 * torch.randn(E, H, H, generator=g, device=DEV)).to(BF)
    slots = torch.arange(E, dtype=torch.int32, device=DEV)
    wsf = torch.empty(A.moe_ffn_workspace_bytes(shape, rows), dtype=torch.uint8, device=DEV)
    x, y = torch.empty_like(xp), torch.empty_like(xp)
    q, s = torch.empty(rows, H, dtype=F8, device=DEV), torch.empty(H // 128, rows, device=DEV)

    def chain(pause):
        st = torch.cuda.current_stream()
        x.copy_(xp)
        for _ in range(8):
            for f in (lambda: A.moe_grouped_ffn(shape, pool, E, slots, off, x, rows, y, wsf, stream=st),
                      lambda: A.moe_grouped_gemm(y, w, off, x, stream=st),
                      lambda: x.copy_(torch.nn.functional.layer_norm(x.float(), (H,))),
                      lambda: A.moe_grouped_ffn(shape, pool, E, slots, off, x, rows, y, wsf, stream=st),
                      lambda: A.moe_fp8_quantize_act(y, q, s, stream=st)):
                f()
                if pause:
                    torch.cuda.synchronize()

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (x, y, q.to(F32), s)]

    chain(True)
    want = results()
    assert bool(torch.isfinite(want[0]).all()) and bool(want[0].any())
    A.moe_profile_enable(True)
    try:
        A.moe_profile_read(reset=True)
        chain(False)
        got = results()
        counts = A.moe_profile_read(reset=True)
    finally:
        A.moe_profile_enable(False)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert counts["gemm"]["launches"] == 8 and counts["quant"]["launches"] == 8 and counts["gemm"]["ms"] > 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(False)
    for _ in range(3):
        for t in (x, y, s):
            t.fill_(7)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
