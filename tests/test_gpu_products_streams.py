"""Products and quantisers whose inputs come from another stream, or from a copy or a fill: a kernel that may
start while the one before it on its stream ends still waits for everything else that it depends on."""
import pytest
import torch

from expert_cached_sparse_b200 import api as A

pytestmark = pytest.mark.gpu
BF, F32, F8, DEV = torch.bfloat16, torch.float32, torch.float8_e4m3fn, "cuda"


def ints(shape, g):
    return torch.randint(-3, 4, shape, generator=g, device=DEV).to(F32).to(BF)


@pytest.mark.parametrize("captured", [False, True], ids=["stream", "graph"])
def test_events_between_two_streams(captured):
    """Stream a makes the rows, stream b multiplies them right behind another product of its own, and a
    overwrites them again once b has read them."""
    g = torch.Generator(device=DEV)
    g.manual_seed(80)
    E, K, N, rows = 6, 512, 768, 600
    off = torch.tensor([100 * e for e in range(E + 1)], dtype=torch.int32, device=DEV)
    src = [ints((rows, K), g) for _ in range(4)]
    w = ints((E, N, K), g)
    want = [torch.bmm(s.float().view(E, 100, K), w.float().transpose(1, 2)).view(rows, N) for s in src]
    x, other = torch.empty(rows, K, dtype=BF, device=DEV), ints((rows, K), g)
    ys, y0 = [torch.empty(rows, N, device=DEV) for _ in src], torch.empty(rows, N, device=DEV)
    big = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    q, s = torch.empty(rows, K, dtype=F8, device=DEV), torch.empty(K // 128, rows, device=DEV)
    dw = torch.empty(E, N, K, device=DEV)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        a.wait_stream(torch.cuda.current_stream())
        b.wait_stream(torch.cuda.current_stream())
        for i, t in enumerate(src):
            with torch.cuda.stream(a):
                big.fill_(i)                      # late, so that b gets there first
                x.copy_(t)
                made = a.record_event()
            with torch.cuda.stream(b):
                A.moe_grouped_gemm(other, w, off, y0, stream=b)
                b.wait_event(made)
                A.moe_grouped_gemm(x, w, off, ys[i], stream=b)
                A.moe_fp8_quantize_act(x, q, s, stream=b)
                A.moe_grouped_gemm_dw(other[:, :K].new_zeros(rows, N), x, off, dw, stream=b)
                a.wait_event(b.record_event())
        torch.cuda.current_stream().wait_stream(a)
        torch.cuda.current_stream().wait_stream(b)

    work()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            work()
    for _ in range(5):
        for t in ys:
            t.fill_(7)
        x.fill_(5)
        graph.replay() if captured else work()
        torch.cuda.synchronize()
        assert all(torch.equal(t, r) for t, r in zip(ys, want))
        assert not bool(dw.any())


def test_behind_fills_and_copies_in_a_graph():
    """A weight gradient without rows is a fill; copies of packed tensors are no kernels either."""
    g = torch.Generator(device=DEV)
    g.manual_seed(81)
    off, none = torch.tensor([0, 40, 40, 130], dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    x0, w, dy = ints((130, 256), g), ints((3, 128, 256), g), ints((130, 128), g)
    x, y, dw = torch.empty_like(x0), torch.empty(130, 128, device=DEV), torch.empty(3, 128, 256, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = torch.cuda.current_stream()
        A.moe_grouped_gemm(x, w, off, y, stream=st)
        x.copy_(x0)
        A.moe_grouped_gemm(x, w, off, y, stream=st)
        A.moe_grouped_gemm_dw(dy[:0], x[:0], none, dw, stream=st)
        A.moe_grouped_gemm_dw(dy, x, off, dw, accumulate=True, stream=st)
    for _ in range(3):
        for t in (x, y, dw):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for e, (lo, hi) in enumerate(((0, 40), (40, 40), (40, 130))):
            assert torch.equal(y[lo:hi], x0[lo:hi].float() @ w[e].float().t())
            assert torch.equal(dw[e], dy[lo:hi].float().t() @ x0[lo:hi].float())


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
def test_quantised_weights_special_values(dt):
    """The rule for rows holds for blocks of weights: a NaN is left out of the maximum and keeps a NaN code,
    an infinity makes its own block's scale infinite, tiny blocks get scale 1 and zeros."""
    w = torch.zeros(1, 256, 384, device=DEV)
    w[0, 3, 5], w[0, 4, 6] = float("nan"), 3.0                     # block (0, 0)
    w[0, 100, 130], w[0, 101, 131] = -float("inf"), 2.0            # (0, 1)
    w[0, 0, 300] = 2.0 ** -101                                     # (0, 2)
    w[0, 200, 10], w[0, 201, 11] = 3.0e38, -1.0e38                 # (1, 0)
    w = w.to(dt)
    q, s = torch.empty(1, 256, 384, dtype=F8, device=DEV), torch.empty(1, 2, 3, device=DEV)
    A.moe_fp8_quantize_weight(w, q, s)
    c, v = s[0].tolist(), q.to(F32)[0]
    big = w[0, 200, 10].double()
    assert c[0][0] == (torch.tensor(3.0) / 448).item() and c[0][1] == float("inf") and c[0][2] == 1 and c[1][1] == 1
    assert c[1][0] == (big.cpu().float() / 448).item()
    nan = torch.isnan(v)
    assert bool(nan[3, 5]) and bool(nan[100, 130]) and int(nan.sum()) == 2
    assert v[4, 6] == 448 and v[101, 131] == 0 and v[0, 300] == 0 and v[200, 10] == 448
    assert v[201, 11] == (w[0, 201, 11] / s[0, 1, 0]).to(F8).to(F32)
    v[nan] = 0
    assert int((v != 0).sum()) == 3
