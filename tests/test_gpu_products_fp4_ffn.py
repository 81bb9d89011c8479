"""Products and quantisers between grouped FFN calls on FP4 weights: the fused decode kernel, the separate
decode tiles and the prefill tiles (whose kernels let the next one start before they have waited themselves).
Every call reads what the one before it wrote: the bits of a chain with a pause after each call are those
of the chain without, on a stream and in a graph."""
import numpy as np
import pytest
import torch

from expert_cached_sparse_b200 import api as A
from expert_cached_sparse_b200 import workloads as W

pytestmark = pytest.mark.gpu
BF, F8, DEV = torch.bfloat16, torch.float8_e4m3fn, "cuda"


@pytest.mark.parametrize("path", ["fused", "decode", "prefill"])
@pytest.mark.parametrize("base", [W.DS_DECODE, W.TRACE40], ids=["mxfp4", "nvfp4"])
def test_chain(base, path, monkeypatch):
    monkeypatch.setenv("MOE_FFN_TILE", "prefill" if path == "prefill" else "decode")
    monkeypatch.delenv("MOE_FFN_UNFUSED", raising=False)
    if path == "decode":
        monkeypatch.setenv("MOE_FFN_UNFUSED", "1")
    counts = [3, 0, 17, 1, 40, 2] if path == "prefill" else [3, 0, 2, 1, 5, 1]
    cfg = W.scaled(base, hidden=512, ffn=256, experts=6, top_k=2, layers=1)
    shape, E, H, rows = A.shape_of(cfg), cfg.experts, 512, sum(counts)
    pool = torch.from_numpy(np.concatenate([A.moe_pack_expert(shape, W.gen_expert(cfg, 4, 0, e)) for e in range(E)])).to(DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(70)
    off = torch.tensor([sum(counts[:e]) for e in range(E + 1)], dtype=torch.int32, device=DEV)
    slots = torch.arange(E, dtype=torch.int32, device=DEV)
    x0 = torch.randn(rows, H, generator=g, device=DEV).to(BF)
    w = (0.05 * torch.randn(E, H, H, generator=g, device=DEV)).to(BF)
    x, y, dx = torch.empty_like(x0), torch.empty_like(x0), torch.empty_like(x0)
    q, s, dw = torch.empty(rows, H, dtype=F8, device=DEV), torch.empty(H // 128, rows, device=DEV), torch.empty(E, H, H, device=DEV)
    ws = torch.empty(A.moe_ffn_workspace_bytes(shape, rows), dtype=torch.uint8, device=DEV)

    def chain(pause):
        st = torch.cuda.current_stream()
        x.copy_(x0)
        for i in range(6):
            for f in (lambda: A.moe_grouped_ffn(shape, pool, E, slots, off, x, rows, y, ws, stream=st),
                      lambda: A.moe_grouped_gemm(y, w, off, x, stream=st),
                      lambda: A.moe_fp8_quantize_act(x, q, s, stream=st),
                      lambda: x.copy_(torch.nn.functional.layer_norm(x.float(), (H,))),
                      lambda: A.moe_grouped_gemm_dx(x, w, off, dx, stream=st),
                      lambda: A.moe_grouped_ffn(shape, pool, E, slots, off, dx, rows, y, ws, stream=st),
                      lambda: A.moe_grouped_gemm_dw(y, x, off, dw, accumulate=i > 0, stream=st)):
                f()
                if pause:
                    torch.cuda.synchronize()

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (x, y, dx, dw, s, q.to(torch.float32))]

    chain(True)
    want = results()
    assert all(bool(torch.isfinite(t.float()).all()) and bool(t.any()) for t in want)
    for _ in range(3):
        chain(False)
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(False)
    for _ in range(3):
        for t in (x, y, dx, dw, s):
            t.fill_(7)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
    assert A.moe_get_device_error() == 0
