"""Bounded waits of the expert products that run out.

moe_test_set_wait shortens the wait limit and makes the first CTA's copy warps
leave their first stage unfilled.  The kernel must record MOE_ERR_TIMEOUT, let
its own copies and MMAs finish and return (no fault, no hang, the context stays
usable), pairs of CTAs included; a normal call afterwards must give the bits of
one made before.  Nothing here faults the GPU: the stage is simply never filled.
"""
import time

import pytest
import torch

from expert_cached_sparse_b200 import _lib as L
from expert_cached_sparse_b200 import api as A

pytestmark = pytest.mark.gpu

SHORT = 2_000_000   # SM cycles, about 1 ms: far above any wait of these small calls
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture
def hook():
    A.moe_test_set_wait(0, False)
    A.moe_get_device_error(clear=True)
    yield
    A.moe_test_set_wait(0, False)
    A.moe_get_device_error(clear=True)


def _call(op, counts, K, N):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    E, rows = len(counts), sum(counts)
    off = torch.tensor([0] + [sum(counts[: e + 1]) for e in range(E)], dtype=torch.int32, device="cuda")
    x, w, dy = (torch.randn(s, generator=g, device="cuda").to(BF) for s in ((rows, K), (E, N, K), (rows, N)))
    out = torch.zeros({"fwd": (rows, N), "dx": (rows, K), "dw": (E, N, K), "fp8": (rows, N)}[op], dtype=F32, device="cuda")
    xq, wq = x.to(F8), w.to(F8)
    xs, ws = torch.rand((K + 127) // 128, rows, device="cuda"), torch.rand(E, (N + 127) // 128, (K + 127) // 128, device="cuda")

    def run():
        out.zero_()
        if op == "fwd":
            A.moe_grouped_gemm(x, w, off, out)
        elif op == "dx":
            A.moe_grouped_gemm_dx(dy, w, off, out)
        elif op == "dw":
            A.moe_grouped_gemm_dw(dy, x, off, out)
        else:
            A.moe_grouped_gemm_fp8(xq, xs, wq, ws, off, out)
        torch.cuda.synchronize()
        return out.clone()

    return run


# few rows an expert and many: single CTAs and pairs, both FP8 forms
@pytest.mark.parametrize("counts", [[1, 3, 0, 2], [300, 17, 0, 90]], ids=["few", "many"])
@pytest.mark.parametrize("op", ["fwd", "dx", "dw", "fp8"])
def test_withheld_stage_times_out_and_the_next_call_is_exact(hook, op, counts):
    run = _call(op, counts, 1040, 520)
    ref = run()
    assert A.moe_get_device_error() == 0
    A.moe_test_set_wait(SHORT, False)      # a short limit alone changes nothing
    assert torch.equal(run(), ref)
    assert A.moe_get_device_error() == 0
    A.moe_test_set_wait(SHORT, True)
    t0 = time.perf_counter()
    run()
    dt = time.perf_counter() - t0
    assert A.moe_get_device_error(clear=True) == L.MOE_ERR_TIMEOUT
    assert A.moe_get_device_error() == 0
    assert dt < 1.0, dt
    A.moe_test_set_wait(0, False)
    assert torch.equal(run(), ref)
    assert A.moe_get_device_error() == 0
