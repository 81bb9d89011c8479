"""Expert matrix products and FP8 quantisation on the host (CPU only): what the
C entry points and the Python binding refuse, before any device work."""
import ctypes as C

import pytest
import torch

from expert_cached_sparse_b200 import _lib as L
from expert_cached_sparse_b200 import api as A

P = C.c_void_p(0x100000)      # aligned dummy address, never read
ODD = C.c_void_p(0x100004)
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def fwd(E=4, i=64, o=64, x=P, ldx=64, w=P, off=P, rows=8, y=P, ldy=64, dt=L.DT_BF16):
    return L.lib.moe_grouped_gemm(E, i, o, x, ldx, w, off, rows, y, ldy, dt, None)


def dx(E=4, i=64, o=64, dy=P, lddy=64, w=P, off=P, rows=8, out=P, ldo=64, dt=L.DT_BF16):
    return L.lib.moe_grouped_gemm_dx(E, i, o, dy, lddy, w, off, rows, out, ldo, dt, None)


def dw(E=4, i=64, o=64, dy=P, lddy=64, x=P, ldx=64, off=P, rows=8, out=P, dt=L.DT_BF16, acc=0):
    return L.lib.moe_grouped_gemm_dw(E, i, o, dy, lddy, x, ldx, off, rows, out, dt, acc, None)


def fp8(E=4, i=64, o=64, xq=P, ldx=64, xs=P, wq=P, ws=P, off=P, rows=8, y=P, ldy=64, dt=L.DT_BF16):
    return L.lib.moe_grouped_gemm_fp8(E, i, o, xq, ldx, xs, wq, ws, off, rows, y, ldy, dt, None)


def act(x=P, dt=L.DT_BF16, ldx=64, rows=8, cols=64, swiglu=0, q=P, ldq=64, s=P):
    return L.lib.moe_fp8_quantize_act(x, dt, ldx, rows, cols, swiglu, q, ldq, s, None)


def weight(w=P, dt=L.DT_BF16, E=4, o=64, i=64, q=P, s=P):
    return L.lib.moe_fp8_quantize_weight(w, dt, E, o, i, q, s, None)


INVALID = [
    *[(f, k) for f in (fwd, dx, dw, fp8) for k in (
        {"E": 0}, {"E": -1}, {"i": 0}, {"i": 60}, {"o": 0}, {"o": 12}, {"rows": -1}, {"off": None}, {"dt": 7})],
    (fwd, {"x": None}), (fwd, {"w": None}), (fwd, {"y": None}), (fwd, {"x": ODD}), (fwd, {"w": ODD}), (fwd, {"y": ODD}),
    (fwd, {"ldx": 56}), (fwd, {"ldx": 68}), (fwd, {"ldy": 56}), (fwd, {"ldy": 68}), (fwd, {"ldx": -64}),
    (dx, {"dy": None}), (dx, {"w": ODD}), (dx, {"out": ODD}), (dx, {"lddy": 60}), (dx, {"ldo": 32}),
    (dw, {"dy": None}), (dw, {"x": None}), (dw, {"out": None}), (dw, {"out": ODD}), (dw, {"ldx": 60}), (dw, {"lddy": 8}),
    (fp8, {"i": 72}), (fp8, {"xq": ODD}), (fp8, {"wq": ODD}), (fp8, {"ldx": 72}), (fp8, {"xs": None}), (fp8, {"ws": None}),
    (fp8, {"xs": C.c_void_p(0x100002)}), (fp8, {"ldy": 60}), (fp8, {"y": None}),
    (act, {"cols": 0}), (act, {"cols": 60}), (act, {"rows": -1}), (act, {"dt": 5}), (act, {"ldx": 60}), (act, {"ldx": 68}),
    (act, {"swiglu": 1}), (act, {"ldq": 60}), (act, {"x": None}), (act, {"x": ODD}), (act, {"q": ODD}), (act, {"s": None}),
    (weight, {"E": 0}), (weight, {"o": 0}), (weight, {"i": 60}), (weight, {"dt": 3}), (weight, {"w": None}),
    (weight, {"w": ODD}), (weight, {"q": ODD}), (weight, {"s": None}),
]
UNSUPPORTED = [
    *[(f, k) for f in (fwd, dx, dw, fp8) for k in (
        {"E": 4097}, {"i": (1 << 20) + 16}, {"o": (1 << 20) + 8}, {"rows": (1 << 30) + 1})],
    (act, {"cols": (1 << 20) + 8, "ldx": 1 << 21, "ldq": 1 << 21}), (act, {"rows": (1 << 30) + 1}),
    (weight, {"E": 4097}), (weight, {"o": (1 << 20) + 1}), (weight, {"i": (1 << 20) + 8}),
]


@pytest.mark.parametrize("f,kw", INVALID, ids=[f"{f.__name__}-{k}" for f, k in INVALID])
def test_invalid_arguments(f, kw):
    assert f(**kw) == L.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("f,kw", UNSUPPORTED, ids=[f"{f.__name__}-{k}" for f, k in UNSUPPORTED])
def test_sizes_above_the_limits(f, kw):
    assert f(**kw) == L.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("f", [fwd, dx, fp8, act])
def test_no_rows_is_no_work(f):
    assert f(rows=0) == L.MOE_OK
    assert (f(rows=0, x=None) if f is act else f(rows=0, off=None)) == L.MOE_OK


def _z(dt, *shape):
    return torch.zeros(*shape, dtype=dt)


def test_binding_checks_types_shapes_and_strides():
    off = _z(torch.int32, 5)
    x, w, y = _z(BF, 8, 64), _z(BF, 4, 72, 64), _z(F32, 8, 72)
    bad = [
        (TypeError, (_z(F32, 8, 64), w, off, y)), (TypeError, (x, _z(torch.float16, 4, 72, 64), off, y)),
        (TypeError, (x, w, off.long(), y)), (TypeError, (x, w, off, _z(torch.float16, 8, 72))), (TypeError, (1, w, off, y)),
        (ValueError, (_z(BF, 8, 72), w, off, y)), (ValueError, (x, w, off[:4], y)), (ValueError, (x, w, off, y[:7])),
        (ValueError, (x, w[0], off, y)), (ValueError, (_z(BF, 64, 8).t(), w, off, y)),
        (ValueError, (x, w.transpose(1, 2).contiguous().transpose(1, 2), off, y)),
        (ValueError, (_z(BF, 1, 64).expand(8, 64), w, off, y)),
        (ValueError, (x, w, off, y)),   # everything right but not on the GPU
    ]
    for exc, args in bad:
        with pytest.raises(exc):
            A.moe_grouped_gemm(*args)
    for exc, args in [(TypeError, (_z(F32, 8, 72), w, off, _z(BF, 8, 64))), (ValueError, (_z(BF, 8, 64), w, off, _z(BF, 8, 64))),
                      (ValueError, (_z(BF, 8, 72), w, off, _z(BF, 8, 72))), (ValueError, (_z(BF, 8, 72), w, off, _z(BF, 8, 64)))]:
        with pytest.raises(exc):
            A.moe_grouped_gemm_dx(*args)
    for exc, args in [(TypeError, (_z(BF, 8, 72), x, off, _z(torch.float16, 4, 72, 64))),
                      (ValueError, (_z(BF, 9, 72), x, off, _z(F32, 4, 72, 64))),
                      (ValueError, (_z(BF, 8, 72), x, off, _z(F32, 4, 64, 72).transpose(1, 2))),
                      (ValueError, (_z(BF, 8, 72), x, off, _z(F32, 4, 72, 64)))]:
        with pytest.raises(exc):
            A.moe_grouped_gemm_dw(*args)


def test_fp8_binding_checks_types_shapes_and_strides():
    off = _z(torch.int32, 5)
    xq, xs, wq, ws, y = _z(F8, 8, 144), _z(F32, 2, 8), _z(F8, 4, 136, 144), _z(F32, 4, 2, 2), _z(BF, 8, 136)
    bad = [
        (TypeError, (xq.view(torch.uint8), xs, wq, ws, off, y)), (TypeError, (xq, xs.double(), wq, ws, off, y)),
        (ValueError, (xq, xs.t(), wq, ws, off, y)), (ValueError, (xq, _z(F32, 8, 2).t(), wq, ws, off, y)),
        (ValueError, (xq, xs, wq, ws[:, :1], off, y)), (ValueError, (xq, xs, wq, ws, off, y.t())),
        (ValueError, (xq, xs, wq, ws, off, y)),
    ]
    for exc, args in bad:
        with pytest.raises(exc):
            A.moe_grouped_gemm_fp8(*args)
    q, s = _z(F8, 8, 144), _z(F32, 2, 8)
    for exc, args, kw in [(TypeError, (_z(torch.float16, 8, 144), q, s), {}), (ValueError, (_z(BF, 8, 144), q, s), {"swiglu": True}),
                          (ValueError, (_z(BF, 8, 288), q, s), {}), (ValueError, (_z(BF, 8, 144), q, s.t()), {}),
                          (ValueError, (_z(BF, 8, 144), q, s), {})]:
        with pytest.raises(exc):
            A.moe_fp8_quantize_act(*args, **kw)
    w, q, s = _z(F32, 2, 130, 136), _z(F8, 2, 130, 136), _z(F32, 2, 2, 2)
    for exc, args in [(TypeError, (w, w, s)), (ValueError, (w, q[:1], s)), (ValueError, (w, q, s[:, :, :1])), (ValueError, (w, q, s))]:
        with pytest.raises(exc):
            A.moe_fp8_quantize_weight(*args)
