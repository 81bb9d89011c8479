"""Python face of the C ABI: the same entry points, argument marshalling only.

Device buffers are torch CUDA tensors, host buffers numpy arrays or pinned
torch tensors, streams torch.cuda.Stream.  Each function raises MoeError on a
non-zero status.  Every computation happens inside libmoe.so.
"""
from __future__ import annotations

import ctypes as C

import numpy as np
import torch

from . import _lib as L
from ._lib import MoeError, check, ptr, stream_handle  # noqa: F401

DT_F32, DT_BF16 = L.DT_F32, L.DT_BF16
W_BF16, W_MXFP4, W_NVFP4 = L.W_BF16, L.W_MXFP4, L.W_NVFP4


def _dt(t) -> int:
    if t.dtype == torch.float32:
        return DT_F32
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return DT_BF16
    raise TypeError(f"activations must be float32 or bf16, got {t.dtype}")


def make_shape(layers, experts, hidden, ffn, top_k, wfmt) -> L.MoeShape:
    return L.shape(layers, experts, hidden, ffn, top_k, wfmt)


def shape_of(cfg) -> L.MoeShape:
    """Shape of a workloads.LayerConfig."""
    return make_shape(cfg.layers, cfg.experts, cfg.hidden, cfg.ffn, cfg.top_k, cfg.wfmt)


# ------------------------------------------------------------------ sizes
def moe_slot_bytes(shape) -> int:
    return L.lib.moe_slot_bytes(C.byref(shape))


def moe_cache_meta_bytes(shape, capacity, trace_capacity) -> int:
    return L.lib.moe_cache_meta_bytes(C.byref(shape), capacity, trace_capacity)


def moe_permute_workspace_bytes(n, experts, top_k) -> int:
    return L.lib.moe_permute_workspace_bytes(n, experts, top_k)


def moe_ffn_workspace_bytes(shape, rows) -> int:
    return L.lib.moe_ffn_workspace_bytes(C.byref(shape), rows)


def moe_layer_workspace_bytes(shape, n) -> int:
    return L.lib.moe_layer_workspace_bytes(C.byref(shape), n)


# ------------------------------------------------------------------ packing (host)
def moe_pack_expert(shape, ew, out: np.ndarray | None = None) -> np.ndarray:
    """Pack one workloads.ExpertWeights into a slot blob (uint8 numpy array or `out`)."""
    nb = moe_slot_bytes(shape)
    if out is None:
        out = np.empty(nb, np.uint8)
    w13 = np.ascontiguousarray(ew.w13)
    w2 = np.ascontiguousarray(ew.w2)
    s13 = None if ew.w13_scales is None else np.ascontiguousarray(ew.w13_scales, np.uint8)
    s2 = None if ew.w2_scales is None else np.ascontiguousarray(ew.w2_scales, np.uint8)
    ts = np.ascontiguousarray(ew.tensor_scales, np.float32)
    rc = L.lib.moe_pack_expert(C.byref(shape), ptr(w13), ptr(s13), ptr(w2), ptr(s2), ptr(ts), ptr(out))
    check("moe_pack_expert", rc)
    return out


# ------------------------------------------------------------------ steps
def moe_router_topk(x, wg, bias, n, hidden, experts, k, logits, topk_idx, topk_w, stream=None):
    rc = L.lib.moe_router_topk(ptr(x), _dt(x), ptr(wg), ptr(bias), n, hidden, experts, k, ptr(logits),
                               ptr(topk_idx), ptr(topk_w), stream_handle(stream))
    check("moe_router_topk", rc)


def moe_permute(topk_idx, n, experts, k, x, hidden, offsets, row_of, assign_of, x_perm, ws, stream=None):
    rc = L.lib.moe_permute(ptr(topk_idx), n, experts, k, ptr(x), _dt(x), hidden, ptr(offsets), ptr(row_of),
                           ptr(assign_of), ptr(x_perm), ptr(ws), ws.numel() * ws.element_size(),
                           stream_handle(stream))
    check("moe_permute", rc)


def moe_permute_noalloc(topk_idx, n, experts, k, x, hidden, offsets, row_of, assign_of, x_perm, stream=None):
    """moe_permute with the library's static scratch instead of a workspace (see include/moe.h)."""
    rc = L.lib.moe_permute_noalloc(ptr(topk_idx), n, experts, k, ptr(x), _dt(x), hidden, ptr(offsets), ptr(row_of),
                                   ptr(assign_of), ptr(x_perm), stream_handle(stream))
    check("moe_permute_noalloc", rc)


def moe_grouped_ffn(shape, pool, pool_slots, slot_of, offsets, x_perm, rows, y_perm, ws, stream=None):
    rc = L.lib.moe_grouped_ffn(C.byref(shape), ptr(pool), pool_slots, ptr(slot_of), ptr(offsets), ptr(x_perm), rows,
                               ptr(y_perm), ptr(ws), ws.numel() * ws.element_size(), stream_handle(stream))
    check("moe_grouped_ffn", rc)


def moe_act_terms(x, rows, K, wfmt, terms, codes, scales, row_exp, stream=None):
    """E2M1 term encoding of activation rows (the FP4 path's operand encoding):
    codes uint8 [rows, terms, K], scales uint8 [rows, terms, K/vs], row_exp int32 [rows]."""
    rc = L.lib.moe_act_terms(ptr(x), _dt(x), rows, K, wfmt, terms, ptr(codes), ptr(scales), ptr(row_exp),
                             stream_handle(stream))
    check("moe_act_terms", rc)


def moe_combine(y_perm, row_of, topk_w, n, k, hidden, out, stream=None):
    rc = L.lib.moe_combine(ptr(y_perm), ptr(row_of), ptr(topk_w), n, k, hidden, ptr(out), _dt(out),
                           stream_handle(stream))
    check("moe_combine", rc)


# ------------------------------------------------------------------ cache
class MoeCache:
    """A moe_cache plus the device buffers it lives in (allocated here by torch).

    host_blobs: list of L*E pinned uint8 tensors / numpy arrays (entries may
    repeat); the object keeps references so they outlive the cache.
    """

    def __init__(self, shape, capacity: int, host_blobs, trace_capacity: int = 1 << 16,
                 device="cuda", stream=None):
        self.shape = shape
        self.slot_bytes = moe_slot_bytes(shape)
        self.trace_capacity = trace_capacity
        mb = moe_cache_meta_bytes(shape, capacity, trace_capacity)
        if mb == 0 or self.slot_bytes == 0:
            raise MoeError("moe_cache_meta_bytes", L.MOE_ERR_INVALID_ARG)
        self.meta = torch.empty(mb, dtype=torch.uint8, device=device)
        self.pool = torch.empty(capacity * self.slot_bytes, dtype=torch.uint8, device=device)
        self._blobs = list(host_blobs)
        arr = (C.c_void_p * len(self._blobs))(*[ptr(b) for b in self._blobs])
        self._arr = arr
        h = C.c_void_p()
        rc = L.lib.moe_cache_create(C.byref(shape), ptr(self.meta), mb, ptr(self.pool), capacity,
                                    trace_capacity, arr, stream_handle(stream), C.byref(h))
        check("moe_cache_create", rc)
        self.handle = h

    @property
    def capacity(self) -> int:
        return L.lib.moe_cache_capacity(self.handle)

    def lookup_update(self, layer, idx, slot_of=None, stream=None, copy_stream=None):
        rc = L.lib.moe_cache_lookup_update(self.handle, layer, ptr(idx), idx.numel(), ptr(slot_of),
                                           stream_handle(stream), stream_handle(copy_stream))
        check("moe_cache_lookup_update", rc)

    def resize(self, new_capacity: int, stream=None, in_place: bool = False):
        mb = moe_cache_meta_bytes(self.shape, new_capacity, self.trace_capacity)
        if in_place and new_capacity <= self.capacity and mb <= self.meta.numel():
            meta, pool = self.meta, self.pool
        else:
            meta = torch.empty(mb, dtype=torch.uint8, device=self.meta.device)
            pool = torch.empty(new_capacity * self.slot_bytes, dtype=torch.uint8, device=self.pool.device)
        rc = L.lib.moe_cache_resize(self.handle, ptr(meta), meta.numel(), ptr(pool), new_capacity,
                                    stream_handle(stream))
        check("moe_cache_resize", rc)
        self.meta, self.pool = meta, pool

    def set_fill_mode(self, mode: int, stream=None):
        """L.FILL_HOST (host-issued DMA copies) or L.FILL_DEVICE (zero-copy fill kernel)."""
        check("moe_cache_set_fill_mode", L.lib.moe_cache_set_fill_mode(self.handle, mode, stream_handle(stream)))

    @property
    def fill_mode(self) -> int:
        return L.lib.moe_cache_fill_mode(self.handle)

    def device_status(self, clear: bool = False) -> int:
        """First error a lookup kernel recorded since the last clear (0 if none)."""
        rc = L.lib.moe_cache_device_status(self.handle, 1 if clear else 0)
        if rc in (L.MOE_ERR_CUDA,):
            raise MoeError("moe_cache_device_status", rc)
        return rc

    def read_trace(self, cap: int | None = None) -> np.ndarray:
        cap = self.trace_capacity if cap is None else cap
        buf = np.zeros(cap, L.TRACE_DTYPE)
        n = C.c_size_t(0)
        check("moe_cache_read_trace", L.lib.moe_cache_read_trace(self.handle, ptr(buf), cap, C.byref(n)))
        return buf[: n.value].copy()

    def stats(self) -> dict:
        s = L.MoeStats()
        check("moe_cache_get_stats", L.lib.moe_cache_get_stats(self.handle, C.byref(s)))
        return {name: getattr(s, name) for name, _ in L.MoeStats._fields_}

    def snapshot(self):
        nk = self.shape.layers * self.shape.experts
        c = self.capacity
        slot_of = np.empty(nk, np.int32)
        key_of = np.empty(c, np.int32)
        stamp = np.empty(c, np.uint64)
        check("moe_cache_snapshot", L.lib.moe_cache_snapshot(self.handle, ptr(slot_of), ptr(key_of), ptr(stamp)))
        return slot_of, key_of, stamp

    def close(self):
        if getattr(self, "handle", None):
            L.lib.moe_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_layer_forward(cache: MoeCache, layer, x, wg, bias, out, ws, stream=None, copy_stream=None,
                      topk_idx_out=None, topk_w_out=None):
    n = x.shape[0]
    rc = L.lib.moe_layer_forward(cache.handle, layer, ptr(x), _dt(x), ptr(wg), ptr(bias), n, ptr(out), ptr(ws),
                                 ws.numel() * ws.element_size(), stream_handle(stream),
                                 stream_handle(copy_stream), ptr(topk_idx_out), ptr(topk_w_out))
    check("moe_layer_forward", rc)


def moe_prefill_workspace_bytes(shape, n) -> int:
    return L.lib.moe_prefill_workspace_bytes(C.byref(shape), n)


def moe_prefill_forward(cache: MoeCache, layer0, xs, wgs, biases, outs, ws, stream=None, copy_stream=None,
                        topk_idx_out=None):
    """Layers layer0 .. layer0+len(xs)-1 over one prompt; xs / wgs / biases / outs are per-layer
    device tensors (biases may be None or hold None; outs[i] may be xs[i+1])."""
    nl = len(xs)
    if not (len(wgs) == len(outs) == nl) or (biases is not None and len(biases) != nl):
        raise ValueError("per-layer lists of different lengths")
    n = xs[0].shape[0] if nl else 0
    arr = lambda ts: (C.c_void_p * max(1, nl))(*[ptr(t) for t in ts])
    xa, wa, oa = arr(xs), arr(wgs), arr(outs)
    ba = None if biases is None else arr(biases)
    rc = L.lib.moe_prefill_forward(cache.handle, layer0, nl, xa, _dt(xs[0]) if nl else 0, wa, ba, n, oa, ptr(ws),
                                   ws.numel() * ws.element_size(), stream_handle(stream), stream_handle(copy_stream),
                                   ptr(topk_idx_out))
    check("moe_prefill_forward", rc)


# ------------------------------------------------------------------ expert matrix products
# These calls are short next to a Python call per check, so a call unpacks the
# shapes and strides and compares; _refuse works out which argument failed.
_BF16, _F32, _I32, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
_OUT = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}
_NOT_AS_REQUIRED = (AttributeError, TypeError, ValueError)   # of unpacking what is no tensor, or of other dimensions


def _refuse(fn, **specs):
    """Raises the error of the first argument that is not as required: name = (tensor, dtypes, shape,
    packed), None in a shape for any extent."""
    for name, (t, dtypes, shape, packed) in specs.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{fn}: {name} must be a torch tensor, got {type(t).__name__}")
        if t.dtype not in dtypes:
            raise TypeError(f"{fn}: {name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
        if t.dim() != len(shape) or any(w is not None and w != g for w, g in zip(shape, t.shape)):
            want = "[" + ", ".join("*" if w is None else str(w) for w in shape) + "]"
            raise ValueError(f"{fn}: {name} must have shape {want}, got {list(t.shape)}")
        if packed and not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must be contiguous")
        if not packed and not _ld(t.stride(), *t.shape):
            raise ValueError(f"{fn}: {name} must have adjacent columns and rows that do not overlap, got strides {t.stride()}")
    for name, (t, *_) in specs.items():
        if t.get_device() != _device():
            raise ValueError(f"{fn}: {name} is on {t.device}, not on the current CUDA device")
    raise ValueError(f"{fn}: arguments do not fit together")


def _dims(t, n):
    """t's shape if it is a tensor of n dimensions, else n Nones."""
    return tuple(t.shape) if isinstance(t, torch.Tensor) and t.dim() == n else (None,) * n


def _ld(strides, rows, cols) -> int:
    """Leading dimension of a row matrix whose columns are adjacent, 0 of any other (one row has no
    next: its stride does not count)."""
    a, b = strides
    if b != 1:
        return 0
    return cols if rows <= 1 else a if a >= cols else 0


def _device() -> int:
    """The current CUDA device, where the calls launch; -2 (no tensor's) without one."""
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -2


def moe_grouped_gemm(x, w, offsets, y, stream=None):
    """y[r] = W_e x[r] for the rows [offsets[e], offsets[e+1]) of every expert e.

    x [rows, in] bf16, w [experts, out, in] bf16, offsets int32 [experts + 1], y [rows, out]
    float32 or bf16; x and y may be column slices of wider matrices."""
    try:
        (E, N, K), (rows, kx), (ne,), (ry, ny) = w.shape, x.shape, offsets.shape, y.shape
        ldx, ldy = _ld(x.stride(), rows, K), _ld(y.stride(), rows, N)
        good = (ldx and ldy and kx == K and ne == E + 1 and ry == rows and ny == N
                and x.dtype is _BF16 and w.dtype is _BF16 and offsets.dtype is _I32 and y.dtype in _OUT
                and w.is_contiguous() and offsets.is_contiguous()
                and x.get_device() == w.get_device() == offsets.get_device() == y.get_device() == _device())
    except _NOT_AS_REQUIRED:
        good = False
    if not good:
        (E, N, K), (rows, _) = _dims(w, 3), _dims(x, 2)
        _refuse("moe_grouped_gemm", w=(w, (_BF16,), (None, None, None), True), x=(x, (_BF16,), (None, K), False),
                offsets=(offsets, (_I32,), (E and E + 1,), True), y=(y, _OUT, (rows, N), False))
    rc = L.lib.moe_grouped_gemm(E, K, N, x.data_ptr(), ldx, w.data_ptr(), offsets.data_ptr(), rows, y.data_ptr(), ldy,
                                _OUT[y.dtype], stream_handle(stream))
    check("moe_grouped_gemm", rc)


def moe_grouped_gemm_dx(dy, w, offsets, dx, stream=None):
    """Gradient of moe_grouped_gemm with respect to x: dx[r] = W_e^T dy[r].

    dy [rows, out] bf16, w [experts, out, in] bf16, dx [rows, in] float32 or bf16."""
    try:
        (E, N, K), (rows, ny), (ne,), (rx, kx) = w.shape, dy.shape, offsets.shape, dx.shape
        lddy, lddx = _ld(dy.stride(), rows, N), _ld(dx.stride(), rows, K)
        good = (lddy and lddx and ny == N and ne == E + 1 and rx == rows and kx == K
                and dy.dtype is _BF16 and w.dtype is _BF16 and offsets.dtype is _I32 and dx.dtype in _OUT
                and w.is_contiguous() and offsets.is_contiguous()
                and dy.get_device() == w.get_device() == offsets.get_device() == dx.get_device() == _device())
    except _NOT_AS_REQUIRED:
        good = False
    if not good:
        (E, N, K), (rows, _) = _dims(w, 3), _dims(dy, 2)
        _refuse("moe_grouped_gemm_dx", w=(w, (_BF16,), (None, None, None), True), dy=(dy, (_BF16,), (None, N), False),
                offsets=(offsets, (_I32,), (E and E + 1,), True), dx=(dx, _OUT, (rows, K), False))
    rc = L.lib.moe_grouped_gemm_dx(E, K, N, dy.data_ptr(), lddy, w.data_ptr(), offsets.data_ptr(), rows, dx.data_ptr(),
                                   lddx, _OUT[dx.dtype], stream_handle(stream))
    check("moe_grouped_gemm_dx", rc)


def moe_grouped_gemm_dw(dy, x, offsets, dw, accumulate=False, stream=None):
    """Gradient of moe_grouped_gemm with respect to w: dW_e = sum of dy[r] x[r]^T over e's rows.

    dy [rows, out] bf16, x [rows, in] bf16, dw [experts, out, in] float32 or bf16; accumulate
    adds to what dw holds instead of storing."""
    try:
        (E, N, K), (rows, ny), (rx, kx), (ne,) = dw.shape, dy.shape, x.shape, offsets.shape
        lddy, ldx = _ld(dy.stride(), rows, N), _ld(x.stride(), rows, K)
        good = (lddy and ldx and ny == N and rx == rows and kx == K and ne == E + 1
                and dy.dtype is _BF16 and x.dtype is _BF16 and offsets.dtype is _I32 and dw.dtype in _OUT
                and dw.is_contiguous() and offsets.is_contiguous()
                and dy.get_device() == x.get_device() == offsets.get_device() == dw.get_device() == _device())
    except _NOT_AS_REQUIRED:
        good = False
    if not good:
        (E, N, K), (rows, _) = _dims(dw, 3), _dims(dy, 2)
        _refuse("moe_grouped_gemm_dw", dw=(dw, _OUT, (None, None, None), True), dy=(dy, (_BF16,), (None, N), False),
                x=(x, (_BF16,), (rows, K), False), offsets=(offsets, (_I32,), (E and E + 1,), True))
    rc = L.lib.moe_grouped_gemm_dw(E, K, N, dy.data_ptr(), lddy, x.data_ptr(), ldx, offsets.data_ptr(), rows,
                                   dw.data_ptr(), _OUT[dw.dtype], 1 if accumulate else 0, stream_handle(stream))
    check("moe_grouped_gemm_dw", rc)


def moe_grouped_gemm_fp8(xq, xs, wq, ws, offsets, y, stream=None):
    """moe_grouped_gemm of e4m3 codes: xq [rows, in] with scales xs [ceil(in/128), rows], wq
    [experts, out, in] with scales ws [experts, ceil(out/128), ceil(in/128)] (float32)."""
    try:
        (E, N, K), (rows, kx), (ne,), (ry, ny) = wq.shape, xq.shape, offsets.shape, y.shape
        nb, kb = (N + 127) // 128, (K + 127) // 128
        ldxq, ldy = _ld(xq.stride(), rows, K), _ld(y.stride(), rows, N)
        good = (ldxq and ldy and kx == K and ne == E + 1 and ry == rows and ny == N
                and xs.shape == (kb, rows) and ws.shape == (E, nb, kb)
                and xq.dtype is _E4M3 and wq.dtype is _E4M3 and xs.dtype is _F32 and ws.dtype is _F32
                and offsets.dtype is _I32 and y.dtype in _OUT
                and xs.is_contiguous() and wq.is_contiguous() and ws.is_contiguous() and offsets.is_contiguous()
                and xq.get_device() == xs.get_device() == wq.get_device() == ws.get_device() == offsets.get_device()
                == y.get_device() == _device())
    except _NOT_AS_REQUIRED:
        good = False
    if not good:
        (E, N, K), (rows, _) = _dims(wq, 3), _dims(xq, 2)
        nb, kb = (None, None) if E is None else ((N + 127) // 128, (K + 127) // 128)
        _refuse("moe_grouped_gemm_fp8", wq=(wq, (_E4M3,), (None, None, None), True), xq=(xq, (_E4M3,), (None, K), False),
                xs=(xs, (_F32,), (kb, rows), True), ws=(ws, (_F32,), (E, nb, kb), True),
                offsets=(offsets, (_I32,), (E and E + 1,), True), y=(y, _OUT, (rows, N), False))
    rc = L.lib.moe_grouped_gemm_fp8(E, K, N, xq.data_ptr(), ldxq, xs.data_ptr(), wq.data_ptr(), ws.data_ptr(),
                                    offsets.data_ptr(), rows, y.data_ptr(), ldy, _OUT[y.dtype], stream_handle(stream))
    check("moe_grouped_gemm_fp8", rc)


def moe_fp8_quantize_act(x, q, s, swiglu=False, stream=None):
    """e4m3 codes q [rows, cols] and scales s [ceil(cols/128), rows] of x [rows, cols] (float32 or
    bf16), or with swiglu of silu(gate) * up of x [rows, 2 cols] = gate | up."""
    try:
        (rows, cols), (rx, width) = q.shape, x.shape
        ldx, ldq = _ld(x.stride(), rows, width), _ld(q.stride(), rows, cols)
        good = (ldx and ldq and rx == rows and width == (2 * cols if swiglu else cols)
                and s.shape == ((cols + 127) // 128, rows)
                and q.dtype is _E4M3 and x.dtype in _OUT and s.dtype is _F32 and s.is_contiguous()
                and x.get_device() == q.get_device() == s.get_device() == _device())
    except _NOT_AS_REQUIRED:
        good = False
    if not good:
        rows, cols = _dims(q, 2)
        width, kb = (None, None) if cols is None else (2 * cols if swiglu else cols, (cols + 127) // 128)
        _refuse("moe_fp8_quantize_act", q=(q, (_E4M3,), (None, None), False), x=(x, _OUT, (rows, width), False),
                s=(s, (_F32,), (kb, rows), True))
    rc = L.lib.moe_fp8_quantize_act(x.data_ptr(), _OUT[x.dtype], ldx, rows, cols, 1 if swiglu else 0, q.data_ptr(), ldq,
                                    s.data_ptr(), stream_handle(stream))
    check("moe_fp8_quantize_act", rc)


def moe_fp8_quantize_weight(w, q, s, stream=None):
    """e4m3 codes q and 128 x 128 block scales s [experts, ceil(out/128), ceil(in/128)] of w
    [experts, out, in] (float32 or bf16)."""
    try:
        E, N, K = w.shape
        good = (q.shape == (E, N, K) and s.shape == (E, (N + 127) // 128, (K + 127) // 128)
                and w.dtype in _OUT and q.dtype is _E4M3 and s.dtype is _F32
                and w.is_contiguous() and q.is_contiguous() and s.is_contiguous()
                and w.get_device() == q.get_device() == s.get_device() == _device())
    except _NOT_AS_REQUIRED:
        good = False
    if not good:
        E, N, K = _dims(w, 3)
        nb, kb = (None, None) if E is None else ((N + 127) // 128, (K + 127) // 128)
        _refuse("moe_fp8_quantize_weight", w=(w, _OUT, (None, None, None), True), q=(q, (_E4M3,), (E, N, K), True),
                s=(s, (_F32,), (E, nb, kb), True))
    rc = L.lib.moe_fp8_quantize_weight(w.data_ptr(), _OUT[w.dtype], E, N, K, q.data_ptr(), s.data_ptr(),
                                       stream_handle(stream))
    check("moe_fp8_quantize_weight", rc)


# ------------------------------------------------------------------ testing hooks
def moe_test_set_wait(cycles: int, withhold: bool = False) -> None:
    """Bounded-wait limit (SM cycles, 0 = default) and stage withholding of later launches of the grouped
    FFN and of the expert products."""
    check("moe_test_set_wait", L.lib.moe_test_set_wait(int(cycles), 1 if withhold else 0))


def moe_get_device_error(clear: bool = False) -> int:
    rc = L.lib.moe_get_device_error(1 if clear else 0)
    if rc == L.MOE_ERR_CUDA:
        raise MoeError("moe_get_device_error", rc)
    return rc


# ------------------------------------------------------------------ profiling
def moe_profile_enable(timing: bool) -> None:
    check("moe_profile_enable", L.lib.moe_profile_enable(1 if timing else 0))


def moe_profile_read(reset: bool = False) -> dict:
    """{kind: {"launches", "timed", "ms"}} for router/lookup/permute/ffn/combine/fill/gemm/quant."""
    arr = (L.MoeProf * len(L.PROF_KINDS))()
    check("moe_profile_read", L.lib.moe_profile_read(arr, len(L.PROF_KINDS), 1 if reset else 0))
    return {k: {"launches": arr[i].launches, "timed": arr[i].timed, "ms": arr[i].ms}
            for i, k in enumerate(L.PROF_KINDS)}
