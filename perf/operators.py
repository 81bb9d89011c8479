"""What the expert matrix products are measured on.

The operators:
  fwd     grouped product: rows of expert e times W_e^T             (moe_grouped_gemm)
  bwd     its gradients with respect to rows and weights            (moe_grouped_gemm_dx, moe_grouped_gemm_dw)
  fp8     grouped product of e4m3 codes with a scale per 1 x 128 block of the rows and per 128 x 128
          block of the weights                                      (moe_grouped_gemm_fp8)
  act     e4m3 codes and 1 x 128 scales of rows, or of silu(gate) * up of gate|up rows
                                                                    (moe_fp8_quantize_act)
  weight  e4m3 codes and 128 x 128 scales of expert weights         (moe_fp8_quantize_weight)

`own` false: the plain form in elementary torch operations.  `own` true: the library's entry points.
"""
import math

import torch

own = False

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
E4M3_MAX = 448.0
TINY_BLOCK = 2.0 ** -100   # blocks with no larger magnitude get scale 1 and zero codes


def _c(name, op, experts, top_k, tokens, d_in, d_out, zipf, **kw):
    c = {"name": name, "op": op, "experts": experts, "top_k": top_k, "tokens": tokens, "in": d_in, "out": d_out,
         "zipf": zipf, "f32": False, "swiglu": False}
    c.update(kw)
    return c


def listed():
    return [
        # one token through the gate|up product of the 128-expert, hidden 2048, ffn 768 layer: decode latency
        _c("fwd 1 token", "fwd", 128, 8, 1, 2048, 2 * 768, 0.0),
        # a decode batch of the 256-expert layer (hidden 4096, ffn 2048), Zipf routing: weights streamed once
        _c("fwd decode batch 16", "fwd", 256, 6, 16, 4096, 4096, 1.1),
        # its prompt: 4096 tokens, skewed expert sizes
        _c("fwd prompt 4096", "fwd", 256, 6, 4096, 4096, 4096, 0.8),
        # the 8-expert layer's 64 tokens with sizes off every tile, float32 gradients
        _c("bwd small odd", "bwd", 8, 2, 61, 264, 1000, 0.5, f32=True),
        # fine-tuning the 128-expert layer: gradients of the down product on 512 tokens
        _c("bwd 512 tokens", "bwd", 128, 8, 512, 768, 2048, 0.0),
        # a full training batch's gate|up gradients
        _c("bwd 4096 tokens", "bwd", 128, 8, 4096, 2048, 2 * 768, 0.3),
        # the decode batch with fp8 weights
        _c("fp8 decode batch 16", "fp8", 256, 6, 16, 4096, 4096, 1.1),
        # the prompt with fp8 weights
        _c("fp8 prompt 4096", "fp8", 256, 6, 4096, 4096, 4096, 0.8),
        # one dense matrix (a shared expert), ragged row count, inner size off the 128 block
        _c("fp8 dense 2000", "fp8", 1, 1, 2000, 2000, 4096, 0.0),
        # activations of a decode batch before the gate|up product
        _c("act decode batch 16", "act", 1, 6, 16, 4096, 0, 0.0),
        # the prompt's silu(gate) * up before the down product
        _c("act swiglu prompt 4096", "act", 1, 6, 4096, 2048, 0, 0.0, swiglu=True),
        # the gate|up matrices of 64 experts (one cache of slots) written as fp8 once
        _c("weight 64 experts", "weight", 64, 1, 1, 4096, 4096, 0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "fp8", "fp8", "act", "weight"])
    step = 16 if op == "fp8" else 8
    while True:
        experts = _log(rng, 1, 256)
        top_k = rng.randint(1, min(8, experts))
        tokens = _log(rng, 1, 4096)
        d_in = step * _log(rng, 64 // step, 4096 // step)
        d_out = 8 * _log(rng, 8, 512)
        if op == "weight":
            tokens = top_k = 1
        if op == "act":
            experts, d_out = 1, 0
        if rng.random() < 0.5:   # half of the cases: sizes of whole tiles, as models have them
            d_in, d_out = -(-d_in // 256) * 256, -(-d_out // 256) * 256
        e_elems, flops = experts * d_in * d_out, tokens * top_k * d_in * d_out
        if op == "bwd" and (e_elems > 128 * 2048 * 1536 or flops > 32768 * 2048 * 1536):
            continue
        if op == "weight" and e_elems > 64 * 4096 * 4096:
            continue
        if e_elems <= 256 * 4096 * 4096 and flops <= 24576 * 4096 * 4096:
            break
    return {"op": op, "experts": experts, "top_k": top_k, "tokens": tokens, "in": d_in, "out": d_out,
            "zipf": round(rng.uniform(0.0, 1.1), 2), "f32": rng.random() < 0.3,
            "swiglu": op == "act" and rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(0x5EED + int(seed))
    return g


def _offsets(case, g):
    """Row ranges of the experts after routing `tokens` tokens to top_k distinct experts with Zipf popularity."""
    E, k, n = case["experts"], case["top_k"], case["tokens"]
    rank = torch.randperm(E, generator=g, device="cuda").float()
    u = torch.rand(n, E, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    score = -case["zipf"] * torch.log(rank + 1) - torch.log(-torch.log(u))
    counts = torch.bincount(score.topk(k, dim=1).indices.flatten(), minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = counts.cumsum(0)
    return off, int(counts.max())


def _normal(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=BF16).mul_(scale)


def _fp8_rows(x):
    """Codes [rows][K] and scales [K / 128 rounded up][rows]."""
    r, K = x.shape
    kb = -(-K // 128)
    v = torch.nn.functional.pad(x.float(), (0, kb * 128 - K)).view(r, kb, 128)
    amax = v.abs().amax(2)
    s = torch.where(amax >= TINY_BLOCK, amax / E4M3_MAX, torch.ones_like(amax))
    q = (v / s[:, :, None]).view(r, kb * 128)[:, :K].to(F8)
    return q, s.t().contiguous()


def _fp8_blocks(w):
    """Codes [E][N][K] and scales [E][N / 128][K / 128] (rounded up)."""
    E, N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    v = torch.nn.functional.pad(w.float(), (0, kb * 128 - K, 0, nb * 128 - N)).view(E, nb, 128, kb, 128)
    amax = v.abs().amax((2, 4))
    s = torch.where(amax >= TINY_BLOCK, amax / E4M3_MAX, torch.ones_like(amax))
    q = (v / s[:, :, None, :, None]).view(E, nb * 128, kb * 128)[:, :N, :K].to(F8)
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    E, K, N = case["experts"], case["in"], case["out"]
    rows = case["tokens"] * case["top_k"]
    y_dtype = F32 if case["f32"] else BF16
    st = {"case": case}
    if case["op"] == "act":
        st["x"] = _normal((rows, 2 * K if case["swiglu"] else K), g)
        st["q"] = torch.empty(rows, K, dtype=F8, device="cuda")
        st["s"] = torch.empty(-(-K // 128), rows, dtype=F32, device="cuda")
        return st
    if case["op"] == "weight":
        st["w"] = _normal((E, N, K), g, 0.02)
        st["q"] = torch.empty(E, N, K, dtype=F8, device="cuda")
        st["s"] = torch.empty(E, -(-N // 128), -(-K // 128), dtype=F32, device="cuda")
        return st
    st["offsets"], st["cap"] = _offsets(case, g)
    x = _normal((rows, K), g)
    if case["op"] == "fp8":
        st["xq"], st["xs"] = _fp8_rows(x)
        st["wq"] = torch.empty(E, N, K, dtype=F8, device="cuda")
        st["ws"] = torch.empty(E, -(-N // 128), -(-K // 128), dtype=F32, device="cuda")
        step = max(1, (64 << 20) // (N * K))
        for e in range(0, E, step):
            st["wq"][e:e + step], st["ws"][e:e + step] = _fp8_blocks(_normal((min(step, E - e), N, K), g, 0.02))
        st["y"] = torch.zeros(rows, N, dtype=y_dtype, device="cuda")
        return st
    st["x"], st["w"] = x, _normal((E, N, K), g, 0.02)
    if case["op"] == "fwd":
        st["y"] = torch.zeros(rows, N, dtype=y_dtype, device="cuda")
    else:
        st["dy"] = _normal((rows, N), g)
        st["dx"] = torch.zeros(rows, K, dtype=y_dtype, device="cuda")
        st["dw"] = torch.empty(E, N, K, dtype=y_dtype, device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def _place(offsets, rows):
    """Expert of each row and the row's place among its expert's rows."""
    r = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets[1:].long(), r, right=True)
    return e, r - offsets.long()[e]


def _padded(x, e, pos, E, cap):
    b = torch.zeros(E, cap, x.shape[1], dtype=F32, device=x.device)
    b[e, pos] = x.float()
    return b


def _spread(s, N, K):
    """128 x 128 block scales over an [N][K] matrix."""
    n, k = torch.arange(N, device=s.device) // 128, torch.arange(K, device=s.device) // 128
    return s[:, n][:, :, k]


def _plain(st):
    case = st["case"]
    E, K, N = case["experts"], case["in"], case["out"]
    rows = case["tokens"] * case["top_k"]
    if case["op"] == "act":
        x = st["x"].float()
        if case["swiglu"]:
            gate, up = x[:, :K], x[:, K:]
            x = gate / (1.0 + torch.exp(-gate)) * up
        return _fp8_rows(x)
    if case["op"] == "weight":
        return _fp8_blocks(st["w"])
    e, pos = _place(st["offsets"], rows)
    cap = st["cap"]
    if case["op"] == "fwd":
        y = torch.bmm(_padded(st["x"], e, pos, E, cap), st["w"].float().transpose(1, 2))
        return y[e, pos].to(st["y"].dtype)
    if case["op"] == "fp8":
        k = torch.arange(K, device="cuda") // 128
        x = st["xq"].float() * st["xs"].t()[:, k]
        w = st["wq"].float().mul_(_spread(st["ws"], N, K))
        y = torch.bmm(_padded(x, e, pos, E, cap), w.transpose(1, 2))
        return y[e, pos].to(st["y"].dtype)
    dy = _padded(st["dy"], e, pos, E, cap)
    dx = torch.bmm(dy, st["w"].float())[e, pos].to(st["dx"].dtype)
    dw = torch.bmm(dy.transpose(1, 2), _padded(st["x"], e, pos, E, cap)).to(st["dw"].dtype)
    return dx, dw


def _own(st):
    from expert_cached_sparse_b200 import api as A
    op, stream = st["case"]["op"], torch.cuda.current_stream()
    if op == "act":
        A.moe_fp8_quantize_act(st["x"], st["q"], st["s"], swiglu=st["case"]["swiglu"], stream=stream)
        return st["q"], st["s"]
    if op == "weight":
        A.moe_fp8_quantize_weight(st["w"], st["q"], st["s"], stream=stream)
        return st["q"], st["s"]
    if op == "fwd":
        A.moe_grouped_gemm(st["x"], st["w"], st["offsets"], st["y"], stream=stream)
        return st["y"]
    if op == "fp8":
        A.moe_grouped_gemm_fp8(st["xq"], st["xs"], st["wq"], st["ws"], st["offsets"], st["y"], stream=stream)
        return st["y"]
    A.moe_grouped_gemm_dx(st["dy"], st["w"], st["offsets"], st["dx"], stream=stream)
    A.moe_grouped_gemm_dw(st["dy"], st["x"], st["offsets"], st["dw"], stream=stream)
    return st["dx"], st["dw"]


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def _touched(case):
    """Expected number of experts with rows (top_k distinct draws taken as independent ones)."""
    E, k, n = case["experts"], case["top_k"], case["tokens"]
    p = [(r + 1) ** -case["zipf"] for r in range(E)]
    t = sum(p)
    return max(min(E, k), sum(1 - (1 - min(1.0, k * v / t)) ** n for v in p))


def work(case):
    E, K, N = case["experts"], case["in"], case["out"]
    rows = case["tokens"] * case["top_k"]
    scales = 4 * -(-K // 128)
    out = 4 if case["f32"] else 2
    if case["op"] == "act":
        return {"bytes": rows * ((4 if case["swiglu"] else 2) * K + K + scales),
                "flops": rows * K * (9 if case["swiglu"] else 3)}
    if case["op"] == "weight":
        return {"bytes": E * (3 * N * K + -(-N // 128) * scales), "flops": 3 * E * N * K}
    live = _touched(case)
    if case["op"] == "fwd":
        return {"bytes": live * N * K * 2 + rows * (2 * K + out * N), "flops": 2 * rows * N * K}
    if case["op"] == "fp8":
        return {"bytes": live * (N * K + -(-N // 128) * scales) + rows * (K + scales + out * N),
                "flops": 2 * rows * N * K}
    return {"bytes": live * N * K * 2 + E * N * K * out + rows * (2 * K + 2 * N + out * K), "flops": 4 * rows * N * K}


# ------------------------------------------------------------------ the definition in 64 bits
def _codes64(v, s):
    """Nearest e4m3 values of v / s in 64 bits: steps of 2^(floor(log2) - 3), 2^-9 below 2^-6, ties to even."""
    r = v / s
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(r / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    st = prepare(case, seed)
    E, K, N = case["experts"], case["in"], case["out"]
    if case["op"] == "act":
        x = st["x"].double()
        if case["swiglu"]:
            x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
        q, s = torch.empty(x.shape, dtype=torch.float64, device="cuda"), st["s"].double()
        for b in range(s.shape[0]):
            m = x[:, 128 * b:128 * b + 128].abs().amax(1)
            s[b] = torch.where(m < TINY_BLOCK, torch.ones_like(m), m / E4M3_MAX)
            q[:, 128 * b:128 * b + 128] = _codes64(x[:, 128 * b:128 * b + 128], s[b][:, None])
        return q, s
    if case["op"] == "weight":
        q, s = torch.empty(st["w"].shape, dtype=F32, device="cuda"), st["s"].double()
        for i in range(s.shape[1]):
            for j in range(s.shape[2]):
                v = st["w"][:, 128 * i:128 * i + 128, 128 * j:128 * j + 128].double()
                m = v.abs().amax((1, 2))
                s[:, i, j] = torch.where(m < TINY_BLOCK, torch.ones_like(m), m / E4M3_MAX)
                q[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128] = _codes64(v, s[:, i, j][:, None, None]).float()
        return q, s
    off = st["offsets"].tolist()
    if case["op"] == "bwd":
        dx, dw = torch.zeros_like(st["dx"], dtype=torch.float64), torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
        for e in range(E):
            a, b = off[e], off[e + 1]
            dx[a:b] = st["dy"][a:b].double() @ st["w"][e].double()
            dw[e] = st["dy"][a:b].double().t() @ st["x"][a:b].double()
        return dx, dw
    y = torch.zeros_like(st["y"], dtype=torch.float64)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        if case["op"] == "fwd":
            y[a:b] = st["x"][a:b].double() @ st["w"][e].double().t()
            continue
        w = st["wq"][e].to(F32).double()
        for i in range(st["ws"].shape[1]):
            for j in range(st["ws"].shape[2]):
                w[128 * i:128 * i + 128, 128 * j:128 * j + 128] *= st["ws"][e, i, j].double()
        for j in range(st["xs"].shape[0]):
            xj = st["xq"][a:b, 128 * j:128 * j + 128].to(F32).double() * st["xs"][j, a:b].double()[:, None]
            y[a:b] += xj @ w[:, 128 * j:128 * j + 128].t()
    return y
