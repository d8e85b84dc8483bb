"""The 8-bit serving path's operators, as cases that can be measured.

Three operators that are used together: the RMSNorm (optionally of a residual
sum) whose output is 8-bit floating point with one scale for each 128
features of a row; the same quantisation of a matrix alone, for each 128
features of a row (activations) or each 128 x 128 block (weights); and the
matrix product of two such tensors. ``run`` computes them in elementary torch
operations, or, where ``own`` is true, by the package's entry points.
``exact`` computes them from their definition in 64 bits.
"""
import torch

own = False

GROUP = 128                    # values that share a scale, along the features
AMAX_MIN = 2.0 ** -100         # least magnitude that a scale is made for
FLOAT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EIGHT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one token of a decode step at 896 features: latency alone
        {"name": "norm-1x896", "op": "norm", "M": 1, "H": 896, "dtype": "bf16", "residual": True, "to": "e4m3"},
        # odd rows and features: a row ends inside a group and starts unaligned
        {"name": "norm-4001x1001", "op": "norm", "M": 4001, "H": 1001, "dtype": "fp16", "residual": False, "to": "e4m3"},
        # a prompt batch of 16384 tokens at 5120 features, between two blocks
        {"name": "norm-16384x5120", "op": "norm", "M": 16384, "H": 5120, "dtype": "bf16", "residual": True, "to": "e4m3"},
        # the first norm over 8 x 4096 tokens at 4096 features
        {"name": "norm-32768x4096", "op": "norm", "M": 32768, "H": 4096, "dtype": "bf16", "residual": False, "to": "e4m3"},
        # a gradient kept in 32 bits, odd rows, to the wider 8-bit format
        {"name": "quant-777x4864", "op": "quant", "M": 777, "H": 4864, "dtype": "fp32", "rows": 1, "to": "e5m2"},
        # the input of a block's last projection (12288 wide) for 8192 tokens
        {"name": "quant-8192x12288", "op": "quant", "M": 8192, "H": 12288, "dtype": "bf16", "rows": 1, "to": "e4m3"},
        # a gate|up weight, quantised when a model is loaded
        {"name": "quant-24576x4096", "op": "quant", "M": 24576, "H": 4096, "dtype": "bf16", "rows": 128, "to": "e4m3"},
        # one token's q|k|v projection at 896 features: latency alone
        {"name": "gemm-1x2048x896", "op": "gemm", "M": 1, "N": 2048, "K": 896, "out": "bf16", "a": "e4m3", "b": "e4m3"},
        # 16 tokens' gate|up projection: the weight's bytes
        {"name": "gemm-16x24576x4096", "op": "gemm", "M": 16, "N": 24576, "K": 4096, "out": "bf16", "a": "e4m3", "b": "e4m3"},
        # 64 tokens' q|k|v projection
        {"name": "gemm-64x6144x4096", "op": "gemm", "M": 64, "N": 6144, "K": 4096, "out": "bf16", "a": "e4m3", "b": "e4m3"},
        # a short prompt: nothing is a multiple of a tile
        {"name": "gemm-333x1001x5121", "op": "gemm", "M": 333, "N": 1001, "K": 5121, "out": "fp16", "a": "e4m3", "b": "e4m3"},
        # a prompt batch's gate|up projection: the tensor cores' rate
        {"name": "gemm-8192x24576x4096", "op": "gemm", "M": 8192, "N": 24576, "K": 4096, "out": "bf16", "a": "e4m3", "b": "e4m3"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], evenly spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "quant", "gemm"])
    if op == "gemm":
        M, N, K = _log(rng, 1, 8192), _log(rng, 16, 24576), _log(rng, 64, 16384)
        return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "a": rng.choice(["e4m3", "e4m3", "e5m2"]), "b": "e4m3"}
    H = _log(rng, 64, 16384)
    M = _log(rng, 1, min(32768, (1 << 27) // H))
    case = {"op": op, "M": M, "H": H, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
            "to": rng.choice(["e4m3", "e4m3", "e5m2"])}
    if op == "norm":
        case["residual"] = rng.choice([False, True])
    else:
        case["rows"] = rng.choice([1, 1, 128])
    return case


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype, std=1.0, mean=0.0, outliers=0.0):
    """N(mean, std); 0.1 % of the entries times `outliers` where it is set, as
    hidden states have them."""
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).add_(mean)
    if outliers:
        n = t.numel()
        at = torch.randint(n, (max(1, n // 1000),), generator=gen, device="cuda")
        t.view(-1)[at] *= outliers
    return t.to(dtype)


def _rows16(t):
    """t with its rows starting at multiples of 16 bytes, as a projection
    reads them."""
    M, K = t.shape
    ld = -(-K // 16) * 16
    buf = torch.zeros(M, ld, device=t.device, dtype=torch.uint8).view(t.dtype)
    buf.view(torch.uint8)[:, :K] = t.view(torch.uint8)
    return buf[:, :K]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    state = dict(case)
    if case["op"] == "norm":
        shape, dtype = (case["M"], case["H"]), FLOAT[case["dtype"]]
        state["x"] = _normal(gen, shape, dtype, outliers=50.0)
        state["w"] = _normal(gen, (case["H"],), dtype, std=0.1, mean=1.0)
        state["r"] = _normal(gen, shape, dtype, outliers=50.0) if case["residual"] else None
    elif case["op"] == "quant":
        blocks = case["rows"] == GROUP
        state["x"] = _normal(gen, (case["M"], case["H"]), FLOAT[case["dtype"]], std=0.02 if blocks else 1.0,
                             outliers=0.0 if blocks else 50.0)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        a = _normal(gen, (M, K), torch.bfloat16, outliers=50.0)
        b = _normal(gen, (N, K), torch.bfloat16, std=0.02)
        qa, state["sa"] = _plain_quant(a.float(), 1, case["a"])
        qb, state["sb"] = _plain_quant(b.float(), GROUP, case["b"])
        state["qa"], state["qb"] = _rows16(qa), _rows16(qb)
    return state


# ------------------------------------------------------------- plain forms
def _plain_quant(y, rows, to):
    """(q, scales) of y [M, H] in 32 bits: a scale for `rows` x 128 values."""
    M, H = y.shape
    padded = torch.nn.functional.pad(y, (0, -H % GROUP, 0, -M % rows))
    R, G = padded.shape[0] // rows, padded.shape[1] // GROUP
    blocks = padded.view(R, rows, G, GROUP)
    amax = blocks.abs().amax(dim=(1, 3), keepdim=True)
    scale = amax.clamp(min=AMAX_MIN) / LARGEST[to]
    q = (blocks / scale).to(EIGHT[to])
    q = q.view(torch.uint8).view(R * rows, G * GROUP)[:M, :H].contiguous().view(EIGHT[to])
    return q, scale.view(R, G)


def _plain_norm(x, r, w, eps, to):
    if r is None:
        h, hf = None, x.float()
    else:
        h = (x.float() + r.float()).to(x.dtype)
        hf = h.float()
    rstd = 1.0 / torch.sqrt(hf.square().mean(dim=-1, keepdim=True) + eps)
    q, scale = _plain_quant(hf * rstd * w.float(), 1, to)
    return {"q": q, "scale": scale, "rstd": rstd.view(-1), "h": h}


def _plain_gemm(qa, sa, qb, sb, dtype):
    M, K = qa.shape
    N = qb.shape[0]
    a = qa.float() * sa.repeat_interleave(GROUP, dim=1)[:, :K]
    b = qb.float() * sb.repeat_interleave(GROUP, dim=0)[:N].repeat_interleave(GROUP, dim=1)[:, :K]
    return (a @ b.t()).to(dtype)


EPS = 1e-6


def run(state):
    op = state["op"]
    if own:
        from rmsnorm_fwd_bwd_02_gb300 import rmsnorm as rn
        if op == "norm":
            out = rn.rmsnorm_fwd_fp8(state["x"], state["w"], r=state["r"], eps=EPS, qdtype=EIGHT[state["to"]])
            h, (q, scale, rstd) = (None, out) if state["r"] is None else (out[0], out[1:])
            return {"q": q, "scale": scale, "rstd": rstd, "h": h}
        if op == "quant":
            q, scale = rn.rmsnorm_quant_fp8(state["x"], block_rows=state["rows"], qdtype=EIGHT[state["to"]])
            return {"q": q, "scale": scale}
        return rn.rmsnorm_gemm_fp8(state["qa"], state["sa"], state["qb"], state["sb"],
                                   out_dtype=FLOAT[state["out"]], static_weights=True)
    if op == "norm":
        return _plain_norm(state["x"], state["r"], state["w"], EPS, state["to"])
    if op == "quant":
        q, scale = _plain_quant(state["x"].float(), state["rows"], state["to"])
        return {"q": q, "scale": scale}
    return _plain_gemm(state["qa"], state["sa"], state["qb"], state["sb"], FLOAT[state["out"]])


def work(case):
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        G = -(-K // GROUP)
        return {"bytes": M * K + N * K + 4 * G * (M + -(-N // GROUP)) + M * N * BYTES[case["out"]],
                "flops": 2 * M * N * K}
    M, H, es = case["M"], case["H"], BYTES[case["dtype"]]
    G = -(-H // GROUP)
    if case["op"] == "quant":
        return {"bytes": M * H * (es + 1) + 4 * G * -(-M // case["rows"]), "flops": 3 * M * H}
    full = 3 if case["residual"] else 1        # x; with a residual also r and the sum written
    return {"bytes": M * H * (full * es + 1) + H * es + 4 * M * (G + 1), "flops": 8 * M * H}


# ------------------------------------------------------- 64-bit definitions
def _exact_round8(v, to):
    """v rounded to nearest (ties to even) in an 8-bit format: 3 or 2
    fraction bits, exponents from -6 or -14, magnitudes up to LARGEST."""
    bits, low = (3, -6) if to == "e4m3" else (2, -14)
    _, e = torch.frexp(v)                       # |v| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=low) - bits)
    return (torch.round(v / step) * step).clamp(-LARGEST[to], LARGEST[to])


def _exact_quant(y, rows, to):
    M, H = y.shape
    q = torch.empty_like(y)
    scale = torch.empty(-(-M // rows), -(-H // GROUP), dtype=torch.float64, device=y.device)
    for g in range(scale.shape[1]):
        cols = y[:, g * GROUP:(g + 1) * GROUP]
        top = cols.abs().amax(dim=1)
        if rows > 1:
            top = torch.cat([top, top.new_zeros(-M % rows)]).view(-1, rows).amax(dim=1)
        scale[:, g] = torch.maximum(top, torch.full_like(top, AMAX_MIN)) / LARGEST[to]
        s = scale[:, g].repeat_interleave(rows)[:M]
        q[:, g * GROUP:(g + 1) * GROUP] = _exact_round8(cols / s[:, None], to)
    return q, scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm":
        # the largest takes about two seconds at a GPU's 64-bit rate
        M, N, K = case["M"], case["N"], case["K"]
        total = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        of = torch.arange(N, device="cuda") // GROUP
        for g in range(s["sa"].shape[1]):
            k = slice(g * GROUP, min(K, (g + 1) * GROUP))
            part = torch.mm(s["qa"][:, k].double(), s["qb"][:, k].double().t())
            part *= s["sa"][:, g].double()[:, None]
            part *= s["sb"][:, g].double()[of][None, :]
            total += part
        return total
    if case["op"] == "quant":
        q, scale = _exact_quant(s["x"].double(), case["rows"], case["to"])
        return {"q": q, "scale": scale}
    h = None
    v = s["x"].double()
    if s["r"] is not None:
        h = (v + s["r"].double()).to(s["x"].dtype)      # the stored sum, which the norm acts on
        v = h.double()
    rstd = (v.pow(2).sum(dim=1) / case["H"] + EPS).pow(-0.5)
    q, scale = _exact_quant(v * rstd[:, None] * s["w"].double()[None, :], 1, case["to"])
    return {"q": q, "scale": scale, "rstd": rstd, "h": h}
