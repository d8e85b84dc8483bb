"""What stands between a decoder block's q|k|v projection and its output
projection, as cases that can be measured.

Three operators that are used together: the rotation of queries and keys by
their positions, after the heads' RMSNorm where there is one, forward and
backward; the same rotation on the way of new keys and values into a paged
cache, in 16 bits or in 4; and attention over the 4-bit cache. ``run``
computes them in elementary torch operations, or, where ``own`` is true, by
the package's entry points. ``exact`` computes them from their definition in
64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
FLOAT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
GROUP = 16                # 4-bit values along the head that share a scale
TILE = 16                 # tokens of a page that are stored together
LEAST = 2.0 ** -9         # least and largest scale (e4m3)
LARGEST = 448.0


def listed():
    return [
        # one token of a decode step at 896 features: latency alone
        {"name": "rope-1x16x64", "op": "rope", "back": False, "T": 1, "Hq": 14, "Hk": 2, "D": 64, "rot": 64,
         "pairs": "half", "norm": False, "dtype": "bf16"},
        # 8 x 4096 tokens of training or prompt at 4096 features, with QK-norm
        {"name": "rope-32768x40x128", "op": "rope", "back": False, "T": 32768, "Hq": 32, "Hk": 8, "D": 128,
         "rot": 128, "pairs": "half", "norm": True, "dtype": "bf16"},
        # the backward pass of half of that
        {"name": "rope-back-16384x40x128", "op": "rope", "back": True, "T": 16384, "Hq": 32, "Hk": 8, "D": 128,
         "rot": 128, "pairs": "half", "norm": True, "dtype": "bf16"},
        # a gradient kept in 32 bits; adjacent pairs, part of the head, odd rows
        {"name": "rope-back-777x7x80", "op": "rope", "back": True, "T": 777, "Hq": 6, "Hk": 1, "D": 80, "rot": 40,
         "pairs": "adjacent", "norm": True, "dtype": "fp32"},
        # 64 sequences' next tokens into a 16-bit cache
        {"name": "append-64x8x128", "op": "append", "bits": 16, "T": 64, "Hq": 32, "Hk": 8, "D": 128, "rot": 128,
         "pairs": "half", "norm": True, "dtype": "bf16", "page": 16},
        # a prompt batch into a 16-bit cache
        {"name": "append-8192x8x128", "op": "append", "bits": 16, "T": 8192, "Hq": 32, "Hk": 8, "D": 128, "rot": 128,
         "pairs": "half", "norm": True, "dtype": "bf16", "page": 64},
        # a prompt into a 4-bit cache, and its rows read back
        {"name": "append4-2001x4x64", "op": "append", "bits": 4, "T": 2001, "Hq": 28, "Hk": 4, "D": 64, "rot": 64,
         "pairs": "half", "norm": False, "dtype": "fp16", "page": 32},
        # one sequence's next token over a few thousand: latency
        {"name": "attend-1x4001", "op": "attend", "B": 1, "n": 1, "least": 4001, "most": 4001, "Hq": 32, "Hk": 8,
         "D": 128, "dtype": "bf16", "page": 16},
        # 64 sequences of all lengths: the cache's bytes
        {"name": "attend-64x8192", "op": "attend", "B": 64, "n": 1, "least": 1, "most": 8192, "Hq": 32, "Hk": 8,
         "D": 128, "dtype": "bf16", "page": 64},
        # four long contexts, groups of five heads
        {"name": "attend-4x131072", "op": "attend", "B": 4, "n": 1, "least": 100000, "most": 131072, "Hq": 40,
         "Hk": 8, "D": 128, "dtype": "bf16", "page": 64},
        # drafted tokens checked together: a few rows a sequence, small heads
        {"name": "attend-16x5x3000", "op": "attend", "B": 16, "n": 5, "least": 500, "most": 3000, "Hq": 14, "Hk": 2,
         "D": 64, "dtype": "fp16", "page": 16},
        # a piece of a prompt behind what is cached of it
        {"name": "attend-2x512x8192", "op": "attend", "B": 2, "n": 512, "least": 6000, "most": 8192, "Hq": 32,
         "Hk": 8, "D": 128, "dtype": "bf16", "page": 64},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], evenly spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    Hk = rng.choice([1, 2, 4, 8])
    if op == "attend":
        D, group = rng.choice([64, 128, 128]), _log(rng, 1, 8)
        most = _log(rng, 1, 131072)
        n = rng.choice([1, 1, 1, _log(rng, 2, 8), _log(rng, 9, 512)])
        B = _log(rng, 1, 64)
        while n > 1 and B * n > 1024:
            B = max(1, B // 2)
        while B > 1 and B * Hk * most * D > 1 << 28:
            B //= 2
        while n > 1 and B * Hk * group * n * most > 1 << 28:
            n = max(1, n // 2)
        n = min(n, most)
        return {"op": op, "B": B, "n": n, "least": max(1, most // rng.choice([1, 2, 100])), "most": most,
                "Hq": Hk * group, "Hk": Hk, "D": D, "dtype": dtype, "page": rng.choice([16, 32, 64, 128])}
    Hq = Hk * _log(rng, 1, 8)
    if op == "rope":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        D = rng.choice([64, 80, 96, 128, 128, 256])
        rot = rng.choice([D, D, D // 2])
        T = _log(rng, 1, min(32768, (1 << 27) // ((Hq + Hk) * D)))
        return {"op": op, "back": rng.choice([False, True]), "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot,
                "pairs": rng.choice(["half", "half", "adjacent"]), "norm": rng.choice([True, False]), "dtype": dtype}
    bits, D = rng.choice([16, 16, 4]), rng.choice([64, 128, 128])
    return {"op": op, "bits": bits, "T": _log(rng, 1, 8192 if bits == 16 else 2048), "Hq": Hq, "Hk": Hk, "D": D,
            "rot": rng.choice([D, D // 2]), "pairs": rng.choice(["half", "adjacent"]),
            "norm": rng.choice([True, False]), "dtype": dtype, "page": rng.choice([16, 32, 64])}


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype, std=1.0, mean=0.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)


def _pages(gen, B, blocks):
    """A page for each block of each sequence, in no order."""
    return torch.randperm(B * blocks, generator=gen, device="cuda").to(torch.int32).view(B, blocks)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    state = dict(case)
    D, Hq, Hk, dtype = case["D"], case["Hq"], case["Hk"], FLOAT[case["dtype"]]
    if case["op"] == "attend":
        B, n, page = case["B"], case["n"], case["page"]
        lens = torch.randint(case["least"], case["most"] + 1, (B,), generator=gen, device="cuda")
        lens[0] = case["most"]
        lens.clamp_(min=min(n, case["most"]))
        blocks = -(-case["most"] // page)
        table = _pages(gen, B, blocks)
        cache = torch.empty(B * blocks, Hk, page // TILE, 18 * D, dtype=torch.uint8, device="cuda")
        at_once = max(1, (1 << 25) // (Hk * page * D))
        for p in range(0, B * blocks, at_once):
            rows = min(at_once, B * blocks - p)
            k = _normal(gen, (rows, Hk, page, D), torch.float32)
            v = _normal(gen, (rows, Hk, page, D), torch.float32, std=0.5)
            cache[p:p + rows] = _packed(*_plain_quant4(k), *_plain_quant4(v))
        state |= {"q": _normal(gen, (B * n, Hq, D), dtype), "cache": cache, "table": table,
                  "lens": lens.to(torch.int32),
                  "starts": None if n == 1 else torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")}
        return state
    T, rot = case["T"], case["rot"]
    # q, k and v as the projection leaves them, side by side in a row
    qkv = _normal(gen, (T, Hq + 2 * Hk, D), dtype)
    state |= {"qkv": qkv, "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hk], "v": qkv[:, Hq + Hk:],
              "freq": 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot),
              "wq": _normal(gen, (D,), dtype, std=0.1, mean=1.0) if case["norm"] else None,
              "wk": _normal(gen, (D,), dtype, std=0.1, mean=1.0) if case["norm"] else None}
    if case["op"] == "rope":
        first = int(torch.randint(0, 1 << 20, (1,), generator=gen, device="cuda"))
        state["at"] = torch.arange(first, first + T, device="cuda") % 131072
        if case["back"]:
            state["dq"], state["dk"] = _normal(gen, (T, Hq, D), dtype, 0.01), _normal(gen, (T, Hk, D), dtype, 0.01)
        return state
    page = case["page"]
    blocks = -(-T // page) + 3
    state["at"] = torch.randint(0, 131072, (T,), generator=gen, device="cuda", dtype=torch.int32)
    state["slots"] = torch.randperm(blocks * page, generator=gen, device="cuda")[:T]
    if case["bits"] == 16:
        state["cache_k"] = _normal(gen, (blocks, page, Hk, D), dtype)
        state["cache_v"] = _normal(gen, (blocks, page, Hk, D), dtype)
    else:
        state["cache"] = torch.zeros(blocks, Hk, page // TILE, 18 * D, dtype=torch.uint8, device="cuda")
    return state


# ------------------------------------------------------------- plain forms
def _plain_angles(state):
    angle = state["at"].double()[:, None] * state["freq"][None, :]
    return torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]


def _plain_turn(x, cos, sin, rot, pairs):
    """x [T, H, D] in 32 bits, its first `rot` columns turned in pairs."""
    if pairs == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], dim=-1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_norm(x, w):
    """(x after the heads' norm, 1 / its rms) in 32 bits."""
    x = x.float()
    if w is None:
        return x, None
    rstd = 1.0 / torch.sqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
    return x * rstd * w.float(), rstd


def _plain_forward(state, name):
    cos, sin = _plain_angles(state)
    return _plain_turn(_plain_norm(state[name], state["w" + name])[0], cos, sin, state["rot"], state["pairs"])


def _plain_backward(state, name):
    """(dx, dw) for the gradient of the turned heads."""
    cos, sin = _plain_angles(state)
    x, w = state[name].float(), state["w" + name]
    g = _plain_turn(state["d" + name].float(), cos, -sin, state["rot"], state["pairs"])
    if w is None:
        return g.to(state[name].dtype), None
    rstd = 1.0 / torch.sqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
    c = (g * w.float() * x).mean(dim=-1, keepdim=True)
    dx = rstd * (g * w.float() - x * rstd.square() * c)
    return dx.to(state[name].dtype), (g * x * rstd).sum(dim=(0, 1))


def _plain_quant4(x):
    """x [..., D] -> (codes 0..15, scales as e4m3): a scale for 16 values; a
    code's three low bits are a place in VALUES. In 64 bits: many values of
    16 bits lie right on the border between two codes."""
    y = x.double().unflatten(-1, (-1, GROUP))
    top = y.abs().amax(dim=-1)
    # by a tensor: a product with 1 / 6 in its place would move the borders
    scale = (top / torch.full_like(top, 6.0)).clamp(LEAST, LARGEST).to(torch.float8_e4m3fn)
    y = y / scale.double()[..., None]
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * torch.signbit(y)
    return code.to(torch.uint8).flatten(-2), scale


def _packed(kc, ks, vc, vs):
    """Codes and scales [pages, heads, page, ...] as a 4-bit cache's bytes:
    for 16 tokens the keys' codes and scales token by token, then the values'
    codes and scales group by group."""
    P, H, page, D = kc.shape
    G = D // GROUP
    kc = kc[..., 0::2] | kc[..., 1::2] << 4
    vc = vc[..., 0::2] | vc[..., 1::2] << 4
    tiles = (P, H, page // TILE)
    parts = [kc.view(*tiles, TILE * D // 2), ks.view(torch.uint8).reshape(*tiles, TILE * G),
             vc.view(*tiles, TILE, G, 8).transpose(3, 4).flatten(3),
             vs.view(torch.uint8).reshape(*tiles, TILE, G).transpose(3, 4).flatten(3)]
    return torch.cat(parts, dim=-1)


def _unpacked(cache, D):
    """Codes and scales [pages, heads, page, ...] of a 4-bit cache's bytes,
    the codes two to a byte."""
    P, H, N, _ = cache.shape
    G, n = D // GROUP, TILE * D // 2
    kc, ks, vc, vs = cache.split([n, TILE * G, n, TILE * G], dim=-1)
    vc = vc.reshape(P, H, N, G, TILE, 8).transpose(3, 4)
    vs = vs.reshape(P, H, N, G, TILE).transpose(3, 4)
    return (kc.reshape(P, H, N * TILE, D // 2), ks.reshape(P, H, N * TILE, G).view(torch.float8_e4m3fn),
            vc.reshape(P, H, N * TILE, D // 2), vs.reshape(P, H, N * TILE, G).view(torch.float8_e4m3fn))


VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _two_values(dtype, device):
    """The two values of each byte, [256, 2]."""
    one = torch.tensor(VALUES + [-x for x in VALUES], dtype=dtype, device=device)
    return torch.stack([one.repeat(16), one.repeat_interleave(16)], dim=1)


def _values(codes, dtype):
    two = _two_values(dtype, codes.device)
    return two.index_select(0, codes.reshape(-1).int()).view(*codes.shape[:-1], -1)


def _plain_append(state):
    q, k = _plain_forward(state, "q"), _plain_forward(state, "k")
    q = q.to(state["q"].dtype)
    slots = state["slots"]
    if state["bits"] == 16:
        state["cache_k"].view(-1, *k.shape[1:])[slots] = k.to(state["k"].dtype)
        state["cache_v"].view(-1, *k.shape[1:])[slots] = state["v"]
        return {"q": q, "k": state["cache_k"], "v": state["cache_v"]}
    kc, ks = _plain_quant4(k)
    vc, vs = _plain_quant4(state["v"].float())
    cache, D = state["cache"], state["D"]
    P, H, N, _ = cache.shape
    page, within = slots // (N * TILE), slots % (N * TILE)
    tile, t = (within // TILE)[:, None], (within % TILE)[:, None]
    head = torch.arange(H, device=cache.device)[None, :]
    page, G, n = page[:, None], D // GROUP, TILE * D // 2
    ck, sk, cv, sv = cache.split([n, TILE * G, n, TILE * G], dim=-1)
    ck.unflatten(-1, (TILE, D // 2))[page, head, tile, t] = kc[..., 0::2] | kc[..., 1::2] << 4
    sk.unflatten(-1, (TILE, G))[page, head, tile, t] = ks.view(torch.uint8)
    by = (vc[..., 0::2] | vc[..., 1::2] << 4).unflatten(-1, (G, 8))
    g = torch.arange(G, device=cache.device)[None, None, :]
    cv.unflatten(-1, (G, TILE, 8))[page[..., None], head[..., None], tile[..., None], g, t[..., None]] = by
    sv.unflatten(-1, (G, TILE))[page[..., None], head[..., None], tile[..., None], g, t[..., None]] = vs.view(torch.uint8)
    # the new rows, read back
    rk, rks, rv, rvs = (x.transpose(1, 2).flatten(0, 1)[slots] for x in _unpacked(cache, D))
    eight = torch.float8_e4m3fn
    return {"q": q, "k": _values(rk, torch.float32).to(eight), "k_scale": rks,
            "v": _values(rv, torch.float32).to(eight), "v_scale": rvs}


def _plain_attend(state):
    q, cache, table, lens = state["q"], state["cache"], state["table"].long(), state["lens"].long()
    B, n, Hq, Hk, D = state["B"], state["n"], state["Hq"], state["Hk"], state["D"]
    P, H, N, _ = cache.shape
    rows = cache[table.view(-1)]                                   # [B * blocks, H, N, 18 D]
    kc, ks, vc, vs = _unpacked(rows, D)

    def dense(codes, scale):                                       # [B, H, L, D]
        x = _values(codes, torch.float32).unflatten(-1, (-1, GROUP)) * scale.float()[..., None]
        return x.flatten(-2).view(B, -1, H, N * TILE, D).transpose(1, 2).flatten(2, 3)

    k, v = dense(kc, ks), dense(vc, vs)
    L = k.shape[2]
    qs = q.float().view(B, n, Hk, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D)
    s = torch.matmul(qs, k.transpose(2, 3)) / math.sqrt(D)         # [B, Hk, n * group, L]
    seen = lens[:, None] - n + 1 + torch.arange(n, device=q.device)[None, :]
    seen = seen.repeat_interleave(Hq // Hk, dim=1)[:, None, :, None]
    s = s.masked_fill(torch.arange(L, device=q.device) >= seen, float("-inf"))
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p, v) / total
    lse = (m + torch.log(total)).view(B, Hk, n, -1).transpose(1, 2).reshape(B * n, Hq)
    out = out.view(B, Hk, n, Hq // Hk, D).transpose(1, 2).reshape(B * n, Hq, D)
    return {"out": out.to(q.dtype), "lse": lse}


def run(state):
    op = state["op"]
    if own:
        from rmsnorm_fwd_bwd_02_gb300 import rmsnorm as rn
        if op == "attend":
            out, lse = rn.rmsnorm_kv4_attention(state["q"], state["cache"], state["table"], state["lens"],
                                                q_starts=state["starts"], want_lse=True)
            return {"out": out, "lse": lse}
        how = {"wq": state["wq"], "wk": state["wk"], "eps": EPS, "interleaved": state["pairs"] == "adjacent"}
        if op == "append" and state["bits"] == 16:
            q = rn.rmsnorm_rope_append(state["k"], state["v"], state["at"], state["freq"], state["slots"],
                                       state["cache_k"], state["cache_v"], q=state["q"], **how)
            return {"q": q, "k": state["cache_k"], "v": state["cache_v"]}
        if op == "append":
            q = rn.rmsnorm_rope_append_kv4(state["k"], state["v"], state["at"], state["freq"], state["slots"],
                                           state["cache"], q=state["q"], **how)
            k, k_scale, v, v_scale = rn.rmsnorm_kv4_read(state["cache"], state["slots"])
            return {"q": q, "k": k, "k_scale": k_scale, "v": v, "v_scale": v_scale}
        if state["back"]:
            dq, dk, dwq, dwk = rn.rmsnorm_rope_bwd(state["dq"], state["q"], state["at"], state["freq"],
                                                   dyk=state["dk"], k=state["k"], **how)
            return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
        q, k, _ = rn.rmsnorm_rope_fwd(state["q"], state["at"], state["freq"], k=state["k"], want_rstd=False, **how)
        return {"q": q, "k": k}
    if op == "attend":
        return _plain_attend(state)
    if op == "append":
        return _plain_append(state)
    if state["back"]:
        (dq, dwq), (dk, dwk) = _plain_backward(state, "q"), _plain_backward(state, "k")
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    return {"q": _plain_forward(state, "q").to(state["q"].dtype), "k": _plain_forward(state, "k").to(state["k"].dtype)}


def work(case):
    D, Hq, Hk, es = case["D"], case["Hq"], case["Hk"], BYTES[case["dtype"]]
    if case["op"] == "attend":
        B, n = case["B"], case["n"]
        # the lengths are even over [least, most], the first is `most`; a row
        # sees its sequence up to its own place
        mean = (case["most"] + (B - 1) * (case["least"] + case["most"]) / 2) / B
        mean = max(mean, min(n, case["most"]))
        seen = sum(max(0.0, mean - n + 1 + i) for i in range(n))
        # a 4-bit value takes 4.5 bits with its share of a scale
        return {"bytes": B * Hk * mean * D * 2 * 9 / 16 + B * n * Hq * (2 * D * es + 4),
                "flops": 4 * B * Hq * seen * D}
    T, rot = case["T"], case["rot"]
    heads = T * (Hq + Hk) * D
    if case["op"] == "rope":
        if not case["back"]:
            return {"bytes": 2 * heads * es + T * 8 + rot * 4, "flops": heads * (3 + 4 * case["norm"])}
        arrays = 3 if case["norm"] else 2          # dy, dx, and x for the norm
        return {"bytes": arrays * heads * es + T * 8 + rot * 4, "flops": heads * (3 + 12 * case["norm"])}
    kv = T * 2 * Hk * D
    stored = kv * es if case["bits"] == 16 else kv * 9 // 16
    back = 0 if case["bits"] == 16 else kv * 9 // 16 + kv + kv // GROUP
    return {"bytes": 2 * T * Hq * D * es + kv * es + stored + back + T * 12, "flops": heads * (3 + 4 * case["norm"])}


# ------------------------------------------------------- 64-bit definitions
def _exact_turn(x, s, sign=1.0):
    """x [T, H, D] turned: each pair as a complex number times e^(i angle)."""
    angle = s["at"].to(torch.float64)[:, None, None] * s["freq"] * sign
    unit = torch.polar(torch.ones_like(angle), angle)
    rot, out = s["rot"], x.clone()
    at = torch.arange(rot, device=x.device)
    first, second = (at[:rot // 2], at[rot // 2:]) if s["pairs"] == "half" else (at[0::2], at[1::2])
    z = torch.complex(x[..., first], x[..., second]) * unit
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_heads(s, name):
    x = s[name].double()
    if s["w" + name] is None:
        return _exact_turn(x, s)
    r = (x.pow(2).sum(-1, keepdim=True) / s["D"] + EPS).pow(-0.5)
    return _exact_turn(x * r * s["w" + name].double(), s)


def _exact_back(s, name):
    x, g = s[name].double(), _exact_turn(s["d" + name].double(), s, -1.0)
    if s["w" + name] is None:
        return g, None
    w = s["w" + name].double()
    r = (x.pow(2).sum(-1, keepdim=True) / s["D"] + EPS).pow(-0.5)
    unit = x * r
    return r * (g * w - unit * (g * w * unit).mean(-1, keepdim=True)), torch.einsum("thd,thd->d", g, unit)


def _exact_quant4(x):
    """(values on the 4-bit grid, scales) of x [T, H, D] in 64 bits."""
    y = x.unflatten(-1, (-1, GROUP))
    top = y.abs().amax(-1)
    top = torch.true_divide(top, torch.full_like(top, 6.0)).clamp(LEAST, LARGEST)
    _, e = torch.frexp(top)
    # three fraction bits: steps of 2^-9 to 2^5, by the exponent
    steps = torch.tensor([2.0 ** i for i in range(-9, 6)], dtype=top.dtype, device=top.device)
    step = steps[(e - 1).clamp(-6, 8) + 6]
    scale = torch.round(top / step) * step
    a = y.abs() / scale[..., None]
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    return ((torch.round(a / step) * step).clamp(max=6.0) * torch.sign(y)).flatten(-2), scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        if case["back"]:
            (dq, dwq), (dk, dwk) = _exact_back(s, "q"), _exact_back(s, "k")
            return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
        return {"q": _exact_heads(s, "q"), "k": _exact_heads(s, "k")}
    if case["op"] == "append":
        q, k, v, slots = _exact_heads(s, "q"), _exact_heads(s, "k"), s["v"].double(), s["slots"]
        if case["bits"] == 16:
            ck, cv = s["cache_k"].double(), s["cache_v"].double()
            ck.view(-1, *k.shape[1:])[slots] = k
            cv.view(-1, *v.shape[1:])[slots] = v
            return {"q": q, "k": ck, "v": cv}
        (k, ks), (v, vs) = _exact_quant4(k), _exact_quant4(v)
        return {"q": q, "k": k, "k_scale": ks, "v": v, "v_scale": vs}
    B, n, Hk, D = case["B"], case["n"], case["Hk"], case["D"]
    group = case["Hq"] // Hk
    out = torch.empty(B * n, case["Hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.empty(B * n, case["Hq"], dtype=torch.float64, device="cuda")
    page = case["page"]
    for b in range(B):
        L = int(s["lens"][b])
        pages = s["cache"][s["table"][b, :-(-L // page)].long()]
        kc, ks, vc, vs = _unpacked(pages, D)
        for h in range(Hk):
            k, v = ((_values(c[:, h], torch.float64).unflatten(-1, (-1, GROUP)) * t[:, h].double()[..., None])
                    .view(-1, D)[:L] for c, t in ((kc, ks), (vc, vs)))
            rows, heads = slice(b * n, (b + 1) * n), slice(h * group, (h + 1) * group)
            x = torch.einsum("ngd,ld->ngl", s["q"][rows, heads].double(), k) * D ** -0.5
            hidden = torch.arange(L, device="cuda")[None, :] > torch.arange(L - n, L, device="cuda")[:, None]
            x.masked_fill_(hidden[:, None, :], float("-inf"))
            lse[rows, heads] = torch.logsumexp(x, dim=-1)
            out[rows, heads] = torch.einsum("ngl,ld->ngd", torch.softmax(x, dim=-1), v)
    return {"out": out, "lse": lse}
