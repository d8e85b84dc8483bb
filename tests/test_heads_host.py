"""CPU tier: the entry points on attention heads reject bad arguments on the
host before any CUDA call, and the binding rejects what the library cannot
see. The argument checks pass made-up addresses; every call below fails a
check (or has nothing to do), so nothing is launched."""
import ctypes

import pytest
import torch

from rmsnorm_fwd_bwd_02_gb300 import rmsnorm as rn
from tests.test_abi_host import (ALIAS, BAD_DTYPE, BAD_EPS, BAD_SHAPE, BAD_STRIDE, BF16, F16, F32,
                                 HEADER, MISALIGNED, NAN, NULLPTR, OK, UNSUPPORTED, WORKSPACE, lib)  # noqa: F401

BAD_FLAGS = -11
AT = [0x7f0000000000 + (i << 36) for i in range(16)]
i64, vp, f32, cint = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int


class Heads(ctypes.Structure):
    _fields_ = [("x", vp), ("x_token", i64), ("x_head", i64), ("w", vp), ("y", vp), ("y_token", i64),
                ("y_head", i64), ("heads", i64)]


class Grad(ctypes.Structure):
    _fields_ = [("dy", vp), ("dy_token", i64), ("dy_head", i64), ("x", vp), ("x_token", i64), ("x_head", i64),
                ("w", vp), ("dx", vp), ("dx_token", i64), ("dx_head", i64), ("dw", vp), ("heads", i64)]


class Rotation(ctypes.Structure):
    _fields_ = [("positions", vp), ("position_bits", cint), ("freq", vp), ("rot", i64), ("adjacent", cint),
                ("amplitude", f32)]


def heads(x=AT[0], y=AT[1], w=None, n=4, D=64, **kw):
    d = {"x": x, "x_token": n * D, "x_head": D, "w": w, "y": y, "y_token": n * D, "y_head": D, "heads": n}
    return Heads(**{**d, **kw})


def grad(dy=AT[0], x=AT[1], w=AT[2], dx=AT[3], dw=AT[4], n=4, D=64, **kw):
    d = {"dy": dy, "dy_token": n * D, "dy_head": D, "x": x, "x_token": n * D, "x_head": D, "w": w, "dx": dx,
         "dx_token": n * D, "dx_head": D, "dw": dw, "heads": n}
    return Grad(**{**d, **kw})


def rotation(**kw):
    d = {"positions": AT[8], "position_bits": 64, "freq": AT[9], "rot": 64, "adjacent": 0, "amplitude": 1.0}
    return Rotation(**{**d, **kw})


def ref(s):
    return None if s is None else ctypes.byref(s)


def fwd(lib, q="default", k=None, rot="default", rstd=None, T=8, D=64, eps=1e-6, dtype=BF16):
    q = heads() if q == "default" else q
    rot = rotation() if rot == "default" else rot
    return lib.rmsnorm_rope_fwd(ref(q), ref(k), ref(rot), rstd, T, D, eps, dtype, None)


def test_rotation_refusals(lib):  # noqa: F811
    assert fwd(lib, dtype=3) == BAD_DTYPE and fwd(lib, rot=rotation(position_bits=16)) == BAD_DTYPE
    assert fwd(lib, T=-1) == BAD_SHAPE and fwd(lib, D=0) == BAD_SHAPE
    assert fwd(lib, rot=rotation(rot=63)) == BAD_SHAPE and fwd(lib, rot=rotation(rot=66)) == BAD_SHAPE
    assert fwd(lib, rot=rotation(rot=-2)) == BAD_SHAPE
    assert fwd(lib, q=heads(n=0)) == BAD_SHAPE and fwd(lib, q=heads(n=4, heads=-1)) == BAD_SHAPE
    assert fwd(lib, D=257) == UNSUPPORTED and fwd(lib, T=2 ** 31) == UNSUPPORTED
    assert fwd(lib, rot=rotation(adjacent=2)) == BAD_FLAGS
    for e in (NAN, -1.0, float("inf")):
        assert fwd(lib, eps=e) == BAD_EPS
    assert fwd(lib, rot=rotation(amplitude=NAN)) == BAD_EPS
    assert fwd(lib, q=None) == NULLPTR
    assert fwd(lib, q=heads(x=None)) == NULLPTR and fwd(lib, q=heads(y=None)) == NULLPTR
    assert fwd(lib, rot=rotation(positions=None)) == NULLPTR and fwd(lib, rot=rotation(freq=None)) == NULLPTR
    assert fwd(lib, q=heads(x_token=-1)) == BAD_STRIDE and fwd(lib, q=heads(x_head=-64)) == BAD_STRIDE
    assert fwd(lib, q=heads(y_head=63)) == BAD_STRIDE          # outputs do not overlap themselves
    assert fwd(lib, q=heads(y_token=255)) == BAD_STRIDE
    assert fwd(lib, q=heads(x_token=2 ** 61)) == BAD_STRIDE
    assert fwd(lib, q=heads(x=AT[0] + 1)) == MISALIGNED and fwd(lib, q=heads(w=AT[2] + 1)) == MISALIGNED
    assert fwd(lib, rot=rotation(freq=AT[9] + 4)) == MISALIGNED
    assert fwd(lib, rot=rotation(positions=AT[8] + 4)) == MISALIGNED
    assert fwd(lib, rstd=AT[5] + 2) == MISALIGNED


def test_rotation_aliasing(lib):  # noqa: F811
    k = heads(x=AT[2], y=AT[3])
    assert fwd(lib, q=heads(y=AT[0] + 128)) == ALIAS           # neither x nor apart from it
    assert fwd(lib, k=heads(x=AT[2], y=AT[1])) == ALIAS        # k's output over q's
    assert fwd(lib, k=heads(x=AT[1], y=AT[3])) == ALIAS        # k's input over q's output
    assert fwd(lib, k=k, rstd=AT[0]) == ALIAS and fwd(lib, k=k, rstd=AT[3]) == ALIAS
    assert fwd(lib, q=heads(w=AT[1] + 64)) == ALIAS            # a weight in the output
    assert fwd(lib, rot=rotation(positions=AT[1] + 8)) == ALIAS
    assert fwd(lib, rot=rotation(freq=AT[1] + 8)) == ALIAS
    # a window of the q|k|v projection over its neighbour's columns
    qkv = {"x_token": 640, "y_token": 640}
    assert fwd(lib, q=heads(x=AT[0], y=AT[0], **qkv), k=heads(x=AT[0] + 256, y=AT[0] + 256, **qkv)) == ALIAS


def test_nothing_to_do(lib):  # noqa: F811
    empty = heads(x=None, y=None)
    assert fwd(lib, q=empty, rot=rotation(positions=None, freq=None), T=0) == OK
    assert fwd(lib, q=empty, rot=None, T=0) == OK
    g = grad(dy=None, x=None, w=None, dx=None, dw=None)
    assert lib.rmsnorm_rope_bwd(ref(g), None, None, None, None, 0, 0, 64, 1e-6, BF16, None) == OK
    assert attend(lib, T=0, B=0, q=None, out=None, table=None, lens=None, ws=None) == OK


def bwd(lib, q="default", k=None, rot="default", rstd=None, ws=AT[6], size=1 << 30, T=8, D=64, eps=1e-6, dtype=BF16):
    q = grad() if q == "default" else q
    rot = rotation() if rot == "default" else rot
    return lib.rmsnorm_rope_bwd(ref(q), ref(k), ref(rot), rstd, ws, size, T, D, eps, dtype, None)


def test_backward_refusals(lib):  # noqa: F811
    assert bwd(lib, dtype=7) == BAD_DTYPE and bwd(lib, T=-1) == BAD_SHAPE and bwd(lib, D=300) == UNSUPPORTED
    assert bwd(lib, q=None) == NULLPTR
    for k in ("dy", "x", "dx", "dw"):
        assert bwd(lib, q=grad(**{k: None})) == NULLPTR, k
    assert bwd(lib, q=grad(dx_head=32)) == BAD_STRIDE and bwd(lib, q=grad(x_token=-4)) == BAD_STRIDE
    assert bwd(lib, q=grad(dy=AT[0] + 1)) == MISALIGNED and bwd(lib, q=grad(dw=AT[4] + 2)) == MISALIGNED
    assert bwd(lib, ws=AT[6] + 8) == MISALIGNED
    assert bwd(lib, q=grad(dx=AT[0] + 64)) == ALIAS and bwd(lib, q=grad(dx=AT[1] + 64)) == ALIAS
    assert bwd(lib, q=grad(dw=AT[3] + 64)) == ALIAS and bwd(lib, q=grad(dx=AT[2])) == ALIAS
    assert bwd(lib, ws=AT[0] - 4096, size=1 << 20) == ALIAS    # the workspace over dy
    assert bwd(lib, rstd=AT[3] + 64) == ALIAS
    assert bwd(lib, k=grad(dy=AT[10], x=AT[11], dx=AT[12], dw=AT[4])) == ALIAS     # both dw in one place
    assert bwd(lib, k=grad(dy=AT[10], x=AT[11], dx=AT[3], dw=AT[13])) == ALIAS     # both dx in one place
    assert bwd(lib, ws=None) == WORKSPACE


def append(lib, q=None, k="default", v="default", rot="default", slots=AT[10], bits=64, pages=4, page=16, kp=None,
           vp=None, T=8, D=64, dtype=BF16, eps=1e-6):
    tok = 4 * 64
    k = heads(x=AT[0], y=AT[1], y_token=tok) if k == "default" else k
    v = heads(x=AT[2], y=AT[3], y_token=tok) if v == "default" else v
    rot = rotation() if rot == "default" else rot
    return lib.rmsnorm_rope_append(ref(q), ref(k), ref(v), ref(rot), slots, bits, pages, page,
                                   page * tok if kp is None else kp, page * tok if vp is None else vp, T, D, eps,
                                   dtype, None)


def append4(lib, q=None, k="default", v="default", rot="default", slots=AT[10], bits=32, cache=AT[5], pages=4,
            page=16, ks=None, vs=None, T=8, D=64, dtype=BF16):
    k = heads(x=AT[0], y=None) if k == "default" else k
    v = heads(x=AT[2], y=None) if v == "default" else v
    rot = rotation() if rot == "default" else rot
    return lib.rmsnorm_rope_append_kv4(ref(q), ref(k), ref(v), ref(rot), slots, bits, cache, pages, page, ks, vs, T,
                                       D, 1e-6, dtype, None)


def test_append_refusals(lib):  # noqa: F811
    assert append(lib, dtype=5) == BAD_DTYPE and append(lib, bits=8) == BAD_DTYPE
    assert append(lib, k=None) == NULLPTR and append(lib, v=None) == NULLPTR
    assert append(lib, slots=None) == NULLPTR and append(lib, k=heads(x=None)) == NULLPTR
    assert append(lib, v=heads(x=AT[2], y=AT[3], n=2)) == BAD_SHAPE
    assert append(lib, pages=-1) == BAD_SHAPE and append(lib, page=0) == BAD_SHAPE
    assert append(lib, v=heads(x=AT[2], y=AT[3], w=AT[4])) == UNSUPPORTED
    assert append(lib, kp=255) == BAD_STRIDE                   # pages over each other
    assert append(lib, k=heads(y_head=32)) == BAD_STRIDE
    assert append(lib, slots=AT[10] + 4) == MISALIGNED
    assert append(lib, v=heads(x=AT[2], y=AT[1])) == ALIAS     # one start for k and v
    assert append(lib, k=heads(x=AT[1], y=AT[1])) == ALIAS     # an input in the cache
    assert append(lib, q=heads(x=AT[6], y=AT[1])) == ALIAS     # q's output in the cache
    assert append(lib, slots=AT[1] + 64) == ALIAS
    assert append(lib, T=0, slots=None) == OK


def test_append_kv4_refusals(lib):  # noqa: F811
    assert append4(lib, page=24) == UNSUPPORTED
    for D in (32, 80, 256):
        assert append4(lib, k=heads(D=D), v=heads(x=AT[2], D=D), D=D, rot=None) == UNSUPPORTED
    assert append4(lib, cache=None) == NULLPTR
    assert append4(lib, cache=AT[5] + 8) == MISALIGNED and append4(lib, ks=AT[6] + 2) == MISALIGNED
    assert append4(lib, cache=AT[0]) == ALIAS and append4(lib, ks=AT[5] + 64) == ALIAS
    assert append4(lib, T=0, cache=None, slots=None) in (OK, NULLPTR)


def read(lib, cache=AT[0], pages=4, page=16, H=2, D=64, slots=AT[1], bits=64, n=8, k=AT[2], ks=AT[3], v=AT[4],
         vs=AT[5]):
    return lib.rmsnorm_kv4_read(cache, pages, page, H, D, slots, bits, n, k, ks, v, vs, None)


def test_read_refusals(lib):  # noqa: F811
    assert read(lib, bits=1) == BAD_DTYPE and read(lib, n=-1) == BAD_SHAPE and read(lib, H=0) == BAD_SHAPE
    assert read(lib, D=96) == UNSUPPORTED and read(lib, page=8) == UNSUPPORTED
    for a in ("cache", "slots", "k", "ks", "v", "vs"):
        assert read(lib, **{a: None}) == NULLPTR
    assert read(lib, k=AT[2] + 8) == MISALIGNED
    assert read(lib, k=AT[0]) == ALIAS and read(lib, vs=AT[2] + 4) == ALIAS
    assert read(lib, n=0, cache=None, slots=None) == OK


def attend(lib, q=AT[0], out=AT[1], lse=None, cache=AT[2], pages=8, page=16, Hk=2, ks=None, vs=None, table=AT[3],
           ld=4, blocks=4, lens=AT[4], starts=None, B=2, T=2, H=4, D=64, scale=0.1, ws=AT[6], size=1 << 30,
           dtype=BF16, qt=None, ot=None):
    return lib.rmsnorm_kv4_attention(q, H * D if qt is None else qt, D, out, H * D if ot is None else ot, D, lse,
                                     cache, pages, page, Hk, ks, vs, table, ld, blocks, lens, starts, B, T, H, D,
                                     scale, ws, size, dtype, None)


def test_attention_refusals(lib):  # noqa: F811
    assert attend(lib, dtype=F32) == BAD_DTYPE and attend(lib, dtype=4) == BAD_DTYPE
    assert attend(lib, T=3) == BAD_SHAPE                       # without starts a token each
    assert attend(lib, H=5) == BAD_SHAPE and attend(lib, Hk=0) == BAD_SHAPE and attend(lib, H=1) == BAD_SHAPE
    assert attend(lib, pages=-1) == BAD_SHAPE and attend(lib, blocks=-1) == BAD_SHAPE
    assert attend(lib, scale=NAN) == BAD_EPS
    assert attend(lib, D=96) == UNSUPPORTED and attend(lib, page=20) == UNSUPPORTED
    assert attend(lib, blocks=2 ** 27, ld=2 ** 27) == UNSUPPORTED
    assert attend(lib, page=1 << 24) == UNSUPPORTED            # a page of 2^31 bytes
    assert attend(lib, B=2 ** 21, T=2 ** 21) == UNSUPPORTED
    assert attend(lib, ld=3) == BAD_STRIDE and attend(lib, ot=255) == BAD_STRIDE and attend(lib, qt=-1) == BAD_STRIDE
    for a in ("q", "out", "cache", "table", "lens"):
        assert attend(lib, **{a: None}) == NULLPTR, a
    assert attend(lib, q=AT[0] + 1) == MISALIGNED and attend(lib, cache=AT[2] + 8) == MISALIGNED
    assert attend(lib, lens=AT[4] + 2) == MISALIGNED and attend(lib, ws=AT[6] + 4) == MISALIGNED
    assert attend(lib, out=AT[0]) == ALIAS and attend(lib, lse=AT[1]) == ALIAS and attend(lib, ws=AT[2]) == ALIAS
    assert attend(lib, out=AT[3]) == ALIAS and attend(lib, lse=AT[4]) == ALIAS


def test_structures_match_the_header():
    """The made-up calls above lay their structures out as the header does."""
    import re
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name, cls in (("rmsnorm_heads", Heads), ("rmsnorm_heads_grad", Grad), ("rmsnorm_rotation", Rotation)):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
        fields = [f.strip().lstrip("*").strip() for line in body.split(";") for f in
                  re.sub(r"^\s*(const\s+)?\w+\s", "", line.strip()).split(",") if f.strip()]
        assert fields == [f for f, _ in cls._fields_], name
    m = re.search(r"#define\s+RMSNORM_ROPE_MAX_D\s+(\d+)", text)
    assert int(m.group(1)) == rn.ROPE_MAX_D


def test_binding_refusals():
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    f, pos = torch.ones(32, dtype=torch.float64), torch.arange(3)
    with pytest.raises(ValueError, match="CUDA"):
        rn.rmsnorm_rope_fwd(q, pos, f)
    with pytest.raises(ValueError, match="3-D"):
        rn.rmsnorm_rope_fwd(q[0], pos, f)
    with pytest.raises(ValueError):
        rn.rmsnorm_rope_append(q, q, pos, f, pos, q, q, wq=q[0, 0])
    with pytest.raises(ValueError):
        rn.rmsnorm_rope_bwd(q, None, pos, f)
    with pytest.raises(ValueError):
        rn.rmsnorm_kv4_read(torch.zeros(1, 1, 1, 18 * 64, dtype=torch.uint8), pos)
    with pytest.raises(ValueError):
        rn.rmsnorm_kv4_attention(q, q, pos, pos)
    with pytest.raises(ValueError, match="multiple"):
        rn.kv4_cache(2, 2, 24, 64, device="cpu")
    with pytest.raises(ValueError, match="64 or 128"):
        rn.kv4_cache(2, 2, 32, 96, device="cpu")
    assert tuple(rn.kv4_cache(3, 2, 32, 128, device="cpu").shape) == (3, 2, 2, 2304)
    for bad in ({"rot": 3}, {"rot": 0}, {"rot": 4, "scaling": "other"}, {"rot": 4, "base": -1.0},
                {"rot": 4, "scaling": "yarn"}, {"rot": 4, "factor": 0.0}):
        with pytest.raises(ValueError):
            rn.rope_frequencies(device="cpu", **bad)


def test_scaled_frequencies():
    f, a = rn.rope_frequencies(8, 100.0, device="cpu")
    assert a == 1.0 and f.tolist() == [100.0 ** (-i / 4) for i in range(4)]
    g, _ = rn.rope_frequencies(8, 100.0, "linear", 4.0, device="cpu")
    assert torch.equal(g, f / 4)
    g, _ = rn.rope_frequencies(8, 100.0, "ntk", 4.0, device="cpu")
    assert g[0] == f[0] and abs(float(g[-1] / f[-1]) - 0.25) < 1e-12
    y, a = rn.rope_frequencies(128, 1e4, "yarn", 16.0, original=4096, device="cpu")
    p, _ = rn.rope_frequencies(128, 1e4, device="cpu")
    assert torch.equal(y[:20], p[:20]) and torch.allclose(y[-10:], p[-10:] / 16) and abs(a - 1.27725887222) < 1e-9
