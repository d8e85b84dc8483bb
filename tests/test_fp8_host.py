"""CPU tier: the 8-bit entry points reject bad arguments on the host before
any CUDA call, and the binding rejects what the library cannot see. The
argument checks pass made-up addresses; every call below fails a check (or
has nothing to do), so nothing is launched."""

import re

import pytest
import torch

from rmsnorm_fwd_bwd_02_gb300 import rmsnorm as rn
from tests.test_abi_host import (ALIAS, BAD_DTYPE, BAD_EPS, BAD_SHAPE, BAD_STRIDE, BF16, F32,
                                 HEADER, MISALIGNED, NAN, NULLPTR, OK, UNSUPPORTED, lib)  # noqa: F401

A, B, C, D, E, F = (0x7f0000000000 + (i << 36) for i in range(6))
E4M3, E5M2 = 0, 1
BAD_FLAGS = -11


def norm(lib, x=A, ldx=256, r=None, ldr=256, w=B, q=C, ldq=256, s=D, h=None, ldh=256, rstd=E,
         M=4, H=256, eps=1e-6, dtype=BF16, qtype=E4M3):
    return lib.rmsnorm_fwd_fp8(x, ldx, r, ldr, w, q, ldq, s, h, ldh, rstd, M, H, eps, dtype, qtype,
                               None)


def test_norm_refusals(lib):  # noqa: F811
    assert norm(lib, dtype=3) == BAD_DTYPE
    assert norm(lib, qtype=2) == BAD_DTYPE and norm(lib, qtype=-1) == BAD_DTYPE
    assert norm(lib, M=-1) == BAD_SHAPE and norm(lib, H=0) == BAD_SHAPE
    assert norm(lib, H=16385, ldx=16385, ldq=16385) == UNSUPPORTED
    for e in (NAN, -1.0, float("inf")):
        assert norm(lib, eps=e) == BAD_EPS
    assert norm(lib, ldx=255) == BAD_STRIDE and norm(lib, ldq=255) == BAD_STRIDE
    assert norm(lib, r=F, h=F + (1 << 30), ldr=255) == BAD_STRIDE
    assert norm(lib, r=F, h=F + (1 << 30), ldh=2 ** 31) == BAD_STRIDE
    for k in ("x", "w", "q", "s"):
        assert norm(lib, **{k: None}) == NULLPTR
    assert norm(lib, r=F) == NULLPTR and norm(lib, h=F) == NULLPTR
    assert norm(lib, x=A + 1) == MISALIGNED and norm(lib, s=D + 2) == MISALIGNED
    assert norm(lib, rstd=E + 2) == MISALIGNED and norm(lib, w=B + 1) == MISALIGNED
    assert norm(lib, q=A) == ALIAS and norm(lib, s=A + 256) == ALIAS
    assert norm(lib, q=B + 511) == ALIAS and norm(lib, rstd=C + 4) == ALIAS
    assert norm(lib, r=F, h=B) == ALIAS                       # h over the weight
    assert norm(lib, r=F, h=A + 512) == ALIAS                 # h one row into x
    assert norm(lib, r=F, h=C) == ALIAS                       # h over q
    assert norm(lib, x=None, w=None, q=None, s=None, rstd=None, M=0) == OK


def quant(lib, x=A, ldx=256, q=B, ldq=256, s=C, M=4, H=256, rows=1, dtype=BF16, qtype=E4M3):
    return lib.rmsnorm_quant_fp8(x, ldx, q, ldq, s, M, H, rows, dtype, qtype, None)


def test_quant_refusals(lib):  # noqa: F811
    assert quant(lib, dtype=9) == BAD_DTYPE and quant(lib, qtype=7) == BAD_DTYPE
    assert quant(lib, M=-1) == BAD_SHAPE and quant(lib, H=0) == BAD_SHAPE
    assert quant(lib, M=2 ** 62) == BAD_SHAPE
    for rows in (0, 2, 64, 256, -1):
        assert quant(lib, rows=rows) == UNSUPPORTED
    assert quant(lib, H=rn.FP8_MAX_K + 1, ldx=2 ** 30, ldq=2 ** 30) == UNSUPPORTED
    assert quant(lib, ldx=255) == BAD_STRIDE and quant(lib, ldq=2 ** 31) == BAD_STRIDE
    for k in ("x", "q", "s"):
        assert quant(lib, **{k: None}) == NULLPTR
    assert quant(lib, x=A + 1) == MISALIGNED and quant(lib, x=A + 2, dtype=F32) == MISALIGNED
    assert quant(lib, q=A) == ALIAS and quant(lib, s=B) == ALIAS
    assert quant(lib, x=None, q=None, s=None, M=0) == OK


def gemm(lib, a=A, lda=256, sa=B, at=E4M3, b=C, ldb=256, sb=D, bt=E4M3, out=E, ldo=128, M=4, N=128,
         K=256, dtype=BF16, flags=0):
    return lib.rmsnorm_gemm_fp8(a, lda, sa, at, b, ldb, sb, bt, out, ldo, M, N, K, dtype, flags, None)


def test_gemm_refusals(lib):  # noqa: F811
    assert gemm(lib, flags=2) == BAD_FLAGS
    assert gemm(lib, dtype=3) == BAD_DTYPE
    assert gemm(lib, at=2) == BAD_DTYPE and gemm(lib, bt=-1) == BAD_DTYPE
    assert gemm(lib, M=-1) == BAD_SHAPE and gemm(lib, N=0) == BAD_SHAPE and gemm(lib, K=0) == BAD_SHAPE
    assert gemm(lib, M=rn.FP8_MAX_ROWS + 1) == UNSUPPORTED
    assert gemm(lib, N=rn.FP8_MAX_ROWS + 1) == UNSUPPORTED
    assert gemm(lib, K=rn.FP8_MAX_K + 1) == UNSUPPORTED
    assert gemm(lib, lda=255) == BAD_STRIDE and gemm(lib, ldb=240) == BAD_STRIDE
    assert gemm(lib, ldo=127) == BAD_STRIDE and gemm(lib, lda=2 ** 31) == BAD_STRIDE
    for k in ("a", "sa", "b", "sb", "out"):
        assert gemm(lib, **{k: None}) == NULLPTR
    assert gemm(lib, a=A + 8) == MISALIGNED and gemm(lib, b=C + 1) == MISALIGNED
    assert gemm(lib, lda=264) == MISALIGNED and gemm(lib, ldb=257) == MISALIGNED
    assert gemm(lib, sa=B + 2) == MISALIGNED and gemm(lib, out=E + 1) == MISALIGNED
    assert gemm(lib, out=A) == ALIAS and gemm(lib, out=D) == ALIAS and gemm(lib, out=B) == ALIAS
    assert gemm(lib, out=C + 4096) == ALIAS
    assert gemm(lib, a=None, sa=None, b=None, sb=None, out=None, M=0) == OK


def test_constants_match_header():
    text = open(HEADER).read()
    for name, value in (("RMSNORM_FP8_MAX_K", rn.FP8_MAX_K),
                        ("RMSNORM_FP8_MAX_ROWS", rn.FP8_MAX_ROWS)):
        m = re.search(rf"#define\s+{name}\s+\(1 << (\d+)\)", text)
        assert m is not None and 1 << int(m.group(1)) == value
    m = re.search(r"#define\s+RMSNORM_GEMM_FP8_STATIC_WEIGHTS\s+(\d+)", text)
    assert m is not None and int(m.group(1)) == rn.GEMM_FP8_STATIC_WEIGHTS
    m = re.search(r"RMSNORM_E4M3\s*=\s*(\d+),\s*RMSNORM_E5M2\s*=\s*(\d+)", text)
    assert {torch.float8_e4m3fn: int(m.group(1)), torch.float8_e5m2: int(m.group(2))} == rn.FP8_TYPES


def test_binding_refuses_cpu_tensors_and_types():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.ones(256, dtype=torch.bfloat16)
    q = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(4, 2)
    with pytest.raises(ValueError):
        rn.rmsnorm_fwd_fp8(x, w)
    with pytest.raises(ValueError):
        rn.rmsnorm_quant_fp8(x)
    with pytest.raises(ValueError):
        rn.rmsnorm_quant_fp8(x[0])
    with pytest.raises(ValueError):
        rn.rmsnorm_gemm_fp8(q, s, q, s[:1])
    with pytest.raises(ValueError):
        rn.rmsnorm_gemm_fp8(x, s, q, s[:1])             # not an 8-bit type
    with pytest.raises(ValueError):
        rn.rmsnorm_gemm_fp8(q, s, q[:, :128], s[:1])    # two K


def test_gemm_refuses_more_tiles_than_a_grid_holds(lib):  # noqa: F811
    """ceil(M / 128) * ceil(N / 128) is below 2^31, whatever the addresses:
    the refusal comes before any of them is looked at (a null output says
    that the size itself was taken)."""
    m, n = 1 << 23, 1 << 22                                   # 2^16 and 2^15 tiles
    assert gemm(lib, M=m, N=n, ldo=n) == UNSUPPORTED
    assert gemm(lib, M=m - 128, N=n, ldo=n, out=None) == NULLPTR
    assert gemm(lib, M=m - 127, N=n, ldo=n, out=None) == UNSUPPORTED
    assert gemm(lib, M=m, N=n - 128, ldo=n, out=None) == NULLPTR
    assert gemm(lib, M=1 << 30, N=1 << 30, ldo=1 << 30) == UNSUPPORTED
