"""GPU tier: the 8-bit entry points (rmsnorm_fwd_fp8, rmsnorm_quant_fp8,
rmsnorm_gemm_fp8) against their definitions in 64 bits.

Tolerances, from the arithmetic. The norm's y, rstd and a group's largest
magnitude are computed in fp32 (a handful of roundings of 2^-24, rsqrtf
within 2 ulp, and a sum of squares whose lanes add at most 64 terms each
before a tree): DELTA = 1e-5 relative covers them. A q must be what rounding
y / scale gives for some y within DELTA of the exact one: rounding is
monotonic, so it lies between the roundings of the two ends. The product
accumulates 128 products and then G groups in fp32, each addition off by at
most 2^-22 of the terms' absolute sum T so far (one rounding is 2^-24; the
tensor cores may truncate): (128 + G) 2^-22 T, and half a step of the
output's type for the last rounding.
"""
import gc
import io

import pytest
import torch

from rmsnorm_fwd_bwd_02_gb300 import rmsnorm as rn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F64 = torch.float64
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
LARGEST = {E4M3: 448.0, E5M2: 57344.0}
BITS = {E4M3: (3, -6), E5M2: (2, -14)}       # fraction bits, least exponent
DELTA = 1e-5
AMAX_MIN = 2.0 ** -100


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tier needs a CUDA device")
    rn.lib()
    rn.set_path_override(rn.PATH_AUTO)
    rn.wait_timeouts(reset=True)
    yield
    assert rn.wait_timeouts(reset=True) == 0


# ------------------------------------------------------------------ oracle
def round8(v, to):
    """v (float64) to the nearest value of the format, ties to even."""
    bits, low = BITS[to]
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=low) - bits)
    return (torch.round(v / step) * step).clamp(-LARGEST[to], LARGEST[to])


def group_amax(y, rows):
    """Largest magnitude [ceil(M / rows), G] of y [M, H]."""
    M, H = y.shape
    p = torch.nn.functional.pad(y.abs(), (0, -H % 128, 0, -M % rows))
    return p.view(p.shape[0] // rows, rows, -1, 128).amax(dim=(1, 3))


def spread(s, rows, M, H):
    """Scales [R, G] as [M, H]."""
    return s.repeat_interleave(rows, 0)[:M].repeat_interleave(128, 1)[:, :H]


def check_q(q, scale, y, rows, to):
    """q, scale (GPU) against exact y [M, H] (float64, finite)."""
    M, H = y.shape
    assert q.dtype == to and tuple(q.shape) == (M, H)
    s = scale.cpu().to(F64)
    want = group_amax(y, rows).clamp(min=AMAX_MIN) / LARGEST[to]
    assert tuple(s.shape) == tuple(want.shape)
    assert bool(((s - want).abs() <= DELTA * want).all()), float(((s - want).abs() / want).max())
    v = y / spread(s, rows, M, H)
    got = q.float().cpu().to(F64)
    a, b = round8(v * (1 - DELTA), to), round8(v * (1 + DELTA), to)
    lo, hi = torch.minimum(a, b), torch.maximum(a, b)
    bad = (got < lo) | (got > hi)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist(),
                                 float(got[bad][0]), float(v[bad][0]))


def norm64(v, w, eps):
    v, w = v.to(F64), w.to(F64)
    rstd = 1.0 / torch.sqrt((v * v).mean(dim=1) + eps)
    return v * rstd[:, None] * w[None, :], rstd


def data(M, H, dtype, seed, outliers=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, H, generator=g)
    if outliers and M * H >= 1000:
        at = torch.randint(M * H, (M * H // 1000,), generator=g)
        x.view(-1)[at] *= 50.0
    r = torch.randn(M, H, generator=g) * 2
    w = 1 + 0.1 * torch.randn(H, generator=g)
    return x.to(dtype), r.to(dtype), w.to(dtype)


SHAPES = [(1, 1), (1, 7), (3, 31), (2, 64), (5, 127), (70, 128), (9, 129), (64, 256), (33, 384),
          (2, 511), (17, 512), (1, 896), (64, 896), (400, 896), (13, 1000), (7, 1001), (5, 2056),
          (320, 4096), (1, 4096), (6, 4100), (310, 5120), (2, 16384), (311, 16384), (3, 16381)]


@pytest.mark.parametrize("M,H", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(M, H, dtype, residual):
    x, r, w = data(M, H, dtype, seed=M * 7 + H)
    to = E5M2 if (M + H) % 3 == 0 else E4M3
    if residual:
        h, q, s, rstd = rn.rmsnorm_fwd_fp8(x.to(DEV), w.to(DEV), r=r.to(DEV), qdtype=to)
        v = (x.to(F64) + r.to(F64)).to(dtype)
        assert torch.equal(h.cpu(), v)
    else:
        q, s, rstd = rn.rmsnorm_fwd_fp8(x.to(DEV), w.to(DEV), qdtype=to)
        v = x
    assert rn.last_path() == rn.PATH_FP8_ROWS
    y, rs = norm64(v, w, 1e-6)
    assert bool(((rstd.cpu().to(F64) - rs).abs() <= DELTA * rs).all())
    check_q(q, s, y, 1, to)


@pytest.mark.parametrize("M,H", SHAPES + [(3, 16385), (2, 40000), (1, 32768)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows", [1, 128])
def test_quant(M, H, dtype, rows):
    x, _, _ = data(M, H, dtype, seed=M + 3 * H)
    to = E5M2 if (M + H) % 3 == 1 else E4M3
    q, s = rn.rmsnorm_quant_fp8(x.to(DEV), block_rows=rows, qdtype=to)
    assert rn.last_path() == (rn.PATH_FP8_ROWS if rows == 1 else rn.PATH_FP8_BLOCKS)
    check_q(q, s, x.to(F64), rows, to)


@pytest.mark.parametrize("rows", [1, 128])
def test_quant_tall(rows):
    """More blocks down than the grid's y holds is out of reach of a test; a
    tall narrow matrix takes many."""
    x, _, _ = data(40000, 130, BF16, seed=5)
    q, s = rn.rmsnorm_quant_fp8(x.to(DEV), block_rows=rows)
    check_q(q, s, x.to(F64), rows, E4M3)


@pytest.mark.parametrize("to", [E4M3, E5M2])
@pytest.mark.parametrize("rows", [1, 128])
def test_quant_every_magnitude(to, rows):
    """fp32 values over the whole range of exponents: tiny groups keep the
    least scale, the largest do not overflow, zeros stay zeros."""
    g = torch.Generator().manual_seed(3)
    e = torch.arange(-140, 127, dtype=torch.float32)
    x = torch.randn(e.numel(), 256, generator=g).clamp(-1.9, 1.9) * torch.exp2(e)[:, None].float()
    x[::7] = 0.0
    x[5, :128] = 0.0
    q, s = rn.rmsnorm_quant_fp8(x.to(DEV), block_rows=rows, qdtype=to)
    want = group_amax(x.to(F64), rows).clamp(min=AMAX_MIN) / LARGEST[to]
    assert bool(((s.cpu().to(F64) - want).abs() <= DELTA * want).all())
    check_q(q, s, x.to(F64), rows, to)
    assert bool((q.float()[5, :128] == 0).all())


def test_quant_is_exact_where_the_values_are():
    """Values of the format times a power of two whose group's largest is the
    format's largest come back bit for bit."""
    codes = torch.arange(256, dtype=torch.uint8)
    for to in (E4M3, E5M2):
        v = codes.view(to).float()
        v = v[torch.isfinite(v)]
        v = torch.cat([v, torch.full((-v.numel() % 128,), LARGEST[to])])
        x = v.view(-1, 128).clone()
        x[:, 0] = LARGEST[to]
        q, s = rn.rmsnorm_quant_fp8((x * 0.25).to(DEV), qdtype=to)
        assert bool((s == 0.25).all())
        assert torch.equal(q.float().cpu(), x)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("H", [384, 301])
def test_quant_of_nonfinite_groups(bad, rows, H):
    x, _, _ = data(130, H, BF16, seed=11)
    x[2, 130] = bad
    q, s = rn.rmsnorm_quant_fp8(x.to(DEV), block_rows=rows)
    s = s.cpu()
    hit = torch.zeros_like(s, dtype=torch.bool)
    hit[2 // rows, 1] = True
    assert torch.equal(torch.isnan(s), hit)
    wide = spread(hit, rows, 130, H)
    qf = q.float().cpu()
    assert bool(torch.isnan(qf[wide]).all()) and bool(torch.isfinite(qf[~wide]).all())


@pytest.mark.parametrize("H", [512, 1001])
def test_norm_of_nonfinite_rows(H):
    """A row with an infinity has rstd 0 (the infinity itself is NaN); a NaN
    takes the whole row. Other rows are untouched by either."""
    x, _, w = data(6, H, F32, seed=12)
    x[1, 5], x[3, 200] = float("inf"), float("nan")
    q, s, rstd = rn.rmsnorm_fwd_fp8(x.to(DEV), w.to(DEV))
    s, qf = s.cpu(), q.float().cpu()
    assert bool(torch.isnan(s[3]).all()) and bool(torch.isnan(qf[3]).all())
    assert bool(torch.isnan(s[1, 0])) and bool(torch.isnan(qf[1, :128]).all())
    assert bool((qf[1, 128:] == 0).all()) and bool(torch.isfinite(s[1, 1:]).all())
    ok = [0, 2, 4, 5]
    y, _ = norm64(x[ok], w, 1e-6)
    check_q(q[ok], s[ok], y, 1, E4M3)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,ld", [(128, 256), (4096, 4608), (896, 904), (1001, 1003)])
def test_strides_and_guards(dtype, H, ld):
    """Row windows of wider buffers, everything around them NaN or a guard
    that must survive; the results are those of dense tensors."""
    M = 37
    x, r, w = data(M, H, dtype, seed=21)

    def window(t):
        buf = torch.full((M, ld), float("nan"), device=DEV, dtype=dtype)
        buf[:, :H] = t.to(DEV)
        return buf, buf[:, :H]

    _, xs = window(x)
    _, rs = window(r)
    hb, hs = window(torch.zeros(M, H, dtype=dtype))
    qb = torch.full((M + 2, ld), 0x5A, device=DEV, dtype=torch.uint8)
    qs = qb[1:M + 1, :H].view(E4M3)
    h, q, s, _ = rn.rmsnorm_fwd_fp8(xs, w.to(DEV), r=rs, h=hs, q=qs)
    h0, q0, s0, _ = rn.rmsnorm_fwd_fp8(x.to(DEV), w.to(DEV), r=r.to(DEV))
    assert torch.equal(h, h0)
    y, _ = norm64(h0.cpu(), w, 1e-6)
    check_q(q, s, y, 1, E4M3)
    check_q(q0, s0, y, 1, E4M3)
    assert bool(torch.isnan(hb[:, H:]).all())
    assert bool((qb[0] == 0x5A).all()) and bool((qb[-1] == 0x5A).all())
    assert bool((qb[:, H:] == 0x5A).all())
    for rows in (1, 128):
        qb.fill_(0x5A)
        q, s = rn.rmsnorm_quant_fp8(xs, q=qs, block_rows=rows)
        check_q(q, s, x.to(F64), rows, E4M3)
        assert bool((qb[0] == 0x5A).all()) and bool((qb[-1] == 0x5A).all())
        assert bool((qb[:, H:] == 0x5A).all())


def test_norm_in_place_and_empty():
    x, r, w = data(40, 896, BF16, seed=31)
    xd, rd = x.to(DEV), r.to(DEV)
    h0, q0, s0, rs0 = rn.rmsnorm_fwd_fp8(xd, w.to(DEV), r=rd)
    h, q, s, rs = rn.rmsnorm_fwd_fp8(xd, w.to(DEV), r=rd, h=xd)
    assert h.data_ptr() == xd.data_ptr() and torch.equal(h, h0)
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s, s0)
    e = torch.empty(0, 896, device=DEV, dtype=BF16)
    q, s, _ = rn.rmsnorm_fwd_fp8(e, w.to(DEV))
    assert q.shape == (0, 896) and s.shape == (0, 7)
    q, s = rn.rmsnorm_quant_fp8(e)
    assert q.shape == (0, 896)
    out = rn.rmsnorm_gemm_fp8(q, s, q0, s0[:1])
    assert out.shape == (0, 40)


# ----------------------------------------------------------------- product
def pair(M, N, K, seed, at=E4M3, bt=E4M3):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn(M, K, generator=g)
    if M * K >= 1000:
        a.view(-1)[torch.randint(M * K, (M * K // 1000,), generator=g)] *= 50.0
    b = torch.randn(N, K, generator=g) * 0.02
    qa, sa = rn.rmsnorm_quant_fp8(a.to(BF16).to(DEV), qdtype=at)
    qb, sb = rn.rmsnorm_quant_fp8(b.to(BF16).to(DEV), block_rows=128, qdtype=bt)
    torch.cuda.synchronize()       # calls with static weights may follow
    return qa, sa, qb, sb


def gemm64(qa, sa, qb, sb):
    """(the product, the absolute sum of its terms), on the GPU in 64 bits."""
    M, K = qa.shape
    N = qb.shape[0]
    a = qa.float().to(F64) * spread(sa.to(F64), 1, M, K)
    b = qb.float().to(F64) * spread(sb.to(F64), 128, N, K)
    return a @ b.t(), a.abs() @ b.abs().t()


HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}     # eps / 2
TINY = {BF16: 0.0, F16: 2.0 ** -25, F32: 0.0}                  # half a subnormal step


def check_out(out, want, T, K, dtype):
    assert out.dtype == dtype and out.shape == want.shape
    err = (out.to(F64) - want).abs()
    bound = HALF[dtype] * want.abs() + (128 + -(-K // 128)) * 2.0 ** -22 * T * (1 + HALF[dtype]) \
        + TINY[dtype] + 1e-300
    bad = ~(err <= bound)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist(),
                                 float(out[bad][0]), float(want[bad][0]), float(bound[bad][0]))


GEMMS = [(1, 1, 1), (1, 128, 128), (1, 2048, 896), (2, 129, 127), (3, 7, 300), (8, 9728, 896),
         (15, 257, 129), (16, 128, 4096), (16, 6144, 4096), (17, 300, 512), (31, 1000, 1000),
         (32, 4096, 640), (33, 130, 1024), (64, 128, 16384), (64, 2048, 896), (63, 999, 5121),
         (65, 128, 128), (100, 1, 257), (128, 512, 512), (129, 129, 129), (200, 640, 1100),
         (256, 2048, 4096), (333, 1001, 5121), (511, 777, 64), (1024, 1024, 1024),
         (1030, 1500, 2000), (1, 200, 70000), (64, 200, 70000), (300, 260, 33000)]


@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm(M, N, K):
    i = GEMMS.index((M, N, K))
    at, bt = ((E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2))[i % 4]
    qa, sa, qb, sb = pair(M, N, K, seed=i, at=at, bt=bt)
    want, T = gemm64(qa, sa, qb, sb)
    first = None
    for dtype in (BF16, F16, F32):
        for static in (False, True):
            out = rn.rmsnorm_gemm_fp8(qa, sa, qb, sb, out_dtype=dtype, static_weights=static)
            assert rn.last_path() >= rn.PATH_FP8_GEMM
            check_out(out, want, T, K, dtype)
            if dtype == F32:
                first = out if first is None else first
                assert torch.equal(first, out)            # the same bits every time


class forced:
    """One kernel of the product for the calls inside."""

    def __init__(self, path):
        self.path = path

    def __enter__(self):
        rn.set_gemm_fp8_test(self.path)

    def __exit__(self, *a):
        rn.set_gemm_fp8_test(0)


PAIRS = [(1, 1, 1), (255, 130, 127), (256, 256, 128), (257, 257, 900), (300, 1000, 1000),
         (2100, 2600, 700), (600, 8000, 130), (20000, 200, 300), (260, 9800, 384),
         (4096, 4096, 4096), (513, 40000, 256)]


@pytest.mark.parametrize("M,N,K", PAIRS)
@pytest.mark.parametrize("path", [rn.PATH_FP8_PAIR, rn.PATH_FP8_GEMM])
def test_gemm_many_rows(M, N, K, path):
    """Both kernels at sizes of many tiles (several a CTA, the last ones
    ragged) and of less than one."""
    i = PAIRS.index((M, N, K))
    at, bt = ((E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2))[i % 4]
    qa, sa, qb, sb = pair(M, N, K, seed=i, at=at, bt=bt)
    want, T = gemm64(qa, sa, qb, sb)
    for dtype in (BF16, F16, F32):
        with forced(path):
            out = rn.rmsnorm_gemm_fp8(qa, sa, qb, sb, out_dtype=dtype)
            again = rn.rmsnorm_gemm_fp8(qa, sa, qb, sb, out_dtype=dtype, static_weights=True)
            assert rn.last_path() == path
        check_out(out, want, T, K, dtype)
        assert torch.equal(out, again)


def test_gemm_takes_pairs_by_size():
    qa, sa, qb, sb = pair(2560, 2560, 256, seed=3)
    rn.rmsnorm_gemm_fp8(qa, sa, qb, sb)
    assert rn.last_path() == rn.PATH_FP8_PAIR
    rn.rmsnorm_gemm_fp8(qa[:64], sa[:64], qb, sb)
    assert rn.last_path() == rn.PATH_FP8_GEMM


@pytest.mark.parametrize("M,N,K", [(1, 130, 1000), (20, 300, 130), (64, 200, 257), (90, 100, 300),
                                   (300, 515, 1000), (600, 1030, 2050)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gemm_reads_and_writes_only_its_rows(M, N, K, dtype):
    """Operands inside larger buffers of NaN bytes, and scales of NaN behind
    the last row: nothing outside [M, K] and [N, K] is read into the result,
    nothing outside [M, N] is written."""
    qa, sa, qb, sb = pair(M, N, K, seed=M)
    ldk = -(-K // 16) * 16 + 32

    def inside(q, s):
        rows = q.shape[0]
        big = torch.full((rows + 200, ldk), 0x7F, device=DEV, dtype=torch.uint8)
        v = big[64:64 + rows, 16:16 + K]
        v.copy_(q.view(torch.uint8))
        bs = torch.full((s.shape[0] + 64, s.shape[1]), float("nan"), device=DEV)
        bs[32:32 + s.shape[0]] = s
        return v.view(E4M3), bs[32:32 + s.shape[0]]

    a, asc = inside(qa, sa)
    b, bsc = inside(qb, sb)
    outs = ((N, 0), (N + 5, 0), (-(-N // 16) * 16 + 16, 0), (N + 3, 1))
    for (ldo, off), path in [(o, p) for o in outs for p in (rn.PATH_FP8_GEMM, rn.PATH_FP8_PAIR)]:
        buf = torch.full((M + 3, ldo), -77.0, device=DEV, dtype=dtype)
        out = buf[1:M + 1, off:off + N]
        with forced(path):
            rn.rmsnorm_gemm_fp8(a, asc, b, bsc, out=out)
        want, T = gemm64(qa, sa, qb, sb)
        check_out(out, want, T, K, dtype)
        buf[1:M + 1, off:off + N] = -77.0
        assert bool((buf == -77.0).all())


def test_gemm_scales_of_every_size():
    """Zero rows, rows and blocks of very large and very small scales, and a
    NaN scale that stays in its row or its columns."""
    for M in (5, 200, 700):
        qa, sa, qb, sb = pair(M, 400, 640, seed=9)
        sa[1] = 0.0
        sa[2, 1], sa[3] = 1e30, 1e-30
        sb[1] *= 1e-6
        out = rn.rmsnorm_gemm_fp8(qa, sa, qb, sb, out_dtype=F32)
        want, T = gemm64(qa, sa, qb, sb)
        check_out(out, want, T, 640, F32)
        assert bool((out[1] == 0).all())
        sa[4, 2] = float("nan")
        out2 = rn.rmsnorm_gemm_fp8(qa, sa, qb, sb, out_dtype=F32)
        assert bool(torch.isnan(out2[4]).all())
        keep = [i for i in range(M) if i != 4]
        assert torch.equal(out2[keep], out[keep])
        sb[3, 0] = float("nan")
        out3 = rn.rmsnorm_gemm_fp8(qa, sa, qb, sb, out_dtype=F32)
        assert bool(torch.isnan(out3[:, 384:]).all())
        assert torch.equal(out3[keep][:, :384], out[keep][:, :384])


@pytest.mark.parametrize("M", [1, 16, 64, 100, 700])
def test_rows_do_not_depend_on_one_another(M):
    """A row's result is that of its own call (the tokens of a batch share
    nothing but the weight), to the tolerance of another kernel's order."""
    qa, sa, qb, sb = pair(M, 384, 1024, seed=40)
    out = rn.rmsnorm_gemm_fp8(qa, sa, qb, sb, out_dtype=F32)
    for i in {0, M // 2, M - 1}:
        one = rn.rmsnorm_gemm_fp8(qa[i:i + 1], sa[i:i + 1], qb, sb, out_dtype=F32)
        want, T = gemm64(qa[i:i + 1], sa[i:i + 1], qb, sb)
        check_out(one, want, T, 1024, F32)
        check_out(out[i:i + 1], want, T, 1024, F32)


# ---------------------------------------------------------- used together
def layer(x, r, w, W, sW, W2, sW2, static):
    """The norm of a residual sum, its projection, and a second projection of
    that projection's output quantised on its own."""
    h, q, s, _ = rn.rmsnorm_fwd_fp8(x, w, r=r, want_rstd=False)
    z = rn.rmsnorm_gemm_fp8(q, s, W, sW, static_weights=static)
    qz, sz = rn.rmsnorm_quant_fp8(z)
    return h, q, s, z, qz, sz, rn.rmsnorm_gemm_fp8(qz, sz, W2, sW2, static_weights=static)


def check_layer(x, r, w, W, sW, W2, sW2, res):
    h, q, s, z, qz, sz, o = res
    v = (x.cpu().to(F64) + r.cpu().to(F64)).to(x.dtype)
    assert torch.equal(h.cpu(), v)
    y, _ = norm64(v, w.cpu(), 1e-6)
    check_q(q, s, y, 1, E4M3)
    check_out(z, *gemm64(q, s, W, sW), q.shape[1], BF16)
    check_q(qz, sz, z.cpu().to(F64), 1, E4M3)
    check_out(o, *gemm64(qz, sz, W2, sW2), qz.shape[1], BF16)


def layer_inputs(M, seed, H=896, N=2432):
    x, r, w = data(M, H, BF16, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    W, sW = rn.rmsnorm_quant_fp8((torch.randn(N, H, generator=g) * 0.02).to(BF16).to(DEV),
                                 block_rows=128)
    W2, sW2 = rn.rmsnorm_quant_fp8((torch.randn(H, N, generator=g) * 0.02).to(BF16).to(DEV),
                                   block_rows=128)
    return x.to(DEV), r.to(DEV), w.to(DEV), W, sW, W2, sW2


@pytest.mark.parametrize("M", [1, 16, 40, 64, 130, 700])
@pytest.mark.parametrize("static", [False, True])
def test_chain(M, static):
    """Back to back, so that each call starts while the one before it ends;
    every iteration has inputs of its own."""
    x, r, w, W, sW, W2, sW2 = layer_inputs(M, seed=50)
    torch.cuda.synchronize()
    xs = [torch.roll(x, i, 0) * (1 + i) for i in range(6)]
    torch.cuda.synchronize()
    res = [layer(xi, r, w, W, sW, W2, sW2, static) for xi in xs]
    torch.cuda.synchronize()
    for xi, ri in zip(xs, res):
        check_layer(xi, r, w, W, sW, W2, sW2, ri)


@pytest.mark.parametrize("M", [1, 24, 300])
def test_chain_in_a_graph(M):
    """Captured once, replayed on new inputs in place; two captured graphs
    do not share anything that a replay of one could spoil for the other."""
    x, r, w, W, sW, W2, sW2 = layer_inputs(M, seed=60)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, r, w, W, sW, W2, sW2, True)
    torch.cuda.current_stream().wait_stream(side)
    x2 = x.clone()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        res1 = layer(x, r, w, W, sW, W2, sW2, True)
    with torch.cuda.graph(g2):
        res2 = layer(x2, r, w, W, sW, W2, sW2, False)
    for i in range(3):
        x.copy_(torch.roll(x2, i + 1, 1) * 3)
        x2.mul_(0.5)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        for st in (s1, s2):
            st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        torch.cuda.synchronize()
        check_layer(x, r, w, W, sW, W2, sW2, res1)
        check_layer(x2, r, w, W, sW, W2, sW2, res2)


def test_two_streams_at_once():
    ins = [layer_inputs(M, seed=70 + M) for M in (1, 64, 200, 16)]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    out = [[] for _ in ins]
    for _ in range(5):
        for k, (args, st) in enumerate(zip(ins, streams)):
            with torch.cuda.stream(st):
                out[k].append(layer(*args, True))
    torch.cuda.synchronize()
    for args, res in zip(ins, out):
        check_layer(*args, res[0])
        for other in res[1:]:
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                       for a, b in zip(res[0], other))


def test_stream_argument():
    """What the call allocates belongs to the stream it is given."""
    x, r, w, W, sW, W2, sW2 = layer_inputs(20, seed=80)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    h, q, s, _ = rn.rmsnorm_fwd_fp8(x, w, r=r, stream=st)
    z = rn.rmsnorm_gemm_fp8(q, s, W, sW, stream=st)
    qz, sz = rn.rmsnorm_quant_fp8(z, stream=st)
    o = rn.rmsnorm_gemm_fp8(qz, sz, W2, sW2, stream=st)
    st.synchronize()
    check_layer(x, r, w, W, sW, W2, sW2, (h, q, s, z, qz, sz, o))


def test_backward_takes_what_the_forward_returns():
    """rstd and h of the 8-bit forward are those of the library's forward, so
    its backward runs on them."""
    x, r, w = (t.to(DEV) for t in data(300, 896, BF16, seed=90))
    h, _, _, rstd = rn.rmsnorm_fwd_fp8(x, w, r=r)
    h0, _, rstd0 = rn.rmsnorm_residual_fwd(x, r, w)
    assert torch.equal(h, h0)
    assert bool(((rstd - rstd0).abs() <= DELTA * rstd0).all())
    dy = torch.randn(300, 896, device=DEV, dtype=F32).to(BF16)
    dx, dw = rn.rmsnorm_residual_bwd(dy, None, h, w, rstd)
    dx0, dw0 = rn.rmsnorm_residual_bwd(dy, None, h0, w, rstd0)
    assert bool(((dx.float() - dx0.float()).abs() <= 2.0 ** -7 * dx0.float().abs() + 1e-4).all())
    assert bool(((dw - dw0).abs() <= 1e-4 * (dw0.abs() + 1)).all())


# ---------------------------------------------------- offsets past 32 bits
def test_rows_past_32_bits():
    """2.3e9 elements in and out: the last rows are those of their own call."""
    M, H = 140000, 16384
    x = torch.zeros(M, H, device=DEV, dtype=BF16)
    tail, _, w = data(70, H, BF16, seed=100)
    x[-70:] = tail.to(DEV)
    q, s, _ = rn.rmsnorm_fwd_fp8(x, w.to(DEV))
    y, _ = norm64(tail, w, 1e-6)
    check_q(q[-70:], s[-70:], y, 1, E4M3)
    assert bool((q[:M - 70].view(torch.uint8)[::997] == 0).all())
    for rows in (1, 128):
        q, s = rn.rmsnorm_quant_fp8(x, q=q, block_rows=rows)
        R = 70 if rows == 1 else 1              # 140000 = 1093 blocks and 96 rows
        got = q[-70:].float().cpu().to(F64)
        want = tail.to(F64) / spread(s[-R:].cpu().to(F64), rows, 70, H)
        a, b = round8(want * (1 - DELTA), E4M3), round8(want * (1 + DELTA), E4M3)
        assert bool(((got >= torch.minimum(a, b)) & (got <= torch.maximum(a, b))).all())


@pytest.mark.parametrize("path", [rn.PATH_FP8_GEMM, rn.PATH_FP8_PAIR])
def test_gemm_past_32_bits(path):
    """An operand and an output of more than 2^31 elements."""
    M, N, K = 70000, 32768, 128
    qa, sa, qb, sb = pair(600, 700, K, seed=101)
    a = torch.zeros(M, K, device=DEV, dtype=torch.uint8).view(E4M3)
    asc = torch.ones(M, 1, device=DEV)
    a.view(torch.uint8)[-600:], asc[-600:] = qa.view(torch.uint8), sa
    b = torch.zeros(N, K, device=DEV, dtype=torch.uint8).view(E4M3)
    bsc = torch.ones(N // 128, 1, device=DEV)
    b.view(torch.uint8)[-640:], bsc[-5:] = qb.view(torch.uint8)[:640], sb[:5]
    torch.cuda.synchronize()
    with forced(path):
        out = rn.rmsnorm_gemm_fp8(a, asc, b, bsc)
    want, T = gemm64(qa, sa, qb[:640], sb[:5])
    check_out(out[-600:, -640:], want, T, K, BF16)
    assert bool((out[-600:, :-640] == 0).all()) and bool((out[:-600] == 0).all())
    del out
    M, N, K = 140000, 130, 16384                # A of 2.3e9 bytes
    a = torch.zeros(M, K, device=DEV, dtype=torch.uint8).view(E4M3)
    qa, sa, qb, sb = pair(300, N, K, seed=102)
    asc = torch.ones(M, K // 128, device=DEV)
    a.view(torch.uint8)[-300:], asc[-300:] = qa.view(torch.uint8), sa
    torch.cuda.synchronize()
    with forced(path):
        out = rn.rmsnorm_gemm_fp8(a, asc, qb, sb)
    check_out(out[-300:], *gemm64(qa, sa, qb, sb), K, BF16)
    assert bool((out[:-300] == 0).all())


def test_first_call_of_a_shape_inside_a_capture():
    """Sizes that no call had before: what the library looks up for them it
    may look up while a stream is being captured."""
    x, r, w, W, sW, W2, sW2 = layer_inputs(11, seed=110, H=1280, N=1152)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = layer(x, r, w, W, sW, W2, sW2, True)
    g.replay()
    torch.cuda.synchronize()
    check_layer(x, r, w, W, sW, W2, sW2, res)


# ---------------------------------------------------------------- refusals
def test_refusals_of_the_binding():
    x, r, w, W, sW, W2, sW2 = layer_inputs(4, seed=95)
    q, s = rn.rmsnorm_quant_fp8(x)
    for call in (lambda: rn.rmsnorm_fwd_fp8(x, w, qdtype=torch.float16),
                 lambda: rn.rmsnorm_fwd_fp8(x, w.float()),
                 lambda: rn.rmsnorm_fwd_fp8(x.t(), w),
                 lambda: rn.rmsnorm_fwd_fp8(x, w, r=r[:3]),
                 lambda: rn.rmsnorm_fwd_fp8(x, w, h=r),
                 lambda: rn.rmsnorm_fwd_fp8(x, w, scale=s[:, :6]),
                 lambda: rn.rmsnorm_fwd_fp8(x, w, q=q[:3]),
                 lambda: rn.rmsnorm_fwd_fp8(x, w, q=q, qdtype=E5M2),
                 lambda: rn.rmsnorm_fwd_fp8(x, w.cpu()),
                 lambda: rn.rmsnorm_quant_fp8(x, block_rows=64),
                 lambda: rn.rmsnorm_quant_fp8(x.long()),
                 lambda: rn.rmsnorm_gemm_fp8(q, s, W, sW.t().contiguous()),
                 lambda: rn.rmsnorm_gemm_fp8(q, s, W, sW[:-1]),
                 lambda: rn.rmsnorm_gemm_fp8(q, s.half(), W, sW),
                 lambda: rn.rmsnorm_gemm_fp8(q, s, W, sW, out=x),
                 lambda: rn.rmsnorm_gemm_fp8(x, s, W, sW),
                 lambda: rn.rmsnorm_gemm_fp8(q, s, W, sW, out_dtype=torch.int32)):
        with pytest.raises(ValueError):
            call()
    odd = torch.zeros(4, 1001, device=DEV, dtype=torch.uint8).view(E4M3)
    so = torch.ones(4, 8, device=DEV)
    with pytest.raises(rn.RmsNormError) as e:      # rows that start at odd addresses
        rn.rmsnorm_gemm_fp8(odd, so, odd, so[:1])
    assert e.value.status == -5
    with pytest.raises(rn.RmsNormError) as e:      # q over the residual
        rn.rmsnorm_fwd_fp8(x, w, r=r, q=r.view(torch.uint8)[:, :896].view(E4M3))
    assert e.value.status == -9


@pytest.mark.parametrize("M,path", [(8, 0), (100, 0), (700, 0), (700, rn.PATH_FP8_PAIR)])
def test_bounded_waits(M, path):
    """A copy that never completes ends the kernel, is counted, and leaves
    the context usable."""
    qa, sa, qb, sb = pair(M, 300, 1024, seed=97)
    with forced(path):
        good = rn.rmsnorm_gemm_fp8(qa, sa, qb, sb)
        torch.cuda.synchronize()
        assert rn.wait_timeouts(reset=True) == 0
        try:
            rn.set_stream_test_fault(16, 2000)
            rn.rmsnorm_gemm_fp8(qa, sa, qb, sb)
            torch.cuda.synchronize()
        finally:
            rn.set_stream_test_fault(0, 0)
        assert rn.wait_timeouts(reset=True) > 0
        assert torch.equal(rn.rmsnorm_gemm_fp8(qa, sa, qb, sb), good)


@pytest.mark.parametrize("M,H", [(1, 1), (1, 896), (3, 130), (7, 1001), (16, 4096), (300, 896)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_new_outputs(M, H, dtype):
    """Outputs that the call allocates: shapes, strides and devices as torch
    makes them, apart in memory; one allocation for small calls, one each for
    larger, and all of it free again with the last of them."""
    x = torch.randn(M, H, device=DEV, dtype=dtype)
    w = torch.ones(H, device=DEV, dtype=dtype)
    gc.collect()                                    # what other tests left in cycles
    before = torch.cuda.memory_allocated()
    h, q, scale, rstd = rn.rmsnorm_fwd_fp8(x, w, r=x)
    G, pitch = -(-H // 128), -(-H // 16) * 16
    assert h.shape == (M, H) and h.dtype == dtype and h.is_contiguous()
    assert q.shape == (M, H) and q.dtype == E4M3 and q.stride() == (pitch, 1)
    assert scale.shape == (M, G) and scale.dtype == F32 and scale.is_contiguous()
    assert rstd.shape == (M,) and rstd.dtype == F32 and rstd.is_contiguous()
    outs = (h, q, scale, rstd)
    spans = sorted((t.data_ptr(), t.data_ptr() + ((t.size(0) - 1) * t.stride(0) + t[0].numel())
                    * t.element_size()) for t in outs)
    for (_, end), (start, _) in zip(spans, spans[1:]):
        assert end <= start
    for t in outs:
        assert t.device == DEV and not t.requires_grad and t.data_ptr() % 256 == 0
        storage = t.untyped_storage()
        last = t.data_ptr() - storage.data_ptr() + ((M - 1) * t.stride(0) + t[0].numel()) * t.element_size()
        assert last <= storage.nbytes()
    size = sum(-(-t.size(0) * t.stride(0) * t.element_size() // 256) * 256 for t in outs)
    storages = {t.untyped_storage().data_ptr() for t in outs}
    assert len(storages) == (1 if size <= 256 * 1024 else 4)
    assert torch.equal(h, (x.float() + x.float()).to(dtype))
    # one output alone keeps its values when the others are gone and their
    # memory may be used again
    want = scale.clone()
    del h, q, rstd, outs, t, storage
    rn.rmsnorm_fwd_fp8(x * 2, w, r=x)
    assert torch.equal(scale, want)
    del scale, want
    assert torch.cuda.memory_allocated() == before


# ------------------------------------------------ the paired kernel's output
@pytest.mark.parametrize("N", [1001, 1043, 1045, 1055, 1071, 2077])
@pytest.mark.parametrize("K", [128, 1024])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_pairs_into_a_padded_output(N, K, dtype):
    """out inside a buffer whose rows start at multiples of 16 bytes while N
    ends inside 16 bytes: a warp then writes some of its passes by tensor
    copies and some element by element, from the same two slots of shared
    memory in turn. N mod 64 is 17 to 47, so that an element-wise pass follows
    a copy; several tiles a pair, called again and again."""
    assert 16 < N % 64 < 48
    M = 4 * 76 * 256 // -(-N // 256)                    # some four tiles a pair
    qa, sa, qb, sb = pair(M, N, K, seed=N + K)
    want, T = gemm64(qa, sa, qb, sb)
    ldo = -(-N // 8) * 8 + 8
    buf = torch.full((M + 2, ldo), -77.0, device=DEV, dtype=dtype)
    out = buf[1:M + 1, :N]
    assert out.data_ptr() % 16 == 0
    for _ in range(5):
        buf[1:M + 1, :N] = float("nan")
        with forced(rn.PATH_FP8_PAIR):
            rn.rmsnorm_gemm_fp8(qa, sa, qb, sb, out=out)
            assert rn.last_path() == rn.PATH_FP8_PAIR
        check_out(out, want, T, K, dtype)
    assert bool((buf[1:M + 1, N:] == -77.0).all())
    assert bool((buf[0] == -77.0).all()) and bool((buf[M + 1] == -77.0).all())


@pytest.mark.parametrize("M", [1, 17, 64, 128])
@pytest.mark.parametrize("N,K", [(256, 128), (300, 2048), (5000, 640)])
def test_tensor_memory_is_free_after_a_timeout(M, N, K):
    """The tile kernel of every width, alone and in clusters, gives up on
    copies that never complete, again and again; each time all of its tensor
    memory is free for the paired kernel, which takes all columns of an SM."""
    qa, sa, qb, sb = pair(M, N, K, seed=98)
    qc, sc, qd, sd = pair(2100, 2600, 256, seed=99)
    good, many = rn.rmsnorm_gemm_fp8(qa, sa, qb, sb), rn.rmsnorm_gemm_fp8(qc, sc, qd, sd)
    assert rn.last_path() == rn.PATH_FP8_PAIR
    torch.cuda.synchronize()
    assert rn.wait_timeouts(reset=True) == 0
    for _ in range(4):
        try:
            rn.set_stream_test_fault(16, 1000)
            rn.rmsnorm_gemm_fp8(qa, sa, qb, sb)
            assert rn.last_path() == rn.PATH_FP8_GEMM
            torch.cuda.synchronize()
        finally:
            rn.set_stream_test_fault(0, 0)
        assert rn.wait_timeouts(reset=True) > 0
        assert torch.equal(rn.rmsnorm_gemm_fp8(qc, sc, qd, sd), many)
        assert torch.equal(rn.rmsnorm_gemm_fp8(qa, sa, qb, sb), good)
    torch.cuda.synchronize()
    assert rn.wait_timeouts() == 0


# ------------------------------------------------------- scales bit for bit
@pytest.mark.parametrize("M,H", [(130, 1001), (300, 4096), (2, 16384), (257, 130)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("to", [E4M3, E5M2])
@pytest.mark.parametrize("rows", [1, 128])
def test_scales_are_the_rounded_quotient(M, H, dtype, to, rows):
    """scale = max / F rounded once to fp32: the bits of a division. q is the
    quotient by it, formed to within 2^-22 (the reciprocal is off by 2^-23 at
    most, the product by 2^-24), rounded to nearest even."""
    x, _, _ = data(M, H, dtype, seed=M + H)
    if dtype == F32:                              # every binade that has a scale of its own
        e = torch.arange(M, dtype=F32) * (220.0 / M) - 99
        x = x.clamp(-60, 60) * torch.exp2(e.round())[:, None]
    q, s = rn.rmsnorm_quant_fp8(x.to(DEV), block_rows=rows, qdtype=to)
    amax = group_amax(x.to(F64), rows).clamp(min=AMAX_MIN).to(F32)      # exact in fp32
    want = amax / torch.tensor(LARGEST[to], dtype=F32)
    assert torch.equal(s.cpu(), want)
    v = x.to(F64) / spread(want.to(F64), rows, M, H)
    a, b = round8(v * (1 - 2.0 ** -22), to), round8(v * (1 + 2.0 ** -22), to)
    got = q.float().cpu().to(F64)
    assert bool(((got >= torch.minimum(a, b)) & (got <= torch.maximum(a, b))).all())


@pytest.mark.parametrize("M,path", [(5, 0), (60, 0), (200, 0), (700, rn.PATH_FP8_PAIR)])
def test_products_of_scales_at_the_edges_of_their_range(M, path):
    """Two scales may lie anywhere as long as their product is zero or a
    normal number: at 2^-126 the terms are exact to fp32's precision, at 2^127
    a group whose sum is zero adds zero. Past the range it is NaN, and only
    in the row and the columns that meet there."""
    qa, sa, qb, sb = pair(M, 400, 640, seed=96)
    sa[0], sb[0] = 2.0 ** -100, 2.0 ** -26            # 2^-126 together
    sa[1], sb[1] = 2.0 ** 100, 2.0 ** 27              # 2^127, of zeros
    qa.view(torch.uint8)[1] = 0
    sa[2] = 0.0
    sb[2] *= 2.0 ** -20
    sa[3] = 1.3 * 2.0 ** -116                         # below 2^-126 with all blocks but one
    with forced(path):
        out = rn.rmsnorm_gemm_fp8(qa, sa, qb, sb, out_dtype=F32)
        want, T = gemm64(qa, sa, qb, sb)
        rows = [i for i in range(M) if i != 3]
        check_out(out[rows], want[rows], T[rows], 640, F32)
        # row 3: below 2^-126 a product of scales is a multiple of 2^-149, off by
        # 2^-150 at most, which its group's sum (of terms T0 together, over the
        # groups) multiplies; each of the five additions is off by 2^-150 more
        _, T0 = gemm64(qa, torch.ones_like(sa), qb, torch.ones_like(sb))
        bound = (128 + 5) * 2.0 ** -22 * T[3] + 2.0 ** -150 * (T0[3] + 5)
        assert bool(((out[3].to(F64) - want[3]).abs() <= bound).all())
        assert bool((out[1] == 0).all()) and bool((out[2] == 0).all())
        sa[1, 2] = 2.0 ** 101
        far = rn.rmsnorm_gemm_fp8(qa, sa, qb, sb, out_dtype=F32)
    assert bool(torch.isnan(far[1, 128:256]).all())
    keep = [i for i in range(M) if i != 1]
    assert torch.equal(far[keep], out[keep])
    assert torch.equal(far[:, :128], out[:, :128]) and torch.equal(far[:, 256:], out[:, 256:])


@pytest.mark.parametrize("H", [1, 3])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_blocks_down_than_the_grid_holds(H, dtype):
    """65537 blocks of 128 rows on 65535 CTAs: the first two CTAs take a second
    block, with the shared sums of the first. Every block is checked."""
    M = 65535 * 128 + 130
    g = torch.Generator(device=DEV).manual_seed(120)
    x = torch.randn(M, H, generator=g, device=DEV)
    x *= torch.exp2(torch.arange(M, device=DEV) // 128 % 7 - 3.0)[:, None]
    x = x.to(dtype)
    q, s = rn.rmsnorm_quant_fp8(x, block_rows=128)
    assert rn.last_path() == rn.PATH_FP8_BLOCKS and s.shape == (65537, 1)
    amax = torch.nn.functional.pad(x.float().abs(), (0, 0, 0, -M % 128)).view(65537, -1).amax(dim=1)
    want = amax / torch.tensor(LARGEST[E4M3], dtype=F32, device=DEV)
    assert torch.equal(s[:, 0], want)
    v = (x.to(F64) / want.to(F64).repeat_interleave(128)[:M, None]).cpu()
    a, b = round8(v * (1 - 2.0 ** -22), E4M3), round8(v * (1 + 2.0 ** -22), E4M3)
    got = q.float().cpu().to(F64)
    assert bool(((got >= torch.minimum(a, b)) & (got <= torch.maximum(a, b))).all())


@pytest.mark.parametrize("M,H", [(1, 128), (128, 896), (200, 1001), (4096, 896)])
@pytest.mark.parametrize("rows", [1, 128])
def test_quantised_weights_can_be_saved(M, H, rows):
    """A checkpoint of quantised weights: each output has a storage of its
    own, which holds nothing else, and comes back from torch.save as it was."""
    x, _, _ = data(M, H, BF16, seed=130)
    q, s = rn.rmsnorm_quant_fp8(x.to(DEV), block_rows=rows)
    assert q.untyped_storage().data_ptr() != s.untyped_storage().data_ptr()
    file = io.BytesIO()
    torch.save({"weight": q, "scale": s}, file)
    file.seek(0)
    back = torch.load(file, weights_only=True)
    assert torch.equal(back["scale"], s) and back["weight"].dtype == q.dtype
    assert torch.equal(back["weight"].view(torch.uint8), q.view(torch.uint8))
    keep = q.view(torch.uint8).clone()
    del s, back
    rn.rmsnorm_quant_fp8(x.to(DEV) * 2, block_rows=rows)
    assert torch.equal(q.view(torch.uint8), keep)


def test_small_outputs_of_the_norm_are_saved_as_clones():
    x, r, w = (t.to(DEV) for t in data(8, 896, BF16, seed=131))
    outs = rn.rmsnorm_fwd_fp8(x, w, r=r)
    file = io.BytesIO()
    torch.save([t.clone() for t in outs], file)
    file.seek(0)
    for a, b in zip(outs, torch.load(file, weights_only=True)):
        assert a.dtype == b.dtype and torch.equal(a.contiguous().view(torch.uint8),
                                                  b.contiguous().view(torch.uint8))
