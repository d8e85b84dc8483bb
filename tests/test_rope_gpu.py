"""GPU tier: the rotation of heads, its backward and the append to a cache
against their definitions in 64 bits.

Tolerances, from the arithmetic. Forward: the norm's sum of D <= 256 squares
(a lane adds at most 16 terms, then a tree of 5: 21 roundings, half of them in
rstd), rsqrtf within 2 ulp, two products, sine and cosine within 3e-9 and two
roundings, the amplitude, two products and a sum: fewer than 24 roundings of
2^-24 of |a| + |b|, the pair's magnitudes: FWD = 24 * 2^-24, and half a step of
the output's type. Backward: dx is a difference of two terms, each within as
many roundings again of its own magnitude: 64 * 2^-24 of the terms' sum. dw: a
lane adds its rows one after another (at most R of them), then a tree over the
groups and the CTAs: (R + 64) 2^-24 of the sum of magnitudes.
"""
import math
from fractions import Fraction

import pytest
import torch

from rmsnorm_fwd_bwd_02_gb300 import autograd
from rmsnorm_fwd_bwd_02_gb300 import rmsnorm as rn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F64 = torch.float64
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ULP = 2.0 ** -24
TINY = {BF16: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -149}     # half the least step
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tier needs a CUDA device")
    rn.lib()


# ------------------------------------------------------------------ oracle
def turn(x, positions, freq, adjacent, amplitude=1.0, back=False):
    """x [T, H, D] float64 turned; also |a| + |b| of each element's pair."""
    rot = 2 * freq.numel()
    angle = positions.to(F64)[:, None, None] * freq.to(F64)
    c, s = torch.cos(angle) * amplitude, torch.sin(angle) * amplitude * (-1 if back else 1)
    i = torch.arange(rot // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)
    y, size = x.clone(), x.abs()
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    pair = (a.abs() + b.abs()) * abs(amplitude)
    size[..., ia] = pair
    size[..., ib] = pair
    return y, size


def norm(x, w):
    if w is None:
        return x.to(F64), None
    x = x.to(F64)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r * w.to(F64), r


def half_step(want, dtype):
    return want.abs() * (torch.finfo(dtype).eps / 2) + TINY[dtype]


def close(got, want, tol):
    err = (got.to(F64) - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist(), float(err[bad][0]),
                                 float(tol[bad][0]))


def check_fwd(y, x, w, positions, freq, adjacent, amplitude=1.0):
    z, _ = norm(x, w)
    want, size = turn(z, positions, freq, adjacent, amplitude)
    close(y, want, 24 * ULP * size + half_step(want, y.dtype))


def normal(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).to(DEV)


def freqs(rot, base=10000.0):
    return rn.rope_frequencies(rot, base, device=DEV)[0]


CASES = [  # T, Hq, Hk, D, rot
    (1, 1, 1, 64, 64), (1, 14, 2, 64, 64), (3, 32, 8, 128, 128), (700, 5, 1, 128, 64), (257, 7, 3, 80, 40),
    (65, 3, 1, 96, 96), (33, 2, 2, 256, 256), (9, 1, 1, 2, 2), (5, 2, 1, 7, 6), (41, 3, 2, 72, 72),
    (2, 1, 1, 1, 0), (130, 4, 1, 64, 0), (17, 40, 8, 128, 126), (2049, 16, 8, 128, 128)]


@pytest.mark.parametrize("T,Hq,Hk,D,rot", CASES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("adjacent", [False, True])
def test_forward_and_backward(T, Hq, Hk, D, rot, dtype, adjacent):
    with_norm = (T + D) % 2 == 1 or T > 600
    qkv = normal((T, Hq + 2 * Hk, D), dtype, T + D)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    wq, wk = (normal((D,), dtype, 1, 0.1, 1.0), normal((D,), dtype, 2, 0.1, 1.0)) if with_norm else (None, None)
    pos = torch.randint(0, 1 << 20, (T,), device=DEV, dtype=torch.int32 if T % 2 else torch.int64)
    f = freqs(rot) if rot else torch.zeros(0, dtype=F64, device=DEV)
    yq, yk, rstd = rn.rmsnorm_rope_fwd(q, pos, f, k=k, wq=wq, wk=wk, interleaved=adjacent)
    assert rn.last_path() == rn.PATH_ROPE
    check_fwd(yq, q, wq, pos, f, adjacent)
    check_fwd(yk, k, wk, pos, f, adjacent)
    if with_norm:
        want = torch.cat([norm(q, wq)[1], norm(k, wk)[1]], dim=1)[..., 0]
        close(rstd, want, 24 * ULP * want)
    else:
        assert rstd is None

    dyq, dyk = normal((T, Hq, D), dtype, 3, 0.1), normal((T, Hk, D), dtype, 4, 0.1)
    for saved in ([rstd, None] if with_norm else [None]):
        dq, dk, dwq, dwk = rn.rmsnorm_rope_bwd(dyq, q if with_norm else None, pos, f, dyk=dyk,
                                               k=k if with_norm else None, wq=wq, wk=wk, rstd=saved,
                                               interleaved=adjacent)
        for dy, x, w, dx, dw in ((dyq, q, wq, dq, dwq), (dyk, k, wk, dk, dwk)):
            check_bwd(dy, x, w, dx, dw, pos, f, adjacent)


def check_bwd(dy, x, w, dx, dw, pos, f, adjacent, amplitude=1.0):
    g, size = turn(dy.to(F64), pos, f, adjacent, amplitude, back=True)
    if w is None:
        assert dw is None
        close(dx, g, 24 * ULP * size + half_step(g, dx.dtype))
        return
    D, x, w = x.shape[-1], x.to(F64), w.to(F64)
    r = norm(x, w)[1]
    c = (w * g * x).mean(-1, keepdim=True)
    want = r * (w * g - x * r * r * c)
    terms = r * (w.abs() * size + x.abs() * r * r * (w.abs() * size * x.abs()).mean(-1, keepdim=True))
    close(dx, want, 64 * ULP * terms + half_step(want, dx.dtype))
    assert dw.dtype == F32
    rows = x.shape[0] * x.shape[1]
    close(dw, (g * x * r).sum((0, 1)), (rows / 64 + 64 + 64) * ULP * (size * (x * r).abs()).sum((0, 1)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("adjacent", [False, True])
def test_amplitude_and_scaled_frequencies(dtype, adjacent):
    for kind, kw in (("linear", {}), ("ntk", {}), ("yarn", {"original": 4096})):
        f, amp = rn.rope_frequencies(64, 5e5, kind, 8.0, device=DEV, **kw)
        assert (amp > 1) == (kind == "yarn")
        q, w = normal((50, 3, 128), dtype, 5), normal((128,), dtype, 6, 0.1, 1.0)
        pos = torch.arange(50, device=DEV) * 1337
        yq, yk, _ = rn.rmsnorm_rope_fwd(q, pos, f, wq=w, interleaved=adjacent, amplitude=amp)
        assert yk is None
        check_fwd(yq, q, w, pos, f, adjacent, float(torch.tensor(amp, dtype=F32)))
        dq, dk, dw, dwk = rn.rmsnorm_rope_bwd(q, q, pos, f, wq=w, interleaved=adjacent, amplitude=amp)
        assert dk is None and dwk is None
        check_bwd(q, q, w, dq, dw, pos, f, adjacent, float(torch.tensor(amp, dtype=F32)))


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def test_far_and_negative_positions():
    """The angle keeps its fraction at any position: against exact rational
    arithmetic on the 64-bit freq. The kernel's fraction of a turn is within
    2^-64 (half a unit and the truncation of the product's), so |position|
    2^-64 of a turn, and 2^-32 for its top half alone."""
    freq = [math.pi / 2, 1.0, 0.1, 2 * math.pi, 1e-4, 7.5, -0.3, 0.0]
    pos = [0, 1 << 40, (1 << 40) + 1, -1, -(1 << 41) - 3, (1 << 33) + 2, -77, 123456789]
    f = torch.tensor(freq, dtype=F64, device=DEV)
    for adjacent in (False, True):
        for kind in (torch.int64, torch.int32):
            at = [p for p in pos if kind == torch.int64 or abs(p) < 1 << 31]
            x = normal((len(at), 2, 16), F32, 7)
            y, _, _ = rn.rmsnorm_rope_fwd(x, torch.tensor(at, dtype=kind, device=DEV), f, interleaved=adjacent)
            turns = [[Fraction(w) * t / (2 * PI) % 1 for w in freq] for t in at]
            angle = torch.tensor([[float(t * 2 * PI) for t in row] for row in turns], dtype=F64, device=DEV)
            # angles below a turn: position 1 at these frequencies, each token its own
            want = torch.cat([turn(x[i:i + 1].to(F64), torch.ones(1, device=DEV), angle[i], adjacent)[0]
                              for i in range(len(at))])
            size = torch.cat([turn(x[i:i + 1].to(F64), torch.ones(1, device=DEV), angle[i], adjacent)[1]
                              for i in range(len(at))])
            off = torch.tensor([abs(t) * 2.0 ** -64 + 2.0 ** -32 for t in at], dtype=F64, device=DEV) * 2 * math.pi
            close(y, want, (24 * ULP + off[:, None, None]) * size)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layouts(dtype):
    """Head-major, padded, unaligned and broadcast heads; outputs in place."""
    T, H, D = 37, 6, 128
    f, w = freqs(D), normal((D,), dtype, 9, 0.1, 1.0)
    pos = torch.arange(T, device=DEV) * 3
    base = normal((T, H, D), dtype, 10)
    views = {"head-major": base.transpose(0, 1).contiguous().transpose(0, 1),
             "padded": torch.nn.functional.pad(base, (0, 24))[..., :D],
             "odd": torch.nn.functional.pad(base, (1, 2))[..., 1:D + 1],
             "tokens apart": base.repeat_interleave(2, 0)[::2]}
    for name, x in views.items():
        y, _, rstd = rn.rmsnorm_rope_fwd(x, pos, f, wq=w)
        check_fwd(y, base, w, pos, f, False)
        out = torch.empty_strided(x.shape, x.stride(), dtype=dtype, device=DEV)
        assert rn.rmsnorm_rope_fwd(x, pos, f, wq=w, yq=out)[0] is out
        assert torch.equal(out, y), name
        dq, _, dw, _ = rn.rmsnorm_rope_bwd(x, x, pos, f, wq=w, rstd=rstd)
        check_bwd(base, base, w, dq, dw, pos, f, False)
        z = x.clone(memory_format=torch.preserve_format)
        # a clone may be dense, and then takes wider packs, which add in another order
        rn.rmsnorm_rope_fwd(z, pos, f, wq=w, yq=z)
        check_fwd(z, base, w, pos, f, False)
    one = base[:, :1].expand(T, H, D)
    y, _, _ = rn.rmsnorm_rope_fwd(one, pos, f, wq=w)
    check_fwd(y, one, w, pos, f, False)
    dq, _, dw, _ = rn.rmsnorm_rope_bwd(one, one, pos, f, wq=w)
    check_bwd(one, one, w, dq, dw, pos, f, False)
    # windows of one buffer, turned in place
    qkv = normal((T, H + 4, D), dtype, 11)
    keep = qkv.clone()
    rn.rmsnorm_rope_fwd(qkv[:, :H], pos, f, k=qkv[:, H:H + 2], yq=qkv[:, :H], yk=qkv[:, H:H + 2])
    check_fwd(qkv[:, :H], keep[:, :H], None, pos, f, False)
    check_fwd(qkv[:, H:H + 2], keep[:, H:H + 2], None, pos, f, False)
    assert torch.equal(qkv[:, H + 2:], keep[:, H + 2:])


def test_one_norm_of_two_and_infinities():
    T, D = 11, 64
    q, k = normal((T, 3, D), BF16, 12), normal((T, 2, D), BF16, 13)
    f, w, pos = freqs(32), normal((D,), BF16, 14, 0.1, 1.0), torch.arange(T, device=DEV)
    yq, yk, rstd = rn.rmsnorm_rope_fwd(q, pos, f, k=k, wk=w)
    check_fwd(yq, q, None, pos, f, False)
    check_fwd(yk, k, w, pos, f, False)
    close(rstd[:, 3:], norm(k, w)[1][..., 0], torch.full((T, 2), 24 * ULP * 100, dtype=F64, device=DEV))
    dq, dk, dwq, dwk = rn.rmsnorm_rope_bwd(q, None, pos, f, dyk=k, k=k, wk=w, rstd=rstd)
    assert dwq is None
    check_bwd(q, None, None, dq, None, pos, f, False)
    check_bwd(k, k, w, dk, dwk, pos, f, False)
    # what does not turn is not touched by its neighbours' infinities
    q[3, 1, 40] = float("inf")
    q[4, 1, 63] = float("nan")
    yq, _, _ = rn.rmsnorm_rope_fwd(q, pos, f)
    assert torch.equal(yq[..., 32:].nan_to_num(7.0), q[..., 32:].nan_to_num(7.0))
    assert bool(torch.isfinite(yq[..., :32]).all())


def test_empty():
    f = freqs(64)
    q = torch.empty(0, 3, 64, dtype=BF16, device=DEV)
    pos = torch.empty(0, dtype=torch.int64, device=DEV)
    y, _, _ = rn.rmsnorm_rope_fwd(q, pos, f)
    assert y.shape == q.shape
    w = torch.ones(64, dtype=BF16, device=DEV)
    dq, _, dw, _ = rn.rmsnorm_rope_bwd(q, q, pos, f, wq=w)
    assert dq.shape == q.shape and bool((dw == 0).all())


def test_gradient_against_differences():
    """<dx, d> against central differences of <dy, y> along d. The quotient's
    own error: each y within 24 roundings of its pair's size, over 2 h; and the
    third-order term, which the same quotient in 64 bits shows."""
    T, H, D, h = 7, 2, 32, 2.0 ** -6
    f, pos = freqs(16), torch.arange(T, device=DEV) * 5
    x, w, dy = normal((T, H, D), F32, 15), normal((D,), F32, 16, 0.1, 1.0), normal((T, H, D), F32, 17)
    dq, _, dw, _ = rn.rmsnorm_rope_bwd(dy, x, pos, f, wq=w)
    dxs, dws = normal((T, H, D), F32, 18), normal((D,), F32, 19)

    def loss(x, w):
        return (dy.to(F64) * rn.rmsnorm_rope_fwd(x, pos, f, wq=w)[0].to(F64)).sum()

    def loss64(x, w):
        return (dy.to(F64) * turn(norm(x, w)[0], pos, f, False)[0]).sum()

    size = turn(norm(x, w)[0], pos, f, False)[1]
    noise = 2 * float((dy.to(F64).abs() * size * 24 * ULP).sum()) / (2 * h) * 2
    for up, down, got in ((lambda t: (x + t * dxs, w), None, (dq.to(F64) * dxs.to(F64)).sum()),
                          (lambda t: (x, w + t * dws), None, (dw.to(F64) * dws.to(F64)).sum())):
        quotient = (loss(*up(h)) - loss(*up(-h))) / (2 * h)
        quotient64 = (loss64(*up(h)) - loss64(*up(-h))) / (2 * h)
        assert abs(float(quotient - quotient64)) <= noise
        fine = (loss64(*(t.to(F64) for t in up(0.0))) * 0)       # shape only
        tiny = 2.0 ** -12
        deriv = (loss64(*(a.to(F64) + s for a, s in zip(up(0.0), step(up, tiny)))) -
                 loss64(*(a.to(F64) - s for a, s in zip(up(0.0), step(up, tiny))))) / (2 * tiny)
        assert abs(float(got - deriv + fine)) <= noise + 1e-4 * abs(float(deriv))


def step(up, t):
    """The step of `up` at t in 64 bits."""
    return [(b.to(F64) - a.to(F64)) * (t / 1.0) for a, b in zip(up(0.0), up(1.0))]


def test_autograd_and_streams():
    T, Hq, Hk, D = 19, 4, 2, 64
    q, k = normal((T, Hq, D), BF16, 20).requires_grad_(), normal((T, Hk, D), BF16, 21).requires_grad_()
    wq, wk = normal((D,), BF16, 22, 0.1, 1.0).requires_grad_(), normal((D,), BF16, 23, 0.1, 1.0).requires_grad_()
    f, pos = freqs(D), torch.arange(T, device=DEV)
    yq, yk = autograd.rms_norm_rope(q, k, pos, f, wq, wk)
    dyq, dyk = normal((T, Hq, D), BF16, 24), normal((T, Hk, D), BF16, 25)
    torch.autograd.backward([yq, yk], [dyq, dyk])
    check_bwd(dyq, q.detach(), wq.detach(), q.grad, rn.rmsnorm_rope_bwd(
        dyq, q.detach(), pos, f, wq=wq.detach())[2], pos, f, False)
    for g in (k.grad, wq.grad, wk.grad):
        assert g is not None and g.dtype == BF16
    # one output unused; a head-major input; no norms
    q2 = normal((Hq, T, D), BF16, 26).transpose(0, 1).requires_grad_()
    k2 = normal((T, Hk, D), BF16, 27).requires_grad_()
    yq, yk = autograd.rms_norm_rope(q2, k2, pos, f)
    yq.backward(dyq)
    check_bwd(dyq, None, None, q2.grad, None, pos, f, False)
    assert bool((k2.grad == 0).all())
    yq, _ = autograd.rms_norm_rope(q, k, pos, f, wq, wk)
    (g,) = torch.autograd.grad(yq.float().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.float().sum(), q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = rn.rmsnorm_rope_fwd(q.detach(), pos, f, k=k.detach(), wq=wq.detach())
    got = rn.rmsnorm_rope_fwd(q.detach(), pos, f, k=k.detach(), wq=wq.detach(), stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[:2], got[:2]))


def test_repeats_and_graph():
    T, Hq, Hk, D = 777, 8, 2, 128
    q, k = normal((T, Hq, D), BF16, 28), normal((T, Hk, D), BF16, 29)
    w, f, pos = normal((D,), BF16, 30, 0.1, 1.0), freqs(D), torch.arange(T, device=DEV)

    def both():
        y = rn.rmsnorm_rope_fwd(q, pos, f, k=k, wq=w, wk=w)
        return y[:2] + rn.rmsnorm_rope_bwd(q, q, pos, f, dyk=k, k=k, wq=w, wk=w, rstd=y[2])

    first = [t.clone() for t in both()]
    assert all(torch.equal(a, b) for a, b in zip(first, both()))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    old = q.clone()
    q.mul_(2)
    g.replay()
    want = both()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    q.copy_(old)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, first))


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,page", [(1, 4, 1, 64, 64, 16), (70, 32, 8, 128, 128, 16),
                                                (333, 5, 5, 80, 40, 7), (50, 0, 2, 64, 0, 1),
                                                (1200, 16, 8, 128, 64, 64)])
@pytest.mark.parametrize("head_major", [False, True])
def test_append(dtype, T, Hq, Hk, D, rot, page, head_major):
    pages = -(-T // page) + 2
    qkv = normal((T, Hq + 2 * Hk, D), dtype, T)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    shape = (pages, Hk, page, D) if head_major else (pages, page, Hk, D)
    ck, cv = normal(shape, dtype, 1), normal(shape, dtype, 2)
    if head_major:
        ck, cv = ck.transpose(1, 2), cv.transpose(1, 2)
    slots = torch.randperm(pages * page, device=DEV)[:T]
    if T > 20:
        slots[3], slots[5], slots[9] = -1, pages * page, -(1 << 40)
    if T % 2:
        slots = slots.clamp(-(1 << 31), (1 << 31) - 1).to(torch.int32)
    wk = normal((D,), dtype, 3, 0.1, 1.0) if T % 3 else None
    f = freqs(rot) if rot else None
    pos = torch.randint(0, 1 << 17, (T,), device=DEV) if rot else None
    old_k, old_v = ck.clone(), cv.clone()
    y = rn.rmsnorm_rope_append(k, v, pos, f, slots, ck, cv, q=q if Hq else None, wk=wk, interleaved=T % 2 == 0)
    assert rn.last_path() == rn.PATH_ROPE_APPEND
    p = pos if rot else torch.zeros(T, device=DEV)
    f = f if rot else torch.zeros(0, dtype=F64, device=DEV)
    if Hq:
        check_fwd(y, q, None, p, f, T % 2 == 0)
    else:
        assert y is None
    s = slots.long()
    kept = (s >= 0) & (s < pages * page)
    got_k, got_v = ck[s[kept] // page, s[kept] % page], cv[s[kept] // page, s[kept] % page]
    check_fwd(got_k, k[kept], wk, p[kept], f, T % 2 == 0)
    assert torch.equal(got_v, v[kept])
    others = torch.ones(pages, page, dtype=torch.bool, device=DEV)
    others[s[kept] // page, s[kept] % page] = False
    assert torch.equal(ck[others], old_k[others]) and torch.equal(cv[others], old_v[others])


def test_append_interleaved_cache_past_32_bits():
    """k and v rows in one buffer; a slot whose byte offset passes 2^32."""
    H, D, page = 8, 128, 64
    pages = (1 << 31) // (page * H * D) + 3
    kv = torch.zeros(pages, 2, page, H, D, dtype=BF16, device=DEV)
    ck, cv = kv[:, 0], kv[:, 1]
    k, v = normal((2, H, D), BF16, 31), normal((2, H, D), BF16, 32)
    slots = torch.tensor([pages * page - 1, 5], device=DEV)
    rn.rmsnorm_rope_append(k, v, None, None, slots, ck, cv)
    assert torch.equal(ck[-1, -1], k[0]) and torch.equal(cv[-1, -1], v[0])
    assert torch.equal(ck[0, 5], k[1]) and torch.equal(cv[0, 5], v[1])
    assert int((kv != 0).any(-1).sum()) == 4 * H


# ------------------------------------------------------------- 4-bit cache
VALUES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64)


def round4(v):
    """v (float64) to the nearest of VALUES and their negatives, ties to the
    even code."""
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(F64)
    return torch.round(a / step) * step * torch.sign(v)


def e4m3(v):
    return v.to(F32).to(torch.float8_e4m3fn).to(F64)


def unpack(cache, D):
    """(k, v) [pages, heads, page, D] float64 of a 4-bit cache without the
    heads' scales, from the layout that the header states."""
    P, H, N, _ = cache.shape
    G = D // 16
    c = cache.cpu()
    lut = torch.cat([VALUES, -VALUES])
    kc = c[..., :8 * D].reshape(P, H, N, 16, D // 2).long()
    ks = c[..., 8 * D:9 * D].reshape(P, H, N, 16, G)
    vc = c[..., 9 * D:17 * D].reshape(P, H, N, G, 16, 8).transpose(3, 4).reshape(P, H, N, 16, D // 2).long()
    vs = c[..., 17 * D:].reshape(P, H, N, G, 16).transpose(3, 4).contiguous()

    def out(codes, s):
        x = torch.stack([lut[codes & 15], lut[codes >> 4]], dim=-1).flatten(-2)
        s = s.contiguous().view(torch.float8_e4m3fn).to(F64)
        return x.reshape(P, H, N * 16, D), s.reshape(P, H, N * 16, G)
    return out(kc, ks) + out(vc, vs)


def check_quant4(codes, scale, x, g, delta):
    """codes and scales [rows, H, ...] against exact x: the scale rounds a
    maximum within delta of the exact one, a code a quotient within delta."""
    y = x.unflatten(-1, (-1, 16))
    t = y.abs().amax(-1) / (6 * g[:, None])
    lo, hi = (e4m3((t * (1 + d)).clamp(2.0 ** -9, 448)) for d in (-delta, delta))
    assert bool(((scale == lo) | (scale == hi)).all())
    v = y / (scale * g[:, None])[..., None]
    a, b = round4(v * (1 - delta)).flatten(-2), round4(v * (1 + delta)).flatten(-2)
    assert bool(((codes >= torch.minimum(a, b)) & (codes <= torch.maximum(a, b))).all())


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,H,D,rot,page", [(1, 1, 64, 64, 16), (67, 2, 64, 32, 32), (130, 8, 128, 128, 16),
                                            (700, 3, 128, 40, 48), (33, 4, 128, 0, 16)])
def test_append_kv4_and_read(dtype, T, H, D, rot, page):
    pages = -(-T // page) + 2
    qkv = normal((T, 3 * H, D), dtype, T)
    q, k, v = qkv[:, :H], qkv[:, H:2 * H], qkv[:, 2 * H:]
    k[0, 0, :16] = 0                             # a group of zeros
    cache = rn.kv4_cache(pages, H, page, D, device=DEV)
    fill = torch.randint(0, 256, cache.shape, device=DEV, dtype=torch.uint8)
    cache.copy_(fill)
    slots = torch.randperm(pages * page, device=DEV)[:T]
    if T > 20:
        slots[3], slots[5] = -1, pages * page
    gs = T % 2 == 0
    ks = torch.rand(H, device=DEV) + 0.01 if gs else None
    vs = torch.rand(H, device=DEV) * 1e-3 + 1e-5 if gs else None
    w = normal((D,), dtype, 3, 0.1, 1.0) if T % 3 else None
    f = freqs(rot) if rot else None
    pos = torch.randint(0, 1 << 17, (T,), device=DEV) if rot else None
    y = rn.rmsnorm_rope_append_kv4(k, v, pos, f, slots, cache, q=q, wq=w, wk=w, k_scale=ks, v_scale=vs)
    assert rn.last_path() == rn.PATH_ROPE_APPEND
    p = pos if rot else torch.zeros(T, device=DEV)
    f = f if rot else torch.zeros(0, dtype=F64, device=DEV)
    check_fwd(y, q, w, p, f, False)
    kept = (slots >= 0) & (slots < pages * page)
    s = slots[kept]
    got = [t.transpose(1, 2).reshape(pages * page, H, -1)[s.cpu()] for t in unpack(cache, D)]
    want_k = turn(norm(k, w)[0], p, f, False)[0][kept].cpu()
    one = torch.ones(H, dtype=F64)
    # an element of k may be small beside its pair: within 24 roundings of the pair's size
    size = turn(norm(k, w)[0], p, f, False)[1][kept].cpu()
    delta = 24 * ULP
    kx = want_k
    yk = kx.unflatten(-1, (-1, 16))
    g = ks.cpu().to(F64) if gs else one
    err = (delta * size).unflatten(-1, (-1, 16))
    top = yk.abs().amax(-1)
    lo, hi = (e4m3(((top + d * err.amax(-1)) / (6 * g[:, None])).clamp(2.0 ** -9, 448)) for d in (-2, 2))
    assert bool(((got[1] == lo) | (got[1] == hi)).all())
    d = (got[1] * g[:, None])[..., None]
    a, b = round4((yk - 2 * err) / d).flatten(-2), round4((yk + 2 * err) / d).flatten(-2)
    assert bool(((got[0] >= a) & (got[0] <= b)).all())
    # the values have no arithmetic before them: only the quotients' roundings
    check_quant4(got[2], got[3], v[kept].cpu().to(F64), vs.cpu().to(F64) if gs else one, 0.0 if not gs else 4 * ULP)
    # read back
    rk, rks, rv, rvs = rn.rmsnorm_kv4_read(cache, slots)
    assert rn.last_path() == rn.PATH_KV4_READ
    for r, want in zip((rk, rks, rv, rvs), got):
        assert torch.equal(r[kept].float().cpu().to(F64), want)
        assert bool((r[~kept].float() == 0).all())
    # rows of other slots keep their bytes
    others = torch.ones(pages * page, dtype=torch.bool)
    others[s.cpu()] = False
    for now, was in zip(unpack(cache, D), unpack(fill, D)):
        now, was = (t.transpose(1, 2).reshape(pages * page, -1)[others] for t in (now, was))
        assert torch.equal(now.nan_to_num(9.0), was.nan_to_num(9.0))


def test_kv4_ties_and_specials():
    """Quotients in the middle between two codes go to the even one; NaN and
    infinities are stored as the largest code."""
    H, D = 1, 64
    cache = rn.kv4_cache(1, H, 16, D, device=DEV)
    v = torch.zeros(3, H, D, dtype=F32, device=DEV)
    v[0, 0, :16] = torch.tensor([6.0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5,
                                 -5, .24])
    v[1, 0, 3], v[1, 0, 20], v[1, 0, 33] = float("nan"), float("inf"), -float("inf")
    v[1, 0, 4], v[2, 0, 0] = 6.0, 1e30
    k = torch.zeros_like(v)
    rn.rmsnorm_rope_append_kv4(k, v, None, None, torch.arange(3, device=DEV), cache)
    _, _, rv, rs = rn.rmsnorm_kv4_read(cache, torch.arange(3, device=DEV))
    rv, rs = rv.float(), rs.float()
    assert rv[0, 0, :16].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, 0]
    assert rs[0, 0, 0] == 1.0 and rs[0, 0, 1] == 2.0 ** -9
    assert rv[1, 0, 3] == 6 and rv[1, 0, 4] == 6 and rs[1, 0, 0] == 1.0
    assert rv[1, 0, 20] == 6 and rs[1, 0, 1] == 448 and rv[1, 0, 33] == -6
    assert rv[2, 0, 0] == 6 and rs[2, 0, 0] == 448
    assert bool(torch.isfinite(rv).all()) and bool(torch.isfinite(rs).all())


@pytest.mark.parametrize("g", [1.0, 0.37, 1e-25, 3e20])
def test_kv4_quotients_are_rounded_once(g):
    """Values right between two codes, and next to that, at scales of the
    heads near one and far from it: the codes of the fp32 division."""
    H, D, n = 1, 128, 2000
    gen = torch.Generator().manual_seed(5)
    gs = torch.tensor([g], dtype=F32)
    middle = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x = middle[torch.randint(0, 8, (n, H, D), generator=gen)] * (torch.randint(0, 2, (n, H, D), generator=gen) * 2 - 1)
    scale = (torch.randint(8, 16, (n, H, D // 16, 1), generator=gen) / 8.0) * \
        2.0 ** torch.randint(-5, 6, (n, H, D // 16, 1), generator=gen)
    v = x.view(n, H, D // 16, 16) * scale * gs
    v = torch.where(torch.rand(v.shape, generator=gen) < 0.3, torch.nextafter(v, torch.zeros(())), v)
    v[..., 0] = (6.0 * scale * gs)[..., 0]
    v = v.view(n, H, D)
    pages = -(-n // 16)
    cache = rn.kv4_cache(pages, H, 16, D, device=DEV)
    slots = torch.arange(n, device=DEV)
    rn.rmsnorm_rope_append_kv4(v.to(DEV), v.to(DEV), None, None, slots, cache, k_scale=gs.to(DEV), v_scale=gs.to(DEV))
    top = (v.view(n, H, D // 16, 16).abs().amax(-1) / (6.0 * gs)).clamp(2.0 ** -9, 448)
    sc = top.to(torch.float8_e4m3fn).float()
    quotient = v.view(n, H, D // 16, 16) / (sc * gs)[..., None]              # fp32, rounded once
    want = round4(quotient.to(F64)).view(n, H, D)
    for got, got_s in zip(*[iter(rn.rmsnorm_kv4_read(cache, slots))] * 2):
        assert torch.equal(got_s.float().cpu(), sc)
        assert torch.equal(got.float().cpu().to(F64), want)
