"""GPU tier: attention over the 4-bit cache against its definition in 64 bits,
and the chain of a decode step: projection, append, attention.

Tolerances, from the arithmetic. A score is a sum of D products in fp32 on the
tensor cores (each addition off by at most 2^-22 of the magnitudes: D 2^-22 of
A = scale sum |q k|), times two factors: dx = (D + 8) 2^-22 A. A weight is off
by dx, by exp2's 2^-22 and by one rounding to fp16, 2^-11 (half a step, 2^-12,
twice: the reference that a term is taken from moves by exp2 again):
eps = dx + 2^-11. A row is a quotient of two sums of such weights: 2 eps of
sum p |v|. Its sums are fp32 additions in order, at most L / 8 of them in a
warp, each off by 2^-22: (L / 8 + 64) 2^-22 of sum p |v|. Weights below 2^-18
of the row's reference (which lies at most 2^11 under its largest) lie under
fp16's normal range, where a rounding is off by at most 2^-25: with 2^4 for the
reference each within 2^-29 of it, and so of the largest. Then half a step of the output. The log of the denominator is off by
dx + (L / 8 + 64) 2^-22, and a few roundings of its own size.
"""
import math

import pytest
import torch

from rmsnorm_fwd_bwd_02_gb300 import rmsnorm as rn
from tests.test_rope_gpu import BF16, DEV, F16, F32, F64, check_fwd, freqs, normal, unpack

pytestmark = pytest.mark.gpu

PATHS = {1: rn.PATH_KV4_ATTENTION, 3: rn.PATH_KV4_ATTENTION, 2: rn.PATH_KV4_PROMPT}
HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {BF16: 2.0 ** -134, F16: 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tier needs a CUDA device")
    rn.lib()
    rn.wait_timeouts(reset=True)
    yield
    assert rn.wait_timeouts(reset=True) == 0


def make_cache(pages, H, page, D, seed, std=1.0):
    """A cache of random tokens, written by the append."""
    cache = rn.kv4_cache(pages, H, page, D, device=DEV)
    n = pages * page
    k, v = normal((n, H, D), F32, seed), normal((n, H, D), F32, seed + 1, std, 0.1)
    rn.rmsnorm_rope_append_kv4(k, v, None, None, torch.arange(n, device=DEV), cache)
    return cache


def dense(cache, D, ks=None, vs=None):
    k, sk, v, sv = unpack(cache, D)
    k = k * sk.repeat_interleave(16, -1)
    v = v * sv.repeat_interleave(16, -1)
    if ks is not None:
        k = k * ks.cpu().to(F64)[None, :, None, None]
    if vs is not None:
        v = v * vs.cpu().to(F64)[None, :, None, None]
    return k, v


def check(out, lse, q, cache, table, lens, starts, scale=None, ks=None, vs=None):
    """Every row of every sequence; rows of none are the caller's."""
    T, H, D = q.shape
    kk, vv = dense(cache, D, ks, vs)
    Hk, page = kk.shape[1], kk.shape[2]
    kk, vv = kk.to(DEV), vv.to(DEV)
    scale = 1 / math.sqrt(D) if scale is None else scale
    for b in range(table.shape[0]):
        q0, q1 = (b, b + 1) if starts is None else (starts[b], starts[b + 1])
        n = q1 - q0
        L = min(max(lens[b], 0), table.shape[1] * page)
        if n <= 0:
            continue
        pages = table[b, :-(-L // page)].to(DEV).long()
        there = ((pages >= 0) & (pages < kk.shape[0])).repeat_interleave(page)[:L]
        pages = pages.clamp(0, kk.shape[0] - 1)
        k = kk[pages].transpose(0, 1).reshape(Hk, -1, D)[:, :L]
        v = vv[pages].transpose(0, 1).reshape(Hk, -1, D)[:, :L]
        v = torch.where(there[None, :, None], v, torch.zeros_like(v))
        k = torch.where(there[None, :, None], k, torch.zeros_like(k))
        qq = q[q0:q1].to(F64).view(n, Hk, H // Hk, D)
        x = torch.einsum("nhgd,hld->nhgl", qq, k) * scale
        size = torch.einsum("nhgd,hld->nhgl", qq.abs(), k.abs()) * abs(scale)
        seen = torch.arange(L, device=DEV)[None, :] < (L - n + 1 + torch.arange(n, device=DEV))[:, None]
        seen = (seen & there[None, :])[:, None, None, :].expand_as(x)
        x = x.masked_fill(~seen, -math.inf)
        none = ~seen.any(-1)
        lse_w = torch.logsumexp(x, -1) if L else torch.full(x.shape[:-1], -math.inf, dtype=F64, device=DEV)
        p = torch.exp(x - torch.where(none, torch.zeros_like(lse_w), lse_w)[..., None])
        want = torch.einsum("nhgl,hld->nhgd", p, v)
        mag = torch.einsum("nhgl,hld->nhgd", p, v.abs())
        dx = ((D + 8) * 2.0 ** -22 * (size * seen).amax(-1) if L else torch.zeros_like(lse_w))[..., None]
        sums = (L / 8 + 64) * 2.0 ** -22
        top = v.abs().amax() if L else 0.0
        # each p within 2^-29 of the largest, which is at most the sum
        small = L * 2.0 ** -29 * top
        dt = out.dtype
        tol = (2 * (dx + 2.0 ** -11) + sums) * mag + small + want.abs() * HALF[dt] + TINY[dt]
        got = out[q0:q1].to(F64).view_as(want)
        err = (got - want).abs()
        bad = ~(err <= tol)
        assert not bool(bad.any()), (b, int(bad.sum()), bad.nonzero()[0].tolist(), float(err[bad][0]),
                                     float(tol[bad][0]))
        assert bool((got[none] == 0).all())
        if lse is not None:
            gl = lse[q0:q1].to(F64).view_as(lse_w)
            assert bool((gl[none] == -math.inf).all())
            e = (gl - lse_w).abs()[~none]
            t = (dx[..., 0] + sums + 2.0 ** -20 + 2.0 ** -21 * (lse_w.abs() + size.amax(-1) if L else 0))[~none]
            assert bool((e <= t).all()), (b, float((e - t).max()))


def table_of(B, blocks, pages, seed):
    g = torch.Generator().manual_seed(seed)
    assert pages >= B * blocks
    return torch.randperm(pages, generator=g)[:B * blocks].to(torch.int32).view(B, blocks)


@pytest.fixture(params=[1, 3, 2], ids=["list", "clusters", "prompt"])
def kernel(request):
    rn.set_kv4_test(request.param)
    yield request.param
    rn.set_kv4_test(0)


@pytest.fixture(params=[1, 3], ids=["list", "clusters"])
def few(request):
    rn.set_kv4_test(request.param)
    yield request.param
    rn.set_kv4_test(0)


def run(T, H, D, dtype, cache, table, lens, starts=None, seed=5, path=None, **kw):
    q = normal((T, H, D), dtype, seed)
    s = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
    out, lse = rn.rmsnorm_kv4_attention(q, cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                        q_starts=s, want_lse=True, **kw)
    assert rn.last_path() == (path or rn.PATH_KV4_ATTENTION)
    check(out, lse, q, cache, table, lens, starts, scale=kw.get("scale"), ks=kw.get("k_scale"),
          vs=kw.get("v_scale"))
    return q, out, lse


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk,G", [(1, 1), (2, 7), (8, 4), (2, 9), (1, 40)])
def test_one_token(dtype, D, Hk, G, few):
    page = 16 if G % 2 else 48
    lens = [1, 0, 15, 16, 17, 31, 32, 33, 255, 256, 257, 300, 513, 767]
    B, blocks = len(lens), -(-768 // page)
    cache = make_cache(B * blocks, Hk, page, D, G)
    run(B, Hk * G, D, dtype, cache, table_of(B, blocks, B * blocks, 3), lens)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,Hk,G", [(64, 2, 7), (128, 2, 4), (128, 1, 8)])
@pytest.mark.parametrize("counts", [(1, 2, 3, 0, 5, 4), (17, 1, 40, 0, 33, 9), (64, 130, 0, 1, 65, 128)])
def test_several_tokens(dtype, D, Hk, G, counts, kernel):
    """Rows see the tokens up to their own; more query tokens than cached ones
    leave the first rows nothing."""
    page, lens = 32, [700, 2, 3, 50, 1, 333]
    B, blocks = len(lens), 22
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    cache = make_cache(B * blocks + 3, Hk, page, D, G)
    run(starts[-1], Hk * G, D, dtype, cache, table_of(B, blocks, B * blocks + 3, 4), lens, starts,
        path=PATHS[kernel])


def test_long_and_one_unit(few):
    """A length that every CTA has a part of; and a table of one unit, where
    nothing is joined."""
    page = 64
    cache = make_cache(640, 2, page, 128, 1)
    run(1, 8, 128, BF16, cache, table_of(1, 640, 640, 1), [640 * 64 - 5])
    run(2, 8, 128, BF16, cache, table_of(2, 300, 640, 1), [19000, 1])
    run(2, 8, 128, F16, cache, table_of(2, 4, 640, 1), [256, 77])
    run(3, 8, 128, F16, cache, table_of(3, 0, 640, 1).view(3, 0), [0, 5, -3])


def test_many_sequences(few):
    B, page, blocks = 333, 16, 5
    cache = make_cache(B * blocks, 1, page, 64, 2)
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 81, (B,), generator=g).tolist()
    run(B, 3, 64, BF16, cache, table_of(B, blocks, B * blocks, 6), lens)


def test_scales_and_softmax_scale(few):
    Hk, G, D, page = 3, 2, 64, 16
    ks, vs = torch.tensor([0.5, 3.0, 1e-3], device=DEV), torch.tensor([2.0, 1e-4, 7.0], device=DEV)
    cache = rn.kv4_cache(20, Hk, page, D, device=DEV)
    k, v = normal((320, Hk, D), F32, 1) * ks[:, None], normal((320, Hk, D), F32, 2) * vs[:, None]
    rn.rmsnorm_rope_append_kv4(k, v, None, None, torch.arange(320, device=DEV), cache, k_scale=ks, v_scale=vs)
    for scale in (None, 0.3, -0.2, 0.0):
        run(2, Hk * G, D, BF16, cache, table_of(2, 10, 20, 2), [150, 77], k_scale=ks, v_scale=vs, scale=scale)


def test_peaked_and_shifted_scores(few):
    """Scores that grow along the sequence (the reference moves again and
    again), and ones far from zero."""
    D, page = 128, 16
    cache = rn.kv4_cache(64, 1, page, D, device=DEV)
    k = normal((1024, 1, D), F32, 1, 0.3) + torch.linspace(-4, 4, 1024, device=DEV)[:, None, None]
    v = normal((1024, 1, D), F32, 2)
    rn.rmsnorm_rope_append_kv4(k, v, None, None, torch.arange(1024, device=DEV), cache)
    table = torch.arange(64, dtype=torch.int32)[None]
    for sign in (1, -1):
        q = (normal((1, 4, D), BF16, 3, 0.2).float() + sign).to(BF16)
        out, lse = rn.rmsnorm_kv4_attention(q, cache, table.to(DEV), torch.tensor([1000], dtype=torch.int32,
                                                                                  device=DEV), want_lse=True)
        check(out, lse, q, cache, table, [1000], None)


def test_garbage_where_nothing_is_seen(kernel):
    """Bytes that stand for NaN behind a sequence's end, in a page's rest and
    in pages that the table does not reach change nothing; neither do pages
    outside the cache, whose tokens are masked."""
    D, page, Hk = 128, 32, 2
    for D in (64, 128):
        cache = make_cache(12, Hk, page, D, 7)
        table = torch.tensor([[3, 5, 7, 9], [2, 4, 12, -1], [0, 1 << 30, 6, 8]], dtype=torch.int32)
        lens, starts = [77, 128, 101], [0, 3, 4, 9]
        bad = cache.clone()
        bad[7, :, 0, :] = 0xFF                       # holds tokens 64 .. 79 of sequence 0: 77 seen
        keep = cache[7, :, 0].clone()
        kc, ks = 8 * D, 9 * D
        for t in range(13):                          # give the seen ones their bytes back
            bad[7, :, 0, t * D // 2:(t + 1) * D // 2] = keep[:, t * D // 2:(t + 1) * D // 2]
            bad[7, :, 0, kc + t * D // 16:kc + (t + 1) * D // 16] = keep[:, kc + t * D // 16:kc + (t + 1) * D // 16]
            for g in range(D // 16):
                a = ks + g * 128 + t * 8
                bad[7, :, 0, a:a + 8] = keep[:, a:a + 8]
                bad[7, :, 0, 17 * D + g * 16 + t] = keep[:, 17 * D + g * 16 + t]
        bad[7, :, 1], bad[9], bad[10], bad[11] = 0xFF, 0xFF, 0xFF, 0xFF
        bad[6, :, 1] = 0x7F                          # tokens 80 .. 95 of sequence 2: seen
        cache[6, :, 1] = 0
        bad[6, :, 1] = 0
        _, a, la = run(9, 4, D, BF16, cache, table, lens, starts, path=PATHS[kernel])
        _, b, lb = run(9, 4, D, BF16, bad, table, lens, starts, path=PATHS[kernel])
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_rows_of_no_sequence_and_unsound_starts(kernel):
    D, page = 64, 16
    cache = make_cache(8, 1, page, D, 3)
    table = torch.arange(8, dtype=torch.int32).view(2, 4)
    q = normal((9, 2, D), F16, 1)
    out, lse = torch.full((9, 2, D), 3.0, dtype=F16, device=DEV), torch.full((9, 2), 4.0, device=DEV)
    lens = torch.tensor([60, 33], dtype=torch.int32, device=DEV)
    s = torch.tensor([2, 4, 7], dtype=torch.int32, device=DEV)
    r = rn.rmsnorm_kv4_attention(q, cache, table.to(DEV), lens, q_starts=s, out=out, lse=lse)
    assert r[0] is out and r[1] is lse
    check(out, lse, q, cache, table, [60, 33], [2, 4, 7])
    for rows in (slice(0, 2), slice(7, 9)):
        assert bool((out[rows] == 3).all()) and bool((lse[rows] == 4).all())
    # starts that run backwards or past the rows: the sound part of them
    s = torch.tensor([-5, 3, 1], dtype=torch.int32, device=DEV)
    out.fill_(3.0)
    rn.rmsnorm_kv4_attention(q, cache, table.to(DEV), lens, q_starts=s, out=out)
    check(out, None, q, cache, table, [60, 33], [0, 3, 1])
    assert bool((out[3:] == 3).all())
    s = torch.tensor([6, 8, 1 << 30], dtype=torch.int32, device=DEV)
    rn.rmsnorm_kv4_attention(q, cache, table.to(DEV), lens, q_starts=s, out=out)
    check(out, None, q, cache, table, [60, 33], [6, 8, 9])


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_layouts(dtype, few):
    """Windows of a fused projection, head-major and unaligned q and out; a
    table with a row stride."""
    D, page, Hk, G, B = 64, 16, 2, 3, 5
    cache = make_cache(40, Hk, page, D, 3)
    table = table_of(B, 8, 40, 2)
    lens = [100, 128, 1, 64, 90]
    wide = torch.zeros(B, 11, dtype=torch.int32, device=DEV)
    wide[:, :8] = table.to(DEV)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    base = normal((B, Hk * G + 4, D), dtype, 4)
    views = [base[:, :Hk * G], base.transpose(0, 1).contiguous().transpose(0, 1)[:, 2:2 + Hk * G],
             torch.nn.functional.pad(base, (1, 1))[:, 1:1 + Hk * G, 1:1 + D]]
    for x in views:
        out = torch.empty_strided(x.shape, x.stride(), dtype=dtype, device=DEV)
        rn.rmsnorm_kv4_attention(x, cache, wide[:, :8], dl, out=out)
        check(out, None, x, cache, table, lens, None)
        got, _ = rn.rmsnorm_kv4_attention(x, cache, wide[:, :8], dl)
        assert torch.equal(got, out)


def test_magnitudes_of_q(few):
    """Rows scaled by any power of two within the type; zeros."""
    D, page = 128, 16
    cache = make_cache(8, 1, page, D, 3)
    table = torch.arange(8, dtype=torch.int32)[None]
    lens = torch.tensor([111], dtype=torch.int32, device=DEV)
    q = normal((1, 6, D), BF16, 4)
    for h, e in enumerate((-60, -20, -8, 2, 4)):
        q[:, h] *= 2.0 ** e
    q[:, 5] = 0
    out, lse = rn.rmsnorm_kv4_attention(q, cache, table.to(DEV), lens, want_lse=True)
    check(out, lse, q, cache, table, [111], None)
    q = normal((1, 6, D), BF16, 5) * 2.0 ** 60          # scale brings it back
    out, lse = rn.rmsnorm_kv4_attention(q, cache, table.to(DEV), lens, scale=2.0 ** -63, want_lse=True)
    check(out, lse, q, cache, table, [111], None, scale=2.0 ** -63)


def test_rows_of_nan_and_infinity(kernel):
    """A NaN or an infinity in a row of q makes that row NaN (or what the
    softmax of infinities is) and leaves its neighbours as they are."""
    D, page, L = 128, 16, 900
    cache = make_cache(60, 1, page, D, 3)
    table = torch.arange(60, dtype=torch.int32, device=DEV)[None]
    lens, s = torch.tensor([L], dtype=torch.int32, device=DEV), torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    q = normal((3, 4, D), BF16, 4)
    want, want_lse = rn.rmsnorm_kv4_attention(q, cache, table, lens, q_starts=s, want_lse=True)
    q[1, 2, 7], q[2, 0, 100] = float("nan"), float("inf")
    out, lse = rn.rmsnorm_kv4_attention(q, cache, table, lens, q_starts=s, want_lse=True)
    bad = torch.zeros(3, 4, dtype=torch.bool, device=DEV)
    bad[1, 2] = bad[2, 0] = True
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])
    assert bool(out[1, 2].isnan().all()) and bool(lse[1, 2].isnan())
    assert bool(out[2, 0].isnan().all())


def test_long_offsets(few):
    """Pages whose byte offset passes 2^32."""
    D, page, Hk = 128, 64, 8
    pages = (1 << 32) // (Hk * page * 9 * D // 8) + 40
    cache = torch.zeros(pages, Hk, page // 16, 18 * D, dtype=torch.uint8, device=DEV)
    k, v = normal((640, Hk, D), F32, 1), normal((640, Hk, D), F32, 2)
    far = torch.arange(pages - 10, pages, device=DEV)
    slots = (far[:, None] * page + torch.arange(page, device=DEV)).flatten()
    rn.rmsnorm_rope_append_kv4(k, v, None, None, slots, cache)
    small = rn.kv4_cache(10, Hk, page, D, device=DEV)
    rn.rmsnorm_rope_append_kv4(k, v, None, None, torch.arange(640, device=DEV), small)
    assert torch.equal(cache[-10:], small)
    q, lens = normal((1, 32, D), BF16, 3), torch.tensor([633], dtype=torch.int32, device=DEV)
    a, _ = rn.rmsnorm_kv4_attention(q, cache, far.to(torch.int32)[None], lens)
    b, _ = rn.rmsnorm_kv4_attention(q, small, torch.arange(10, dtype=torch.int32, device=DEV)[None], lens)
    assert torch.equal(a, b)
    rk, _, rv, _ = rn.rmsnorm_kv4_read(cache, slots)
    sk, _, sv, _ = rn.rmsnorm_kv4_read(small, torch.arange(640, device=DEV))
    assert torch.equal(rk.view(torch.uint8), sk.view(torch.uint8))
    assert torch.equal(rv.view(torch.uint8), sv.view(torch.uint8))


def test_repeats_and_captured_calls(few):
    """The same bits again; two captured graphs, replayed in turn with other
    lengths, tables and queries."""
    D, page, Hk, G, B = 128, 16, 2, 4, 3
    cache = make_cache(300, Hk, page, D, 3)
    qs = [normal((B, Hk * G, D), BF16, 40 + i) for i in range(2)]
    lens = [torch.tensor([1600, 900, 40], dtype=torch.int32, device=DEV) for _ in range(2)]
    tables = [table_of(B, 100, 300, i).to(DEV) for i in range(2)]
    want = [rn.rmsnorm_kv4_attention(qs[i], cache, tables[i], lens[i]) for i in range(2)]
    again = rn.rmsnorm_kv4_attention(qs[0], cache, tables[0], lens[0])
    assert torch.equal(want[0][0], again[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(rn.rmsnorm_kv4_attention(qs[i], cache, tables[i], lens[i])[0])
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w[0]) for o, w in zip(outs, want))
    lens[0].copy_(torch.tensor([5, 1300, 1599], dtype=torch.int32))
    tables[0].copy_(table_of(B, 100, 300, 77).to(DEV))
    qs[0].mul_(-1)
    graphs[0].replay()
    fresh = rn.rmsnorm_kv4_attention(qs[0], cache, tables[0], lens[0])[0]
    torch.cuda.synchronize()
    assert torch.equal(outs[0], fresh)
    check(outs[0], None, qs[0], cache, tables[0].cpu(), [5, 1300, 1599], None)


def test_two_streams_at_once(few):
    D, page, Hk = 128, 16, 2
    cache = make_cache(400, Hk, page, D, 3)
    q = [normal((4, 8, D), BF16, i) for i in range(2)]
    table = table_of(4, 100, 400, 1).to(DEV)
    lens = torch.tensor([1600, 1599, 800, 3], dtype=torch.int32, device=DEV)
    want = [rn.rmsnorm_kv4_attention(x, cache, table, lens)[0] for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(rn.rmsnorm_kv4_attention(q[i], cache, table, lens, stream=s)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for i, w in enumerate(want) for o in got[i])


def test_waits_that_run_out(kernel):
    """The test hook makes the stages' waits run out: the call ends, counts
    them, and the next one is right again."""
    D, page = 128, 16
    cache = make_cache(60, 1, page, D, 3)
    table = torch.arange(60, dtype=torch.int32)[None]
    q, lens = normal((1, 4, D), BF16, 4), torch.tensor([900], dtype=torch.int32, device=DEV)
    s = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    rn.wait_timeouts(reset=True)
    rn.set_stream_test_fault(16, 2000)
    try:
        rn.rmsnorm_kv4_attention(q, cache, table.to(DEV), lens, q_starts=s)
        torch.cuda.synchronize()
    finally:
        rn.set_stream_test_fault(0, 0)
    assert rn.wait_timeouts(reset=True) > 0
    out, lse = rn.rmsnorm_kv4_attention(q, cache, table.to(DEV), lens, q_starts=s, want_lse=True)
    check(out, lse, q, cache, table, [900], None)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,Hk,G,page", [(128, 8, 4, 64), (64, 2, 7, 16), (128, 2, 1, 48)])
def test_pieces_of_prompts(dtype, D, Hk, G, page):
    """Sizes that the rule gives to the kernel for many rows, ragged ones, a
    prompt from its first token, scores that move the reference."""
    lens, counts = [1500, 640, 333, 777], [600, 640, 64, 300]
    B, blocks = 4, -(-1536 // page)
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    cache = make_cache(B * blocks, Hk, page, D, G)
    table = table_of(B, blocks, B * blocks, 3)
    wide = starts[-1] * G * Hk >= 2 * 4400 and D == 128        # where the rule takes it by itself
    rn.set_kv4_test(0 if wide else 2)
    try:
        run(starts[-1], Hk * G, D, dtype, cache, table, lens, starts, path=rn.PATH_KV4_PROMPT)
        ks, vs = torch.rand(Hk, device=DEV) + 0.1, torch.rand(Hk, device=DEV) + 0.1
        run(starts[-1], Hk * G, D, dtype, cache, table, lens, starts, path=rn.PATH_KV4_PROMPT, scale=-0.4,
            k_scale=ks, v_scale=vs)
        # the largest scores late: one key grows along the sequence
        k = normal((B * blocks * page, Hk, D), F32, 3, 0.2) + \
            torch.linspace(-3, 3, B * blocks * page, device=DEV)[:, None, None]
        rn.rmsnorm_rope_append_kv4(k, k, None, None, torch.arange(B * blocks * page, device=DEV), cache)
        q = (normal((starts[-1], Hk * G, D), dtype, 3, 0.2).float() + 0.7).to(dtype)
        s = torch.tensor(starts, dtype=torch.int32, device=DEV)
        dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
        plain = torch.arange(B * blocks, dtype=torch.int32).view(B, blocks)
        out, lse = rn.rmsnorm_kv4_attention(q, cache, plain.to(DEV), dl, q_starts=s, want_lse=True)
        check(out, lse, q, cache, plain, lens, starts)
        # the same bits again, and from a window that is not aligned
        again, _ = rn.rmsnorm_kv4_attention(q, cache, plain.to(DEV), dl, q_starts=s)
        assert torch.equal(out, again)
        odd = torch.nn.functional.pad(q, (1, 1))[..., 1:1 + D]
        again, _ = rn.rmsnorm_kv4_attention(odd, cache, plain.to(DEV), dl, q_starts=s)
        assert torch.equal(out, again)
    finally:
        rn.set_kv4_test(0)


def test_decode_step_in_a_run():
    """Residual norm and q|k|v projection in one call, QK-norm, rotation and
    append, attention: three steps of two sequences, captured and eager, the
    cache growing by a token each; against the same in 64 bits from the
    projection's output on."""
    H, Hq, Hk, D, page, B = 896, 14, 2, 64, 16, 2
    A = normal((D * (Hq + 2 * Hk), H), BF16, 1, 0.03)
    w, wq, wk = normal((H,), BF16, 2, 0.1, 1.0), normal((D,), BF16, 3, 0.1, 1.0), normal((D,), BF16, 4, 0.1, 1.0)
    f = freqs(D)
    cache = make_cache(12, Hk, page, D, 9)
    ref_cache = cache.clone()
    table = torch.tensor([[3, 1, 4, 0, 5], [9, 2, 6, 11, 7]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([30, 63], dtype=torch.int32, device=DEV)
    x, r = normal((B, H), BF16, 5), normal((B, H), BF16, 6)
    pos, slots = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int64, device=DEV)
    torch.cuda.synchronize()

    def step(c):
        qkv, _, _ = rn.rmsnorm_gemv_fwd(x, w, A, r=r)
        heads = qkv.view(B, Hq + 2 * Hk, D)
        yq = rn.rmsnorm_rope_append_kv4(heads[:, Hq:Hq + Hk], heads[:, Hq + Hk:], pos, f, slots, c,
                                        q=heads[:, :Hq], wq=wq, wk=wk)
        out, _ = rn.rmsnorm_kv4_attention(yq, c, table, lens)
        return heads, yq, out

    def tokens():
        pos.copy_(lens)
        slots.copy_(table.gather(1, (lens // page).long()[:, None])[:, 0] * page + lens % page)
        lens.add_(1)

    start = lens.clone()
    tokens()
    step(ref_cache.clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step(cache)
    lens.copy_(start)
    cache.copy_(ref_cache)
    for i in range(3):
        x.copy_(normal((B, H), BF16, 50 + i))
        tokens()
        g.replay()
        heads, yq, out = step(ref_cache)
        torch.cuda.synchronize()
        assert torch.equal(cache, ref_cache) and torch.equal(captured[2], out)
        check_fwd(yq, heads[:, :Hq], wq, pos, f, False)
        check(out, None, yq, cache, table.cpu(), lens.tolist(), None)


@pytest.mark.parametrize("starts", [[0, 0, 0, 0], [5, 5, 5, 5], [9, 4, 2, 0]])
def test_sequences_without_rows(kernel, starts):
    """Starts that give no sequence a row: nothing is written."""
    cache = make_cache(6, 2, 16, 64, 3)
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(3, 2)
    q, out = normal((9, 4, 64), BF16, 1), torch.full((9, 4, 64), 5.0, dtype=BF16, device=DEV)
    rn.rmsnorm_kv4_attention(q, cache, table, torch.tensor([20, 30, 1], dtype=torch.int32, device=DEV),
                             q_starts=torch.tensor(starts, dtype=torch.int32, device=DEV), out=out)
    torch.cuda.synchronize()
    assert bool((out == 5).all())


def test_many_sequences_in_clusters():
    """More than 32 sequences, each a cluster of its own; lengths of all sorts."""
    B, Hk, page, blocks = 70, 2, 16, 30
    cache = make_cache(B * blocks, Hk, page, 64, 2)
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 481, (B,), generator=g).tolist()
    rn.set_kv4_test(3)
    try:
        run(B, Hk * 7, 64, BF16, cache, table_of(B, blocks, B * blocks, 6), lens)
    finally:
        rn.set_kv4_test(0)


def test_captured_piece_of_a_prompt():
    """Replayed with other lengths, starts and rows behind the last sequence."""
    D, page, Hk, G, T = 128, 64, 8, 4, 700
    cache = make_cache(60, Hk, page, D, 3)
    q = normal((T, Hk * G, D), BF16, 40)
    table = table_of(2, 30, 60, 1)
    lens = torch.tensor([1900, 1100], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 500, 690], dtype=torch.int32, device=DEV)
    dt = table.to(DEV)
    rn.rmsnorm_kv4_attention(q, cache, dt, lens, q_starts=starts)
    assert rn.last_path() == rn.PATH_KV4_PROMPT
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = rn.rmsnorm_kv4_attention(q, cache, dt, lens, q_starts=starts, want_lse=True)
    for new_lens, new_starts in (([1900, 1100], [0, 500, 690]), ([77, 1800], [3, 60, 700]), ([600, 0], [0, 600, 640])):
        lens.copy_(torch.tensor(new_lens, dtype=torch.int32))
        starts.copy_(torch.tensor(new_starts, dtype=torch.int32))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check(out, lse, q, cache, table, new_lens, new_starts)
        behind = torch.ones(T, dtype=torch.bool, device=DEV)
        behind[new_starts[0]:new_starts[2]] = False
        assert bool((out[behind] == 7).all()) and bool((lse[behind] == 7).all())


def test_first_calls_inside_a_capture():
    """In a process of its own, the library's very first calls are captured."""
    code = """
import torch
from rmsnorm_fwd_bwd_02_gb300 import rmsnorm as rn
dev = torch.device("cuda:0")
q, k = torch.randn(64, 4, 128, device=dev).bfloat16(), torch.randn(64, 2, 128, device=dev).bfloat16()
f, _ = rn.rope_frequencies(128, device=dev)
pos = torch.arange(64, device=dev)
cache = rn.kv4_cache(4, 2, 16, 128, device=dev)
table = torch.arange(4, dtype=torch.int32, device=dev)[None]
lens, starts = torch.tensor([64], dtype=torch.int32, device=dev), torch.tensor([0, 64], dtype=torch.int32, device=dev)
torch.cuda.synchronize()
def chain():
    y = rn.rmsnorm_rope_append_kv4(k, k, pos, f, pos, cache, q=q)
    a = rn.rmsnorm_kv4_attention(y[63:], cache, table, lens)[0]
    rn.set_kv4_test(2)
    b = rn.rmsnorm_kv4_attention(y, cache, table, lens, q_starts=starts)[0]
    rn.set_kv4_test(1)
    c = rn.rmsnorm_kv4_attention(y, cache, table, lens, q_starts=starts)[0]
    rn.set_kv4_test(0)
    return (a, b, c) + rn.rmsnorm_rope_bwd(q, q, pos, f, wq=q[0, 0].contiguous())[:1]
w = q[0, 0].contiguous()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = chain()
g.replay()
torch.cuda.synchronize()
want = chain()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, want))
print("fine")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
