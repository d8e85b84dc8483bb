"""GPU tier: calls on attention heads that their documentation allows beside
those of the other files: failed waits, small outputs that are saved, far ends
of the number range, frequencies of any size, parts without heads.

Tolerances as in test_rope_gpu.py and test_kv4_attention_gpu.py, or derived
beside the test.
"""
import io
import math
from fractions import Fraction

import pytest
import torch

from rmsnorm_fwd_bwd_02_gb300 import autograd
from rmsnorm_fwd_bwd_02_gb300 import rmsnorm as rn
from tests.test_kv4_attention_gpu import check, dense, make_cache, table_of
from tests.test_rope_gpu import (BF16, DEV, F16, F32, F64, PI, ULP, check_bwd, check_fwd, close, freqs, half_step,
                                 normal, turn)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tier needs a CUDA device")
    rn.lib()
    rn.wait_timeouts(reset=True)
    yield
    assert rn.wait_timeouts(reset=True) == 0


@pytest.mark.parametrize("T,H", [(8, 8), (8, 1), (1, 8), (1, 1)])
@pytest.mark.parametrize("head_major", [False, True])
def test_in_place_where_tokens_and_heads_are_as_many(T, H, head_major):
    """Outputs that are their inputs exactly, whatever stride a direction of
    one step has."""
    D = 128
    f, pos, w = freqs(D), torch.arange(T, device=DEV) * 7, normal((D,), BF16, 2, 0.1, 1.0)
    base = normal((T, H, D), BF16, 3)
    x = (base.transpose(0, 1) if head_major else base).clone(memory_format=torch.contiguous_format)
    x = x.transpose(0, 1) if head_major else x
    y = torch.as_strided(x, x.shape, (x.stride(0) if T > 1 else 5 * D, x.stride(1) if H > 1 else 3 * D, 1))
    rn.rmsnorm_rope_fwd(x, pos, f, wq=w, yq=y)
    check_fwd(x, base, w, pos, f, False)
    dy = normal((T, H, D), BF16, 4)
    g = torch.empty_strided(x.shape, x.stride(), dtype=BF16, device=DEV).copy_(dy)
    dq, _, dw, _ = rn.rmsnorm_rope_bwd(g, base, pos, f, wq=w, dq=g)
    assert dq is g
    check_bwd(dy, base, w, g, dw, pos, f, False)


@pytest.mark.parametrize("D", [64, 128])
def test_pieces_of_prompts_between_other_tensor_memory_kernels(D):
    """Calls that allocate tensor memory, one right behind the other on a
    stream, each launched while the one before it ends."""
    Hk, G, page, T = 2, 4, 16, 400
    cache = make_cache(60, Hk, page, D, 3)
    q = normal((T, Hk * G, D), BF16, 1)
    table = torch.arange(60, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([900], dtype=torch.int32, device=DEV)
    s = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    x, wn, W = normal((16, 512), BF16, 2), normal((512,), BF16, 3, 0.1, 1.0), normal((1024, 512), BF16, 4)
    Wq, Ws = rn.rmsnorm_quant_fp8(W, block_rows=128)
    xq, xs = rn.rmsnorm_fwd_fp8(x, wn)[:2]
    torch.cuda.synchronize()
    rn.set_kv4_test(2)
    try:
        def chain():
            a = rn.rmsnorm_kv4_attention(q, cache, table, lens, q_starts=s)[0]
            b = rn.rmsnorm_gemm_fp8(xq, xs, Wq, Ws)
            c = rn.rmsnorm_kv4_attention(q, cache, table, lens, q_starts=s)[0]
            d = rn.rmsnorm_gemv_fwd(x, wn, W)[0]
            return a, b, c, d
        want = [t.clone() for t in chain()]
        torch.cuda.synchronize()
        for _ in range(20):
            got = chain()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        check(want[0], None, q, cache, table.cpu(), [900], [0, T])
    finally:
        rn.set_kv4_test(0)


@pytest.mark.parametrize("kernel", [1, 3, 2], ids=["list", "clusters", "prompt"])
@pytest.mark.parametrize("B,Hk", [(1, 1), (60, 4)])
def test_rows_whose_waits_run_out_are_not_written(kernel, B, Hk):
    """The test hook makes every stage's wait run out: the rows keep what was
    there, whatever the workspace held. One sequence is split over many warps;
    of sixty a warp has several, and parts of some."""
    D, page, blocks = 128, 16, 60 if B == 1 else 6
    cache = make_cache(B * blocks, Hk, page, D, 3)
    table = table_of(B, blocks, B * blocks, 1).to(DEV)
    g = torch.Generator().manual_seed(3)
    most = blocks * page
    lens = torch.randint(most // 2, most + 1, (B,), generator=g).to(torch.int32).to(DEV)
    n = 1 if kernel == 3 or B > 1 else 2
    q = normal((B * n, Hk * 4, D), BF16, 4)
    s = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV)
    out, lse = torch.full_like(q, 3.0), torch.full((B * n, Hk * 4), 4.0, device=DEV)
    ws = torch.ones(rn.lib().rmsnorm_kv4_attention_workspace_bytes(D) // 4, device=DEV)
    rn.wait_timeouts(reset=True)
    rn.set_kv4_test(kernel)
    rn.set_stream_test_fault(16, 2000)
    try:
        rn.rmsnorm_kv4_attention(q, cache, table, lens, q_starts=s, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
    finally:
        rn.set_stream_test_fault(0, 0)
    try:
        assert rn.wait_timeouts(reset=True) > 0
        assert bool((out == 3).all()) and bool((lse == 4).all())
        rn.rmsnorm_kv4_attention(q, cache, table, lens, q_starts=s, out=out, lse=lse, workspace=ws)
        check(out, lse, q, cache, table.cpu(), lens.tolist(), s.tolist())
    finally:
        rn.set_kv4_test(0)


def saved(**tensors):
    f = io.BytesIO()
    torch.save(tensors, f)
    f.seek(0)
    back = torch.load(f)
    assert all(torch.equal(back[k], t) for k, t in tensors.items())


def test_small_outputs_can_be_saved_together():
    """torch.save refuses tensors of two types in one storage."""
    T, D = 5, 64
    q, k, w = normal((T, 4, D), BF16, 1), normal((T, 2, D), BF16, 2), normal((D,), BF16, 3, 0.1, 1.0)
    f, pos = freqs(D), torch.arange(T, device=DEV)
    yq, yk, rstd = rn.rmsnorm_rope_fwd(q, pos, f, k=k, wq=w, wk=w)
    saved(yq=yq, yk=yk, rstd=rstd)
    dq, dk, dwq, dwk = rn.rmsnorm_rope_bwd(q, q, pos, f, dyk=k, k=k, wq=w, wk=w, rstd=rstd)
    saved(dq=dq, dk=dk, dwq=dwq, dwk=dwk)
    cache = make_cache(4, 2, 16, D, 3)
    out, lse = rn.rmsnorm_kv4_attention(q[:1], cache, torch.arange(4, dtype=torch.int32, device=DEV)[None],
                                        torch.tensor([50], dtype=torch.int32, device=DEV), want_lse=True)
    saved(out=out, lse=lse)


@pytest.mark.parametrize("size", [1e-18, 1e-15, 1e-13, 1e13, 1e16, 1e18])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keep", [False, True])
def test_backward_over_the_number_range(size, dtype, keep):
    """Rows whose 1 / rms cubed leaves fp32's range, with eps 0: as test_rope_gpu's
    backward bound."""
    T, H, D = 9, 3, 128
    f, pos, w = freqs(D), torch.arange(T, device=DEV) * 3, normal((D,), dtype, 1, 0.1, 1.0)
    x, dy = normal((T, H, D), dtype, 2, size), normal((T, H, D), dtype, 3)
    rstd = rn.rmsnorm_rope_fwd(x, pos, f, wq=w, eps=0.0)[2]
    dx, _, dw, _ = rn.rmsnorm_rope_bwd(dy, x, pos, f, wq=w, rstd=rstd if keep else None, eps=0.0)
    x64, w64 = x.to(F64), w.to(F64)
    r = 1 / torch.sqrt((x64 * x64).mean(-1, keepdim=True))
    g, mag = turn(dy.to(F64), pos, f, False, back=True)
    want = r * (w64 * g - x64 * r * r * (w64 * g * x64).mean(-1, keepdim=True))
    terms = r * (w64.abs() * mag + x64.abs() * r * r * (w64.abs() * mag * x64.abs()).mean(-1, keepdim=True))
    close(dx, want, 64 * ULP * terms + half_step(want, dtype))
    close(dw, (g * x64 * r).sum((0, 1)), (T * H / 64 + 128) * ULP * (mag * (x64 * r).abs()).sum((0, 1)))


def test_frequencies_of_any_size():
    """The header's bound against exact rational arithmetic: an angle is within
    |position| 2^-64 + 2^-32 of a turn for |freq| up to 2^64."""
    freq = [1e9, -(2.0 ** 40), 12345.678, 1e6 / 3, 2 * math.pi * 2 ** 30, 3e15, 2.0 ** 63, 1e-9]
    pos = [1, 1 << 20, (1 << 20) + 1, 1 << 40, -(1 << 33) - 5, -77, 1 << 45, 999999937]
    f = torch.tensor(freq, dtype=F64, device=DEV)
    for adjacent in (False, True):
        x = normal((len(pos), 2, 16), F32, 7)
        y, _, _ = rn.rmsnorm_rope_fwd(x, torch.tensor(pos, device=DEV), f, interleaved=adjacent)
        for i, t in enumerate(pos):
            angle = torch.tensor([float(Fraction(w) * t / (2 * PI) % 1 * 2 * PI) for w in freq], dtype=F64,
                                 device=DEV)
            want, size = turn(x[i:i + 1].to(F64), torch.ones(1, device=DEV), angle, adjacent)
            off = (abs(t) * 2.0 ** -64 + 2.0 ** -32) * 2 * math.pi
            close(y[i:i + 1], want, (24 * ULP + off) * size)


@pytest.mark.parametrize("norm_q", [False, True])
def test_gradient_of_a_norm_without_heads(norm_q):
    """k with no heads: its weight's gradient is a sum over nothing."""
    T, D = 6, 64
    q, k, w = normal((T, 2, D), BF16, 1), torch.empty(T, 0, D, dtype=BF16, device=DEV), normal((D,), BF16, 2, 0.1, 1.0)
    f, pos = freqs(D), torch.arange(T, device=DEV)
    wq = w if norm_q else None
    # what the gradients' allocation held before
    junk = [torch.full((n,), float("nan"), device=DEV) for n in (64, 128, 256, 512)]
    torch.cuda.synchronize()
    del junk
    dq, dk, dwq, dwk = rn.rmsnorm_rope_bwd(q, q if norm_q else None, pos, f, dyk=k, k=k, wq=wq, wk=w)
    assert dk.shape == k.shape and bool((dwk == 0).all())
    check_bwd(q, q, wq, dq, dwq, pos, f, False)


def test_parts_without_heads():
    """k, or the append's q, with no heads, made by the call or windows of
    another tensor."""
    T, D = 6, 64
    x, w = normal((T, 5, D), BF16, 1), normal((D,), BF16, 2, 0.1, 1.0)
    f, pos = freqs(D), torch.arange(T, device=DEV)
    for none in (torch.empty(T, 0, D, dtype=BF16, device=DEV), x[:, 5:], x[:, 2:2].transpose(0, 1)[:0].transpose(0, 1)):
        yq, yk, rstd = rn.rmsnorm_rope_fwd(x, pos, f, k=none, wq=w, wk=w)
        check_fwd(yq, x, w, pos, f, False)
        assert yk.shape == (T, 0, D) and rstd.shape == (T, 5)
        leaves = [t.clone().requires_grad_() for t in (x, none, w, w)]
        yq, yk = autograd.rms_norm_rope(*leaves[:2], pos, f, *leaves[2:])
        yq.backward(x)
        check_bwd(x, x, w, leaves[0].grad, rn.rmsnorm_rope_bwd(x, x, pos, f, wq=w)[2], pos, f, False)
        assert bool((leaves[3].grad == 0).all())
        cache = rn.kv4_cache(1, 5, 16, D, device=DEV)
        assert rn.rmsnorm_rope_append_kv4(x, x, pos, f, pos, cache, q=none).shape == (T, 0, D)
        again = rn.kv4_cache(1, 5, 16, D, device=DEV)
        rn.rmsnorm_rope_append_kv4(x, x, pos, f, pos, again)
        assert torch.equal(cache, again) and bool(cache.any())


def test_autograd_gives_each_leaf_its_own_gradient():
    T, Hq, Hk, D = 19, 4, 2, 64
    f, pos = freqs(32), torch.arange(T, device=DEV) * 11
    for interleaved in (False, True):
        q, k = normal((T, Hq, D), F32, 20).requires_grad_(), normal((T, Hk, D), F32, 21).requires_grad_()
        wq, wk = normal((D,), F32, 22, 0.3, 1.0).requires_grad_(), normal((D,), F32, 23, 0.3, 2.0).requires_grad_()
        dyq, dyk = normal((T, Hq, D), F32, 24), normal((T, Hk, D), F32, 25)
        yq, yk = autograd.rms_norm_rope(q, k, pos, f, wq, wk, interleaved=interleaved, amplitude=1.25)
        torch.autograd.backward([yq, yk], [dyq, dyk])
        for x, w, y, dy in ((q, wq, yq, dyq), (k, wk, yk, dyk)):
            check_fwd(y.detach(), x.detach(), w.detach(), pos, f, interleaved, 1.25)
            check_bwd(dy, x.detach(), w.detach(), x.grad, w.grad, pos, f, interleaved, 1.25)
        # outputs that nothing uses: zeros for what depends on them alone
        for used in (0, 1):
            leaves = [t.detach().clone().requires_grad_() for t in (q, k, wq, wk)]
            y = autograd.rms_norm_rope(*leaves[:2], pos, f, *leaves[2:], interleaved=interleaved, amplitude=1.25)
            y[used].backward((dyq, dyk)[used])
            for i, (leaf, whole) in enumerate(zip(leaves, (q, k, wq, wk))):
                if i % 2 == used:
                    assert torch.equal(leaf.grad, whole.grad)
                else:
                    assert bool((leaf.grad == 0).all())


@pytest.mark.parametrize("kernel", [1, 3], ids=["list", "clusters"])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_of_fp16_rows_keep_their_second_half(kernel, D):
    """Weights that are nearly equal over values of both signs: a row is small
    beside the sum of p |v|, and so is its own rounding; a weight rounded to
    fp16 would show. q has four features that are not zero, so a score is a
    sum of four products, each within 8 2^-24 of itself with the factors'
    roundings; less the reference it is rounded at 8, 2^-21; exp2 2^-22; the
    halves together 2^-22: below 2^-19 of the weight, and twice that for the
    quotient. Both halves of 32 tokens are four MMAs, each within 17 2^-23 of
    its magnitudes."""
    B, Hk, G, page, L = 6, 2, 4, 16, 32
    cache = rn.kv4_cache(B * 2, Hk, page, D, device=DEV)
    n = B * 2 * page
    k = normal((n, Hk, D), F32, 1)
    size = normal((n // 2, Hk, D), F32, 2)
    v = torch.stack([size, -size], dim=1).flatten(0, 1)
    rn.rmsnorm_rope_append_kv4(k, v, None, None, torch.arange(n, device=DEV), cache)
    q = torch.zeros(B, Hk * G, D, dtype=F16, device=DEV)
    q[..., 3::D // 4] = normal((B, Hk * G, 4), F16, 3, 0.03)
    table = torch.arange(B * 2, dtype=torch.int32).view(B, 2)
    rn.set_kv4_test(kernel)
    try:
        out, _ = rn.rmsnorm_kv4_attention(q, cache, table.to(DEV), torch.full((B,), L, dtype=torch.int32, device=DEV))
    finally:
        rn.set_kv4_test(0)
    kk, vv = (t.to(DEV) for t in dense(cache, D))
    kk, vv = (t[table.to(DEV).long()].transpose(1, 2).reshape(B, Hk, L, D) for t in (kk, vv))
    x = torch.einsum("bhgd,bhld->bhgl", q.to(F64).view(B, Hk, G, D), kk) / math.sqrt(D)
    p = torch.exp(x - x.amax(-1, keepdim=True))

    def row(weights):
        return torch.einsum("bhgl,bhld->bhgd", weights, vv) / p.sum(-1, keepdim=True)

    want, mag = row(p), torch.einsum("bhgl,bhld->bhgd", p, vv.abs()) / p.sum(-1, keepdim=True)
    tol = (2 * 2.0 ** -19 + 4 * 17 * 2.0 ** -23) * mag + half_step(want, F16)
    close(out.view_as(want), want, tol)
    # the bound would show weights of one half
    one = row((p * 256).to(F16).to(F64) / 256)
    assert float(((one - want).abs() > tol).double().mean()) > 0.3


@pytest.mark.parametrize("byte", [0x7F, 0x80, 0xF8])
@pytest.mark.parametrize("kernel", [1, 3, 2], ids=["list", "clusters", "prompt"])
def test_bytes_behind_a_sequence_change_nothing(kernel, byte):
    """Whole tiles behind the end, and a page that the table does not reach,
    filled with bytes that are NaN or extreme as scales."""
    D, page, Hk = 64, 48, 2
    cache = make_cache(6, Hk, page, D, 7)
    table = torch.tensor([[3, 5], [2, 4]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([64, 41], dtype=torch.int32, device=DEV)     # 64: page 5's first tile; 41: page 2's third
    s = torch.tensor([0, 3, 5], dtype=torch.int32, device=DEV)
    q = normal((5, 4, D), BF16, 1)
    bad = cache.clone()
    bad[5, :, 1:], bad[4], bad[0], bad[1] = byte, byte, byte, byte
    rn.set_kv4_test(kernel)
    try:
        a, la = rn.rmsnorm_kv4_attention(q, cache, table, lens, q_starts=s, want_lse=True)
        b, lb = rn.rmsnorm_kv4_attention(q, bad, table, lens, q_starts=s, want_lse=True)
    finally:
        rn.set_kv4_test(0)
    assert torch.equal(a, b) and torch.equal(la, lb)
    check(a, la, q, cache, table.cpu(), [64, 41], [0, 3, 5])


def test_starts_that_give_every_row_to_thousands_of_sequences():
    """Starts that run back and forth: the rows of 2048 sequences each make
    more than 2^32 entries together, and nothing is written. Then the same
    rows once."""
    B, T, Hk, G, D, page, blocks = 4096, 1 << 14, 8, 4, 64, 16, 125
    cache = make_cache(2, Hk, page, D, 3)
    table = torch.zeros(B, blocks, dtype=torch.int32, device=DEV)
    lens = torch.full((B,), blocks * page, dtype=torch.int32, device=DEV)
    tiles, cost = T * G // 8, blocks * page // 32 + 3
    assert B // 2 * tiles * Hk * cost >= 1 << 32
    s = torch.tensor([0, T], dtype=torch.int32, device=DEV).repeat(B // 2 + 1)[:B + 1].contiguous()
    q = normal((T, Hk * G, D), BF16, 1)
    out, lse = torch.full_like(q, 3.0), torch.full((T, Hk * G), 4.0, device=DEV)
    rn.rmsnorm_kv4_attention(q, cache, table, lens, q_starts=s, out=out, lse=lse)
    assert rn.last_path() == rn.PATH_KV4_ATTENTION
    torch.cuda.synchronize()
    assert bool((out == 3).all()) and bool((lse == 4).all())
    s = (torch.arange(B + 1, device=DEV) * (T // B)).to(torch.int32)
    rn.rmsnorm_kv4_attention(q, cache, table, lens, q_starts=s, out=out, lse=lse)
    assert rn.last_path() == rn.PATH_KV4_ATTENTION
    first = 8
    check(out[:first * 4], lse[:first * 4], q[:first * 4], cache, table[:first].cpu(), [blocks * page] * first,
          s[:first + 1].tolist())
    # every sequence sees the same tokens
    assert bool(torch.isfinite(lse).all())
