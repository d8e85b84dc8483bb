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
