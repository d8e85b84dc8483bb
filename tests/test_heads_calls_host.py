"""CPU tier: refusals of the entry points on attention heads, beside those of
test_heads_host.py. Made-up addresses; every call below fails a check (or has
nothing to do), so nothing is launched."""
import pytest

from rmsnorm_fwd_bwd_02_gb300 import rmsnorm as rn
from tests.test_abi_host import ALIAS, OK, lib  # noqa: F401
from tests.test_heads_host import AT, append, append4, bwd, fwd, grad, heads


@pytest.mark.parametrize("n", [2, 4, 8])
def test_a_transposed_buffer_is_not_in_place(lib, n):  # noqa: F811
    """As many tokens as heads: a buffer and its transpose span the same bytes
    in rows of one width."""
    D = 64
    turned = {"y": AT[0], "y_token": D, "y_head": n * D, "n": n}
    k = {"x": AT[2], "y": AT[2], "y_token": D, "y_head": n * D, "n": n}
    assert fwd(lib, q=heads(**turned), T=n) == ALIAS
    assert fwd(lib, q=heads(n=n), k=heads(**k), T=n) == ALIAS
    # and the other way round: head-major inputs
    assert fwd(lib, q=heads(y=AT[0], x_token=D, x_head=n * D, n=n), T=n) == ALIAS
    for at in (AT[0], AT[1]):                                  # over dy, over x
        g = grad(dx=at, dx_token=D, dx_head=n * D, n=n)
        assert bwd(lib, q=g, T=n) == ALIAS
        other = {a: b for a, b in zip(("dy", "x", "w", "dw"), (AT[10], AT[11], AT[12], AT[13]))}
        over = AT[10] if at == AT[0] else AT[11]
        assert bwd(lib, q=grad(n=n), k=grad(**other, dx=over, dx_token=D, dx_head=n * D, n=n), T=n) == ALIAS
    for call in (append, append4):
        q = heads(x=AT[6], y=AT[6], y_token=D, y_head=n * D, n=n)
        assert call(lib, q=q, T=n) == ALIAS


def test_q_does_not_go_over_the_heads_scales(lib):  # noqa: F811
    """The append reads the scales while it writes q."""
    q = heads(x=AT[6], y=AT[7], n=4)
    for at in (AT[7], AT[7] + 8 * 4 * 64 * 2 - 4, AT[7] - 12):       # the first bytes, the last, half inside
        assert append4(lib, q=q, ks=at) == ALIAS
        assert append4(lib, q=q, vs=at) == ALIAS


def test_no_tokens_want_no_cache(lib):  # noqa: F811
    assert append4(lib, T=0, cache=None, slots=None) == OK
    assert append(lib, T=0, k=heads(x=None, y=None), v=heads(x=None, y=None), slots=None) == OK


@pytest.mark.parametrize("bad", [{"base": 1.0}, {"base": 0.5}, {"beta_fast": 0.0}, {"beta_slow": 0.0},
                                 {"beta_slow": -1.0}, {"original": 0}])
def test_yarn_refuses_what_has_no_logarithm(bad):
    """A base of one turns every pair alike: no pair turns so and so often."""
    args = {"rot": 64, "base": 1e4, "scaling": "yarn", "factor": 4.0, "original": 4096, "device": "cpu"}
    rn.rope_frequencies(**args)
    with pytest.raises(ValueError):
        rn.rope_frequencies(**{**args, **bad})
