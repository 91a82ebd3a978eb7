"""What the 8-bit cache's calls leave behind when they cannot do their work."""
import pytest
import torch

from bit_kv_cache_int2_gb300 import build as B
from bit_kv_cache_int2_gb300 import oscar

pytestmark = pytest.mark.gpu

from kv8_scenario import Pair, check_decode  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    oscar.lib()


@pytest.mark.parametrize("kind", [oscar.KV8_E4M3, oscar.KV8_INT8])
@pytest.mark.parametrize("batch,n,Hkv,G", [(2, 3000, 2, 4), (40, 700, 8, 1), (1, 5, 1, 8)])
def test_a_wait_that_runs_out_leaves_weights_and_gives_nan(kind, batch, n, Hkv, G):
    """With no polls no piece of the cache is ever there: every output and lse is
    NaN, whatever an earlier call left in the scratch, the weights stay, and the
    next decode with polls is as ever."""
    p = Pair(kind, Hkv, G, batch, -(-n // 64), seed=batch)
    try:
        p.append(n)
        q = p.query()
        out, lse = p.decode(q, 1.0)
        check_decode(p, q, out, lse, 1.0)
        before = p.weights.clone()
        oscar.oscar_set_option(p.ctx, oscar.OPT_WAIT_POLLS, 0)
        for _ in range(2):
            out, lse = p.decode(p.query(), 0.5)
            assert oscar.oscar_get_error(p.ctx) == oscar.ERR_TIMEOUT
            assert torch.equal(p.weights, before)
            assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
        oscar.oscar_set_option(p.ctx, oscar.OPT_WAIT_POLLS, oscar.WAIT_POLLS_DEFAULT)
        out, lse = p.decode(q, 0.5)
        worst = check_decode(p, q, out, lse, 0.5)
        p.check_state(weight_tol=4 * worst)
        assert oscar.oscar_get_error(p.ctx) == 0
    finally:
        p.close()


@pytest.mark.parametrize("polls", [1, 3, 10, 30, 100])
def test_a_wait_that_may_run_out_takes_whole_heads(polls, kind=oscar.KV8_INT8):
    """Whichever waits run out: a (request, head) is lost with its weights as they
    were, or has its result."""
    p = Pair(kind, 4, 4, 6, 47, seed=5)
    try:
        p.append(3000)
        q = p.query()
        good, good_lse = p.decode(q, 1.0)
        base = p.weights.clone()
        good, good_lse = p.decode(q, 1.0)
        good_w = p.weights.clone()
        for _ in range(5):
            p.weights.copy_(base)
            oscar.oscar_set_option(p.ctx, oscar.OPT_WAIT_POLLS, polls)
            out, lse = p.decode(q, 1.0)
            err = oscar.oscar_get_error(p.ctx)
            oscar.oscar_set_option(p.ctx, oscar.OPT_WAIT_POLLS, oscar.WAIT_POLLS_DEFAULT)
            lost = torch.isnan(lse.view(6, 4, 4))
            assert torch.equal(lost.all(-1), lost.any(-1))
            lost = lost[..., 0]
            assert err == (oscar.ERR_TIMEOUT if bool(lost.any()) else 0)
            o, g = out.view(6, 4, -1), good.view(6, 4, -1)
            assert bool(torch.isnan(o[lost]).all()) and torch.equal(o[~lost], g[~lost])
            assert torch.equal(lse.view(6, 4, 4)[~lost], good_lse.view(6, 4, 4)[~lost])
            assert torch.equal(p.weights[lost], base[lost]) and torch.equal(p.weights[~lost], good_w[~lost])
    finally:
        p.close()


def test_calls_without_tokens_or_requests(kind=oscar.KV8_E4M3):
    """Tensors without elements have no address: the last, empty chunk of a prompt,
    or a step in which no request is active, is nothing to do and no error."""
    p = Pair(kind, 2, 2, 2, 12, seed=3)
    try:
        p.append(400)
        k = torch.zeros(2, 400, 2, 128, dtype=torch.bfloat16, device="cuda")
        q = torch.zeros(0, 4, 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(0, 4, device="cuda")
        assert k[:, 400:].data_ptr() == 0 and q.data_ptr() == 0
        oscar.oscar_append_kv8(p.ctx, p.cache, kind, k[:, 400:], k[:, 400:], 0, 2, weights=p.weights)
        oscar.oscar_append_kv8(p.ctx, p.cache, kind, k[:0], k[:0], 400, 0, weights=p.weights)
        oscar.oscar_decode_kv8(p.ctx, p.cache, kind, q, torch.empty_like(q), lse, p.scratch, 0, weights=p.weights)
        p.check_state()
        assert oscar.oscar_get_error(p.ctx) == 0
    finally:
        p.close()
