"""Waits of the chunk attention that run out: an error and NaN, no hang, and the next call is whole."""
import pytest
import torch

from bit_kv_cache_int2_gb300 import build as B
from bit_kv_cache_int2_gb300 import oscar

pytestmark = pytest.mark.gpu

from kv8_scenario import Pair  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    oscar.lib()


def call(p, q, k, v, out, lse, scratch):
    out.fill_(3.0)
    lse.fill_(3.0)
    oscar.oscar_prefill_kv8(p.ctx, p.cache, p.kind, q, k, v, q.shape[1], out, lse, scratch, q.shape[0])
    torch.cuda.synchronize()
    return oscar.oscar_get_error(p.ctx)


@pytest.mark.parametrize("kind", [oscar.KV8_E4M3, oscar.KV8_INT8])
@pytest.mark.parametrize("batch,n,Hkv,G,T", [(2, 3000, 2, 4, 5), (1, 0, 8, 1, 700), (1, 9000, 1, 8, 64), (30, 400, 2, 2, 70)])
def test_a_wait_that_runs_out_gives_nan(kind, batch, n, Hkv, G, T):
    p = Pair(kind, Hkv, G, batch, n // 64 + 2, seed=n, weights=False)
    try:
        if n:
            p.append(n, oracle=False)
        k, v = (x.cuda() for x in p.draw(T))
        q = torch.randn(batch, T, Hkv * G, 128, generator=p.g).bfloat16().cuda()
        out, lse = torch.empty_like(q), torch.empty(batch, T, Hkv * G, device="cuda")
        sc = oscar.alloc_scratch_kv8(p.cfg, prefill=True)
        assert call(p, q, k, v, out, lse, sc) == 0
        want, want_lse = out.clone(), lse.clone()
        oscar.oscar_set_option(p.ctx, oscar.OPT_WAIT_POLLS, 0)
        assert call(p, q, k, v, out, lse, sc) == oscar.ERR_TIMEOUT
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
        for polls in (1, 2, 5, 20, 100):  # some waits run out, or none: a row is whole or NaN
            oscar.oscar_set_option(p.ctx, oscar.OPT_WAIT_POLLS, polls)
            err = call(p, q, k, v, out, lse, sc)
            assert err in (0, oscar.ERR_TIMEOUT)
            bad = torch.isnan(out).all(-1)
            assert torch.equal(bad, torch.isnan(out).any(-1)) and torch.equal(bad, torch.isnan(lse))
            assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])
            assert err != 0 or not bool(bad.any())
        oscar.oscar_set_option(p.ctx, oscar.OPT_WAIT_POLLS, oscar.WAIT_POLLS_DEFAULT)
        assert call(p, q, k, v, out, lse, sc) == 0
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    finally:
        p.close()
