"""Calls on the 8-bit cache's prompt side that have nothing to do need no arrays: no scratch either."""
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


@pytest.mark.parametrize("T,batch", [(0, 2), (5, 0), (0, 0)])
def test_nothing_to_do_needs_no_addresses(T, batch):
    p = Pair(oscar.KV8_INT8, 2, 2, 2, 4, weights=False)
    try:
        before = {x: p.cache[x].clone() for x in p.cache}
        oscar.oscar_prefill_kv8(p.ctx, p.cache, p.kind, None, None, None, T, None, None, None, batch)
        oscar.bind_prefill_kv8(p.ctx, p.cache, p.kind, None, None, None, T, None, None, None, batch)()
        small = torch.zeros(256, dtype=torch.uint8, device="cuda")
        oscar.oscar_prefill_kv8(p.ctx, p.cache, p.kind, None, None, None, T, None, None, small[8:], batch)
        for kind, t, b in ((2, T, batch), (1, -1, batch), (1, T, 3)):  # arguments that are there are checked all the same
            with pytest.raises(oscar.OscarError) as e:
                oscar.oscar_prefill_kv8(p.ctx, p.cache, kind, None, None, None, t, None, None, None, b)
            assert e.value.status == oscar.ERR_INVALID_ARG
        q = torch.zeros(2, 5, 4, 128, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(oscar.OscarError) as e:  # with something to do there has to be scratch
            oscar.oscar_prefill_kv8(p.ctx, p.cache, p.kind, q, q, q, 5, q.clone(), None, None, 1)
        assert e.value.status == oscar.ERR_INVALID_ARG
        torch.cuda.synchronize()
        assert oscar.oscar_get_error(p.ctx) == 0
        for x in before:
            assert torch.equal(before[x].view(torch.uint8), p.cache[x].view(torch.uint8)), x
    finally:
        p.close()
