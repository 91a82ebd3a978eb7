"""Attention of a chunk over 8-bit history where values or logits are very large, very small or far
apart, against the definition in 64 bits on the device's own state.

The limits are those of the ordinary chunks (test_gpu_kv8_prompt.limits): they are relative to
sum p |v|, whatever the values' size.  Of 32-bit sums below the smallest normal number half a step is
2^-150, which next to 2^-100 is nothing."""
import pytest
import torch

from bit_kv_cache_int2_gb300 import build as B
from bit_kv_cache_int2_gb300 import oscar

pytestmark = pytest.mark.gpu

from kv8_scenario import Pair  # noqa: E402
from test_gpu_kv8_prompt import check_chunk_dense, ok, prefill  # noqa: E402

KINDS = [oscar.KV8_E4M3, oscar.KV8_INT8]


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    oscar.lib()


def regions(L, T):
    """Where sink, history, window and chunk begin and end."""
    H = max(0, -(-(L - 320) // 16) * 16)
    s = min(L, 64)
    return [(0, s), (s, s + H), (s + H, L), (L, L + T)]


def sized(p, L, T, sizes, keys, sign, lead=0.0):
    """An appended prompt of L tokens and a chunk of T, values about 2^size in each region: of one sign or of both.
    lead: every query row looks at one region (in turn) or at all, whose logits are higher by so many nats."""
    g = torch.Generator().manual_seed(L + T)
    n, shape = L + T, (p.B, L + T, p.Hkv, 128)
    k = torch.randn(shape, generator=g) * keys
    v = torch.randn(shape, generator=g)
    if sign:
        v = v.abs() * 0.25 + 0.5
    q = torch.randn(p.B, T, p.Hkv * p.G, 128, generator=g)
    k[..., :4] = 0
    for i, (a, b) in enumerate(regions(L, T)):
        v[:, a:b] *= 2.0 ** sizes[i]
        k[:, a:b, :, i] = 8.0
    q[..., :4] = 0
    for t in range(T):
        if lead and t % 5 < 4:
            q[:, t, :, t % 5] = lead * 128 ** 0.5 / 8
    k, v, q = k.bfloat16(), v.bfloat16(), q.bfloat16()
    if L:
        p.append(L, (k[:, :L].contiguous(), v[:, :L].contiguous()), oracle=False)
    return q, k[:, L:].contiguous(), v[:, L:].contiguous()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lead", [60.0, 100.0, 210.0])
@pytest.mark.parametrize("G,T,L", [(4, 9, 700), (4, 32, 700), (1, 40, 500), (8, 3, 900)])
def test_rows_that_count_in_some_tiles_only(kind, lead, G, T, L):
    """Units that one CTA has whole, of one row tile: the two softmax groups have every other token tile each.
    Neighbouring rows look at different regions, by up to 2^300: what one group has counts for some rows
    of a warp and underflows for others."""
    p = Pair(kind, 8, G, 38, L // 64 + 2, seed=3, weights=False)
    try:
        q, k, v = sized(p, L, T, (0, 0, 0, 0), 0.3, False, lead)
        out, lse = prefill(p, q, k, v)
        n = slice(0, 3)
        check_chunk_dense(p, q[n], k[n], v[n], out[n], lse[n])
        ok(p)
    finally:
        p.close()
