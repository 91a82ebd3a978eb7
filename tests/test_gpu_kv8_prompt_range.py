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

from kv8_scenario import Pair, dense  # noqa: E402
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


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("L,T", [(0, 5), (0, 300), (40, 70), (700, 5), (700, 130), (3000, 300)])
@pytest.mark.parametrize("sizes", [(120, 120, 120, 120), (110, 110, 110, 110), (120, 0, 0, 0), (0, 0, 120, 0), (0, 0, 0, 120), (80, 80, 80, 80)])
def test_large_values(kind, L, T, sizes):
    """Finite values give finite rows: near-equal logits of values of one sign add up without an overflow."""
    for keys, sign in ((0.05, True), (1.0, False)):
        p = Pair(kind, 2, 4, 1, L // 64 + 2, seed=1, weights=False)
        try:
            q, k, v = sized(p, L, T, sizes, keys, sign)
            out, lse = prefill(p, q, k, v)
            assert bool(torch.isfinite(out).all())
            check_chunk_dense(p, q, k, v, out, lse)
            ok(p)
        finally:
            p.close()


def test_large_values_of_a_long_prompt(kind=oscar.KV8_INT8):
    p = Pair(kind, 1, 2, 1, 2, seed=1, weights=False)
    try:
        q, k, v = sized(p, 0, 8191, (0, 0, 0, 119), 0.05, True)
        out, lse = prefill(p, q, k, v)
        assert bool(torch.isfinite(out).all())
        check_chunk_dense(p, q, k, v, out, lse)
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes", [(0, 100, 0, 0), (0, 120, 0, 0), (60, 100, -60, 110), (-60, 110, 0, -60), (110, -60, 60, -60),
                                   (-60, 0, 110, 0), (0, 100, 100, -60), (60, 0, -60, 120)])
def test_values_of_sizes_very_far_apart(kind, sizes):
    """Each row within its own rounding, also where it looks at one region alone, by 2^300."""
    for (L, T), lead in (((700, 70), 210.0), ((700, 70), 40.0), ((2000, 5), 210.0), ((0, 40), 0.0), ((333, 40), 60.0)):
        p = Pair(kind, 1, 4, 1, L // 64 + 2, seed=2, weights=False)
        try:
            q, k, v = sized(p, L, T, sizes, 0.3, False, lead)
            out, lse = prefill(p, q, k, v)
            check_chunk_dense(p, q, k, v, out, lse)
            ok(p)
        finally:
            p.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [9, 64])
@pytest.mark.parametrize("sizes", [(120, 120, 120, 120), (80, 100, 80, 80), (0, 100, 100, -60), (0, 120, 0, 0), (0, 0, 120, 120),
                                   (100, -60, -60, -60), (-60, -60, 110, 0), (-60, 110, -60, 100)])
def test_whole_units(kind, T, sizes):
    """Enough requests for units that one CTA has whole: history and BF16 tokens in one running state."""
    for keys, sign, lead in ((0.05, True, 0.0), (0.3, False, 210.0), (0.3, False, 40.0)):
        p = Pair(kind, 8, 4, 38, 12, seed=3, weights=False)
        try:
            q, k, v = sized(p, 700, T, sizes, keys, sign, lead)
            out, lse = prefill(p, q, k, v)
            assert bool(torch.isfinite(out).all())
            n = slice(0, 3)
            check_chunk_dense(p, q[n], k[n], v[n], out[n], lse[n])
            ok(p)
        finally:
            p.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("L,T,batch", [(700, 9, 38), (700, 64, 38), (700, 9, 1), (3000, 130, 1), (100000, 4, 1)])
@pytest.mark.parametrize("size", [-90, -100])
def test_small_values(kind, L, T, batch, size):
    """The whole history (the others' values 0, or as small), in whole units and in split ones; near-equal logits."""
    for sizes in ((size,) * 4, (-140, size, -140, -140)):
        p = Pair(kind, 8 if batch > 1 else 1, 4, batch, L // 64 + 2, seed=4, weights=False)
        try:
            q, k, v = sized(p, L, T, sizes, 0.05, True)
            out, lse = prefill(p, q, k, v)
            n = slice(0, 3)
            check_chunk_dense(p, q[n], k[n], v[n], out[n], lse[n])
            ok(p)
        finally:
            p.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [9, 64])
@pytest.mark.parametrize("sizes", [(-100, 110, -100, -100), (110, -100, 60, -60), (-60, -100, 110, 0), (0, 100, 100, -100),
                                   (-100, 0, -60, 120), (-100, -100, -100, 0), (0, -100, -100, -100)])
def test_small_values_beside_others(kind, T, sizes):
    for batch, lead in ((38, 210.0), (38, 40.0), (1, 210.0)):
        p = Pair(kind, 8, 4, batch, 12, seed=5, weights=False)
        try:
            q, k, v = sized(p, 700, T, sizes, 0.3, False, lead)
            out, lse = prefill(p, q, k, v)
            n = slice(0, 2)
            check_chunk_dense(p, q[n], k[n], v[n], out[n], lse[n])
            ok(p)
        finally:
            p.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("a", [8, 9.5, 11, 12, 13, 14, 20, 45, 60])
@pytest.mark.parametrize("top", [0, 1, 2, 3, None])
def test_large_logits(kind, a, top):
    """Queries and keys with one channel, s 2^a and c 2^a: a logit is s c 2^2a / sqrt(128), c a quarter or more apart or
    the same.  Ties have the same weight, the others nothing (2^-2000).  A tie's weight has one rounding of P
    (BF16: 2^-8), the output another; the logit of the sum of exponentials, by which a row is divided, one of 2^-24
    of itself in 32 bits and the lse some more (scale, its product with two constants, the logit's, its own).
    Beyond 2^22 a row is NaN; where only some of its logits are beyond 2^21, it may be."""
    for batch, L, T in ((1, 700, 40), (19, 700, 9), (19, 420, 64), (1, 0, 130), (1, 3000, 5)):
        for positive in (False, True):
            g = torch.Generator().manual_seed(L + T)
            p = Pair(kind, 2 if batch == 1 else 8, 4, batch, L // 64 + 2, seed=6, weights=False)
            try:
                n, shape = L + T, (batch, L + T, p.Hkv)
                c = torch.randint(-4, 5, shape, generator=g).float()
                (h0, h1), places = regions(L, T)[1], regions(L, T)
                if h1 > h0:  # in the history a block has one key, of sizes that no other token has
                    c[:, h0:h1] = (torch.randint(-2, 3, (batch, (h1 - h0) // 16, p.Hkv), generator=g) * 2.5).repeat_interleave(16, 1)
                if top is not None and places[top][1] > places[top][0]:
                    b0, b1 = places[top]
                    c[:, b0:b1] = torch.where(c[:, b0:b1].abs() >= 4, c[:, b0:b1].sign() * 6, c[:, b0:b1])
                if positive:
                    c = c.abs() + 1
                    c[:, h0:h1] += 0.25
                k = torch.zeros(*shape, 128)
                k[..., 0] = c * 2.0 ** a if a % 1 == 0 else c * 2.0 ** (a - 0.5) * 1.5
                v = torch.randn(*shape, 128, generator=g)
                q = torch.zeros(batch, T, p.Hkv * 4, 128)
                q[..., 0] = (torch.randint(0, 2, q.shape[:3], generator=g) * 2 - 1) * 2.0 ** int(a)
                k, v, q = k.bfloat16(), v.bfloat16(), q.bfloat16()
                if L:
                    p.append(L, (k[:, :L].contiguous(), v[:, :L].contiguous()), oracle=False)
                k, v = k[:, L:].contiguous(), v[:, L:].contiguous()
                out, lse = prefill(p, q, k, v)
                hide = torch.arange(n, device="cuda") > L + torch.arange(T, device="cuda")[:, None, None]
                for h in range(p.Hkv):
                    K, V = (torch.cat([x, y[0, :, h].cuda().double()]) for x, y in zip(dense(p, 0, h), (k, v)))
                    mine = slice(4 * h, 4 * h + 4)
                    z = (q[0, :, mine].cuda().double() @ K.T / 128 ** 0.5).masked_fill(hide, -float("inf"))
                    w, rl = torch.softmax(z, 2), torch.logsumexp(z, 2)
                    o, ls = out[0, :, mine].double(), lse[0, :, mine].double()
                    nan = torch.isnan(ls)
                    assert torch.equal(torch.isnan(o).all(-1), nan) and torch.equal(torch.isnan(o).any(-1), nan)
                    assert bool(nan[rl.abs() > 2.0 ** 22].all())
                    size = z.masked_fill(hide, 0).abs().amax(2)
                    assert not bool(nan[size < 2.0 ** 21].any())
                    lim = (2.0 ** -7 + 2.0 ** -14 + 2.0 ** -22 * rl.abs())[..., None] * (w @ V.abs())
                    assert bool(((o - w @ V).abs() <= lim)[~nan].all()), h
                    assert bool(((ls - rl).abs() <= 2.0 ** -21 * rl.abs() + 2.0 ** -18)[~nan].all()), h
                ok(p)
            finally:
                p.close()
