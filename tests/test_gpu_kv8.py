"""The 8-bit-history cache on the GPU against the 64-bit oracle: appended state
bit for bit, attention and block weights within rounding, eviction exactly."""
import numpy as np
import pytest
import torch

from bit_kv_cache_int2_gb300 import build as B
from bit_kv_cache_int2_gb300 import oscar

pytestmark = pytest.mark.gpu

from kv8_scenario import Pair, check_decode, check_decode_dense  # noqa: E402

KINDS = [oscar.KV8_E4M3, oscar.KV8_INT8]


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    oscar.lib()


def ok(p):
    assert oscar.oscar_get_error(p.ctx) == 0


# -------------------------------------------------------------------- append
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hkv,steps", [
    (1, [1] * 40),
    (2, [63, 1, 1, 14, 1, 1, 175, 1, 63, 1, 1, 16, 1, 1]),        # borders of sink, block and window
    (3, [320, 1, 1, 15, 16, 17, 240, 1]),
    (8, [337, 1, 64, 1, 5]),
    (2, [700, 3, 255, 256, 257, 1]),
    (1, [64, 256, 272, 1, 1000, 31]),
    (5, [79, 250, 33, 300]),
])
def test_append_leaves_the_oracles_state(kind, Hkv, steps):
    p = Pair(kind, Hkv, 1, 2, 40, seed=len(steps))
    try:
        for T in steps:
            p.append(T)
            p.check_state()
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("kind", KINDS)
def test_append_requests_of_different_lengths(kind):
    p = Pair(kind, 2, 2, 6, 30, seed=5)
    try:
        lens = [0, 1, 64, 320, 333, 900]
        for b, n in enumerate(lens):  # each alone, into its row
            if n:
                one = Pair.draw(p, n, B=1)
                row = {x: p.cache[x][b:b + 1] if x != "pool" else p.cache[x] for x in p.cache}
                oscar.oscar_append_kv8(p.ctx, row, kind, one[0].cuda(), one[1].cuda(), n, 1,
                                       weights=p.weights[b:b + 1])
                for t in range(n):
                    p.req[b].append(one[0][0, t].double().numpy(), one[1][0, t].double().numpy())
        p.check_state()
        for T in (1, 1, 70, 1):
            p.append(T)
            p.check_state()
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("kind", KINDS)
def test_append_quantises_extremes_and_ties(kind):
    """Zeros, tiny and huge magnitudes, exact ties, one infinity and one NaN."""
    p = Pair(kind, 2, 1, 1, 12)
    try:
        k, v = p.draw(64 + 256 + 160)
        at = 64
        k[0, at:at + 16] = 0
        v[0, at:at + 16] = 2.0 ** -120                      # below the smallest scale
        k[0, at + 16:at + 32] = (torch.arange(16 * 128 * 2).view(16, 2, 128) % 509 - 254).bfloat16()
        k[0, at + 16, 0, 0] = 254.0                         # int8: step 2, odd numbers are ties
        v[0, at + 16:at + 32] = (torch.arange(16 * 128 * 2).view(16, 2, 128) % 257).bfloat16() * 1.75
        v[0, at + 16, :, 0] = 448.0
        k[0, at + 32:at + 48] = 3.38e38
        v[0, at + 32:at + 48] *= 2.0 ** 120
        k[0, at + 48, 0, 5] = float("inf")
        v[0, at + 49, 1, 7] = float("nan")
        v[0, at + 64:at + 80] = 2.0 ** -133                 # subnormal
        k[0, at + 64, 0, 3] = 2.0 ** -99
        p.append(k.shape[1], (k, v))
        p.check_state()
        ok(p)
    finally:
        p.close()


def test_append_refuses_a_request_and_leaves_it(kind=oscar.KV8_INT8):
    """A missing page, a bad one, too few pages and impossible lengths: those
    requests stay as they were, the others get their tokens."""
    p = Pair(kind, 2, 1, 5, 8, seed=2)
    try:
        p.append(320 + 96)
        table, hist, seq = (p.cache[x] for x in ("page_table", "hist_lens", "seq_lens"))
        table[0, 1] = -1
        table[1, 3] = p.cfg.num_pages
        seq[3] = 5000  # a window of 4840 tokens
        hist[4] += 8
        before = {x: p.cache[x].clone() for x in p.cache}
        wb = p.weights.clone()
        k, v = p.draw(150)
        p.append(150, (k, v), oracle=False)
        assert oscar.oscar_get_error(p.ctx) in (oscar.ERR_NO_PAGE, oscar.ERR_RANGE, oscar.ERR_STATE)
        for b in (0, 1, 3, 4):
            for x in ("sink_k", "sink_v", "ring_k", "ring_v", "seq_lens", "hist_lens"):
                assert torch.equal(p.cache[x][b:b + 1].view(torch.uint8), before[x][b:b + 1].view(torch.uint8)), (b, x)
            assert torch.equal(p.weights[b], wb[b])
        r = p.req[2]
        for t in range(150):
            r.append(k[2, t].double().numpy(), v[2, t].double().numpy())
        assert (int(seq[2]), int(hist[2])) == (r.L, r.H)
        p.cache["page_table"].copy_(before["page_table"])
        p.append(600, oracle=False)  # beyond 8 pages
        assert oscar.oscar_get_error(p.ctx) != 0
        assert int(seq[2]) == r.L
    finally:
        p.close()


# -------------------------------------------------------------------- decode
LENGTHS = [0, 1, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 79, 80, 81, 96, 319, 320, 321, 335, 336, 337, 352, 384, 385,
           400, 641, 1000, 1601]


def lengths_pair(kind, Hkv, G, lens, seed=0, weights=True, scale=1.0):
    p = Pair(kind, Hkv, G, len(lens), max(1, -(-max(lens) // 64)), seed=seed, weights=weights)
    for b, n in enumerate(lens):
        if n:
            k, v = p.draw(n, scale, B=1)
            row = {x: p.cache[x][b:b + 1] if x != "pool" else p.cache[x] for x in p.cache}
            oscar.oscar_append_kv8(p.ctx, row, kind, k.cuda(), v.cuda(), n, 1,
                                   weights=p.weights[b:b + 1] if weights else None)
            kn, vn = k.double().numpy(), v.double().numpy()
            for t in range(n):
                p.req[b].append(kn[0, t], vn[0, t])
    return p


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 2), (2, 4), (1, 8), (3, 4)])
def test_decode_matches_the_oracle(kind, Hkv, G):
    p = lengths_pair(kind, Hkv, G, LENGTHS, seed=Hkv * 10 + G)
    try:
        for step, decay in enumerate((1.0, 0.9)):
            q = p.query(1.5)
            out, lse = p.decode(q, decay)
            worst = check_decode(p, q, out, lse, decay)
            p.check_state(weight_tol=2 * worst)
        q = p.query()
        plain = p.decode(q, weights=False)
        check_decode(p, q, *plain)
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("kind", KINDS)
def test_decode_long_and_uneven(kind):
    p = lengths_pair(kind, 2, 4, [9000, 3, 0, 20011, 400], seed=3)
    try:
        q = p.query(2.0)
        out, lse = p.decode(q, 1.0)
        worst = check_decode(p, q, out, lse, 1.0)
        p.check_state(weight_tol=2 * worst)
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("kind,Hkv,G,lens", [
    (0, 1, 8, [200000]),             # over a thousand pages per CTA's turns of the stage ring
    (1, 2, 4, [150000, 131071]),
    (0, 8, 2, [40000, 100, 0, 70001, 65]),
    (1, 8, 1, [3000] * 40),          # several requests per CTA
    (0, 4, 4, [33] * 150 + [700] * 150),
])
def test_decode_many_units_per_cta(kind, Hkv, G, lens):
    p = Pair(kind, Hkv, G, len(lens), max(1, -(-max(lens) // 64)), seed=G)
    try:
        for b, n in enumerate(lens):
            if n == 0:
                continue
            g = torch.Generator(device="cuda").manual_seed(b)
            k = torch.randn(1, n, Hkv, 128, device="cuda", generator=g).bfloat16()
            v = torch.randn(1, n, Hkv, 128, device="cuda", generator=g).bfloat16()
            row = {x: p.cache[x][b:b + 1] if x != "pool" else p.cache[x] for x in p.cache}
            oscar.oscar_append_kv8(p.ctx, row, kind, k, v, n, 1, weights=p.weights[b:b + 1])
        for decay in (1.0, 0.75):
            before = p.weights.clone()
            q = p.query(1.5)
            out, lse = p.decode(q, decay)
            check_decode_dense(p, q, out, lse, before, decay)
        ok(p)
    finally:
        p.close()


def test_decode_with_scales_far_apart(kind=oscar.KV8_E4M3):
    """Blocks whose values differ by 2^60 and weights that favour the small ones."""
    p = Pair(kind, 1, 2, 1, 10)
    try:
        n = 64 + 256 + 320
        k, v = p.draw(n)
        big = (torch.arange(n) // 16 % 2 == 0)
        v[0, big] *= 2.0 ** -30
        v[0, ~big] *= 2.0 ** 30
        q = p.query()
        k[0, big, 0] += 6 * q[0, 0]       # the small blocks take nearly all the weight of head 0
        k[0, 64:96, 0] -= 20 * q[0, 0]
        v[0, :64] *= 2.0 ** -30
        p.append(n, (k, v))
        out, lse = p.decode(q)
        check_decode(p, q, out, lse, 1.0)
        ok(p)
    finally:
        p.close()


def test_decode_shows_a_nan_block_only_where_it_is(kind=oscar.KV8_INT8):
    p = Pair(kind, 2, 2, 2, 10)
    try:
        k, v = p.draw(600)
        k[1, 100, 1, 3] = float("nan")
        p.append(600, (k, v))
        q = p.query()
        out, lse = p.decode(q, weights=False)
        nan = torch.isnan(out.float()).all(-1).cpu().view(2, 2, 2)
        assert nan[1, 1].all() and not nan[0].any() and not nan[1, 0].any()
        ok(p)
    finally:
        p.close()


def test_decode_leaves_bad_pages_out(kind=oscar.KV8_E4M3):
    p = lengths_pair(kind, 2, 2, [800, 800, 321], seed=9)
    try:
        table = p.cache["page_table"]
        keep = table.clone()
        table[0, 2] = -1
        table[2, 0] = p.cfg.num_pages + 3
        q = p.query()
        out, lse = p.decode(q, 1.0)
        assert oscar.oscar_get_error(p.ctx) in (oscar.ERR_NO_PAGE, oscar.ERR_RANGE)
        for b, r in enumerate(p.req):  # the oracle without those tokens
            for h in range(2):
                gone = range(8, 12) if b == 0 else range(0, 1) if b == 2 else []
                r.blocks[h] = [x for j, x in enumerate(r.blocks[h]) if j not in gone]
                r.w_hist[h] = [x for j, x in enumerate(r.w_hist[h]) if j not in gone]
        check_decode(p, q, out, lse)
        w = p.weights.cpu()
        assert (w[0, :, 16 + 8:16 + 12] == 0).all() and (w[2, :, 16] == 0).all()
        table.copy_(keep)
    finally:
        p.close()


# ------------------------------------------------------------------ eviction
def settle(p, seed, values=None):
    """Block weights from fp32 draws, the same in the oracle."""
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(p.weights.shape, generator=g) if values is None else \
        values[torch.randint(0, len(values), p.weights.shape, generator=g)]
    p.weights.copy_(w)
    for b, r in enumerate(p.req):
        for h in range(p.Hkv):
            r.w_hist[h] = [float(x) for x in w[b, h, 16:16 + len(r.blocks[h])]]
            r.w_ring[h] = w[b, h, :16].double().numpy()
    return w


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("budget", [0, 1, 16, 250, 512, 1000, 100000])
def test_evict_matches_the_oracle(kind, budget):
    p = lengths_pair(kind, 2, 1, [0, 50, 320, 321, 576, 577, 832, 1500, 3000], seed=budget % 97)
    try:
        w = settle(p, 4)
        oscar.oscar_evict_kv8(p.ctx, p.cache, p.weights, budget, p.scratch, p.B)
        for b, r in enumerate(p.req):
            r.evict(budget, w[b, :, 16:].numpy())
            assert r.H <= budget + 255 or r.H < 256
        p.check_state()
        q = p.query()
        out, lse = p.decode(q)
        check_decode(p, q, out, lse, 1.0)
        p.append(40)  # the window went on where it was
        p.check_state(weight_tol=1e-4)
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("values", [[0.0], [0.0, 1.0], [1e-30, 1e-38, 0.0, -0.0, 2.0, float("inf")],
                                    [-1.0, 0.5, float("nan"), float("-inf")]])
def test_evict_ties_and_odd_weights(values):
    p = lengths_pair(oscar.KV8_INT8, 2, 1, [2000, 5000], seed=1)
    try:
        w = settle(p, 8, torch.tensor(values))
        if 0.0 in values and any(np.signbit(values)):
            w = torch.where(w == 0, torch.zeros(()), w)  # -0 sorts below 0 on the device: one zero only
            p.weights.copy_(w)
            for b, r in enumerate(p.req):
                for h in range(2):
                    r.w_hist[h] = [float(x) for x in w[b, h, 16:16 + len(r.blocks[h])]]
        oscar.oscar_evict_kv8(p.ctx, p.cache, p.weights, 700, p.scratch, p.B)
        for b, r in enumerate(p.req):
            r.evict(700, w[b, :, 16:].numpy())
        got = p.weights.cpu().numpy()
        for b, r in enumerate(p.req):
            for h in range(2):
                np.testing.assert_array_equal(got[b, h, 16:16 + r.H // 16], np.float32(r.w_hist[h]))
                r.w_hist[h] = [0.0] * (r.H // 16)
        p.weights[:, :, 16:] = 0
        p.check_state()
        ok(p)
    finally:
        p.close()


def test_evict_refuses_bad_pages(kind=oscar.KV8_E4M3):
    p = lengths_pair(kind, 1, 1, [1500, 1500], seed=1)
    try:
        w = settle(p, 3)
        p.cache["page_table"][0, 7] = -1
        before = p.cache["pool"].clone()
        oscar.oscar_evict_kv8(p.ctx, p.cache, p.weights, 256, p.scratch, 2)
        assert oscar.oscar_get_error(p.ctx) == oscar.ERR_NO_PAGE
        p.req[1].evict(256, w[1, :, 16:].numpy())
        assert p.cache["seq_lens"].tolist() == [1500, p.req[1].L]
        mine = p.cache["page_table"][0].long()
        mine = mine[mine >= 0]
        same = (p.cache["pool"].view(-1, 16416)[mine] == before.view(-1, 16416)[mine]).all()
        assert bool(same)
    finally:
        p.close()
