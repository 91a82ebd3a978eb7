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
    (12, [1, 600, 1, 20]),
    (16, [700, 1, 300]),
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


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,where", [(321, "block"), (640, "page"), (70, "sink"), (200, "window"), (5, "all")])
def test_decode_shows_nan_where_nothing_else_is_near(kind, n, where):
    """NaN keys that fill a block alone in its page, a whole page, a unit of the
    sink or window, or all there is: the outputs that see them are NaN, and lse."""
    p = Pair(kind, 2, 2, 2, 8)
    try:
        k, v = p.draw(n)
        at = {"block": (64, 80), "page": (128, 192), "sink": (32, 64), "window": (160, 192), "all": (0, n)}[where]
        k[1, at[0]:at[1], 1] = float("nan")
        p.append(n, (k, v))
        out, lse = p.decode(p.query(), weights=False)
        nan = torch.isnan(out.float()).all(-1).cpu().view(2, 2, 2)
        assert nan[1, 1].all() and torch.isnan(lse.cpu().view(2, 2, 2)[1, 1]).all()
        assert not nan[0].any() and not nan[1, 0].any() and not torch.isnan(lse[0]).any()
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_decode_with_a_query_that_is_not_finite(bad, kind=oscar.KV8_INT8):
    p = lengths_pair(kind, 2, 4, [5, 900], seed=77)
    try:
        q = p.query()
        q[:, 3, 17] = bad
        out, lse = p.decode(q, weights=False)
        o, ls = out.float().cpu(), lse.cpu()
        assert torch.isnan(o[:, 3]).all() and torch.isnan(ls[:, 3]).all()
        rest = [h for h in range(8) if h != 3]
        assert torch.isfinite(o[:, rest]).all() and torch.isfinite(ls[:, rest]).all()
        ok(p)
    finally:
        p.close()


def test_decode_of_lengths_no_append_leaves(kind=oscar.KV8_E4M3):
    """Empty outputs and OSCAR_ERR_STATE for them, the others as ever."""
    p = lengths_pair(kind, 2, 2, [500, 500, 500, 500, 500], seed=78)
    try:
        p.cache["seq_lens"][0] = 900       # a window of 644 tokens
        p.cache["hist_lens"][1] += 8       # half a block
        p.cache["hist_lens"][2] = 16 * 64  # more than there is
        p.cache["seq_lens"][3] = -5
        q = p.query()
        before = p.weights.clone()
        out, lse = p.decode(q, 1.0)
        assert oscar.oscar_get_error(p.ctx) == oscar.ERR_STATE
        assert bool((out[:4] == 0).all()) and bool(torch.isneginf(lse[:4]).all())
        assert torch.equal(p.weights[:4], before[:4])
        one = Pair.__new__(Pair)
        one.__dict__.update(p.__dict__)
        one.B, one.req = 1, p.req[4:]
        check_decode(one, q[4:], out[4:], lse[4:])
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


def test_evict_more_blocks_than_the_selection_keeps(kind=oscar.KV8_INT8):
    """A history beyond 800K tokens, whose last weights the selection reads again."""
    n = 54000
    p = Pair(kind, 1, 1, 1, n // 4 + 2, seed=5, dirty=False)
    try:
        g = torch.Generator(device="cuda").manual_seed(3)
        p.cache["hist_lens"][0] = 16 * n
        p.cache["seq_lens"][0] = 16 * n + 64 + 250
        p.cache["pool"].copy_(torch.randint(0, 256, p.cache["pool"].shape, dtype=torch.uint8, device="cuda", generator=g))
        w = (torch.randint(0, 3000, (n,), device="cuda", generator=g).float() / 3000) ** 4  # many ties
        p.weights[0, 0, 16:16 + n] = w
        blocks = p.cache["pool"].view(-1, 16416)[p.cache["page_table"][0].long()][:, :16384].reshape(-1, 4096).clone()
        budget = 16 * 20000
        e = (16 * n - budget) // 256 * 16
        keep = n - e
        gone = torch.zeros(n, dtype=torch.bool, device="cuda")
        gone[torch.sort(w, stable=True)[1][:e]] = True
        idx = torch.arange(n, device="cuda")
        holes, ends = (gone & (idx < keep)).nonzero()[:, 0], (~gone & (idx >= keep)).nonzero()[:, 0]
        oscar.oscar_evict_kv8(p.ctx, p.cache, p.weights, budget, p.scratch, 1)
        assert p.cache["hist_lens"].tolist() == [16 * keep]
        w[holes], blocks[holes] = w[ends], blocks[ends]
        assert torch.equal(p.weights[0, 0, 16:16 + keep], w[:keep])
        got = p.cache["pool"].view(-1, 16416)[p.cache["page_table"][0].long()][:, :16384].reshape(-1, 4096)
        assert torch.equal(got[:keep], blocks[:keep])
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


# -------------------------------------------------------- as they would be used
def advance(p, T, q, decay, budget, call=None):
    """One turn on both sides: append, attend, evict when due; the eviction goes by the device's weights."""
    p.append(T, call=call)
    out, lse = p.decode(q, decay)
    worst = check_decode(p, q, out, lse, decay)
    if any(r.H - budget >= 256 for r in p.req):
        w = p.weights.cpu().numpy()
        oscar.oscar_evict_kv8(p.ctx, p.cache, p.weights, budget, p.scratch, p.B)
        for b, r in enumerate(p.req):
            r.evict(budget, w[b, :, 16:])
    return worst


@pytest.mark.parametrize("kind", KINDS)
def test_append_decode_evict_together(kind):
    """A few hundred tokens in steps and chunks, attended to and evicted, stay
    with the oracle: state bit for bit, weights within the roundings added up."""
    p = Pair(kind, 2, 4, 3, 14, seed=21)
    try:
        worst = 0.0
        for T in (500, 1, 1, 1, 60, 1, 30, 1, 200, 1, 1, 17, 1, 250, 1, 1, 90, 1):
            worst += advance(p, T, p.query(1.2), 0.95, 300)
            p.check_state(weight_tol=2 * worst)
        assert all(r.H < 300 + 256 for r in p.req) and all(r.L < 1000 for r in p.req)
        ok(p)
    finally:
        p.close()


def test_captured_steps_replay(kind=oscar.KV8_INT8):
    """A decode step and an eviction captured once and replayed many times
    follow the lengths on the device, on a stream of their own."""
    p = Pair(kind, 2, 2, 2, 14, seed=22)
    try:
        p.append(590)
        k, v = torch.zeros(2, 1, 2, 128, dtype=torch.bfloat16).cuda(), torch.zeros(2, 1, 2, 128, dtype=torch.bfloat16).cuda()
        q = p.query().cuda()
        out = torch.empty_like(q)
        lse = torch.empty(2, 4, dtype=torch.float32, device="cuda")
        st = torch.cuda.Stream()
        g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        before = {x: p.cache[x].clone() for x in p.cache}
        with torch.cuda.stream(st):
            with torch.cuda.graph(g1, stream=st):
                oscar.oscar_append_kv8(p.ctx, p.cache, kind, k, v, 1, 2, weights=p.weights)
                oscar.oscar_decode_kv8(p.ctx, p.cache, kind, q, out, lse, p.scratch, 2, weights=p.weights, decay=0.9)
            with torch.cuda.graph(g2, stream=st):
                oscar.oscar_evict_kv8(p.ctx, p.cache, p.weights, 256, p.scratch, 2)
        torch.cuda.synchronize()
        assert torch.equal(p.cache["seq_lens"], before["seq_lens"])  # capturing ran nothing
        worst = 0.0
        for i in range(300):
            kn, vn = p.draw(1)
            qn = p.query()
            with torch.cuda.stream(st):
                k.copy_(kn)
                v.copy_(vn)
                q.copy_(qn)
                g1.replay()
            for b, r in enumerate(p.req):
                r.append(kn[b, 0].double().numpy(), vn[b, 0].double().numpy())
            st.synchronize()
            worst += check_decode(p, qn, out, lse, 0.9)
            if p.req[0].H >= 512:
                w = p.weights.cpu().numpy()
                with torch.cuda.stream(st):
                    g2.replay()
                for b, r in enumerate(p.req):
                    r.evict(256, w[b, :, 16:])
        st.synchronize()
        p.check_state(weight_tol=2 * worst)
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,Hkv,G,start", [(1, 8, 4, 5000), (3, 2, 8, 330), (40, 2, 1, 700)])
def test_back_to_back_equals_one_at_a_time(kind, B, Hkv, G, start):
    """Kernels of one call start before the call before has ended: 150 steps,
    chunks and evictions without a pause give the same bits, outputs, weights and
    state, as with a synchronisation after every call."""
    def play(pause):
        p = Pair(kind, Hkv, G, B, -(-(start + 900) // 64), seed=6, dirty=False)
        g = torch.Generator(device="cuda").manual_seed(8)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
        try:
            outs = []
            k, v = rand(B, start, Hkv, 128), rand(B, start, Hkv, 128)
            oscar.oscar_append_kv8(p.ctx, p.cache, kind, k, v, start, B, weights=p.weights)
            steps = [(rand(B, T, Hkv, 128), rand(B, T, Hkv, 128), rand(B, Hkv * G, 128), T)
                     for T in ([1] * 40 + [37]) * 4]
            torch.cuda.synchronize()
            for i, (k, v, q, T) in enumerate(steps):
                out, lse = torch.empty_like(q), torch.empty(B, Hkv * G, device="cuda")
                oscar.oscar_append_kv8(p.ctx, p.cache, kind, k, v, T, B, weights=p.weights)
                if pause:
                    torch.cuda.synchronize()
                oscar.oscar_decode_kv8(p.ctx, p.cache, kind, q, out, lse, p.scratch, B, weights=p.weights, decay=0.99)
                if pause:
                    torch.cuda.synchronize()
                if i % 50 == 20:
                    oscar.oscar_evict_kv8(p.ctx, p.cache, p.weights, start // 2, p.scratch, B)
                    if pause:
                        torch.cuda.synchronize()
                outs += [out, lse]
            torch.cuda.synchronize()
            ok(p)
            return outs + [p.weights, p.cache["seq_lens"], p.cache["hist_lens"], p.cache["pool"], p.cache["ring_k"],
                           p.cache["ring_v"]]
        finally:
            p.close()

    for a, b in zip(play(False), play(True)):
        assert torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))


def test_between_int2_calls_without_a_pause(kind=oscar.KV8_INT8):
    """8-bit and INT2 calls of one context in turn on a stream: the INT2 decode
    reads its lengths before its own wait, so no 8-bit kernel may let it start
    before the INT2 append has ended."""
    def play(pause):
        p = Pair(kind, 2, 4, 2, 40, seed=9, dirty=False)
        int2 = oscar.alloc_cache(p.cfg)
        int2["page_table"].copy_(torch.arange(80).int().view(2, 40))
        sc = oscar.alloc_scratch(p.cfg)
        g = torch.Generator(device="cuda").manual_seed(2)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
        sync = torch.cuda.synchronize if pause else lambda: None
        try:
            k, v = rand(2, 1000, 2, 128), rand(2, 1000, 2, 128)
            oscar.oscar_append_kv8(p.ctx, p.cache, kind, k, v, 1000, 2, weights=p.weights)
            oscar.oscar_import_tokens(p.ctx, 0, int2, k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous(), 2, 1000)
            steps = [(rand(2, 1, 2, 128), rand(2, 1, 2, 128), rand(2, 8, 128)) for _ in range(120)]
            torch.cuda.synchronize()
            outs = []
            for k, v, q in steps:
                a, b = torch.empty_like(q), torch.empty_like(q)
                oscar.oscar_append(p.ctx, 0, int2, k, v, 2)
                sync()
                oscar.oscar_append_kv8(p.ctx, p.cache, kind, k, v, 1, 2, weights=p.weights)
                sync()
                oscar.oscar_decode(p.ctx, 0, int2, q, a, None, sc, 2)
                sync()
                oscar.oscar_decode_kv8(p.ctx, p.cache, kind, q, b, None, p.scratch, 2, weights=p.weights)
                sync()
                outs += [a, b]
            torch.cuda.synchronize()
            ok(p)
            return outs + [int2["seq_lens"], p.cache["seq_lens"], p.weights]
        finally:
            p.close()

    for a, b in zip(play(False), play(True)):
        torch.testing.assert_close(a, b, rtol=2.0 ** -7, atol=2.0 ** -9)  # (INT2 partials may join in another order)


def test_requests_may_share_pages_when_read(kind=oscar.KV8_E4M3):
    """A common prefix: the second request's table names the first one's pages."""
    p = lengths_pair(kind, 2, 4, [1344, 0], seed=24)
    try:
        for x in p.cache:
            if x != "pool":
                p.cache[x][1] = p.cache[x][0]
        p.req[1] = p.req[0]
        q = p.query()
        out, lse = p.decode(q, weights=False)
        check_decode(p, q, out, lse)
        ok(p)
    finally:
        p.close()


def test_two_calls_at_once_on_two_streams(kind=oscar.KV8_E4M3):
    """Different caches of one context on two streams, each with its own scratch."""
    a = lengths_pair(kind, 2, 4, [4000, 900], seed=31)
    b = Pair(kind, 2, 4, 2, a.pages, seed=32)
    try:
        b.append(2000)
        sb = oscar.alloc_scratch_kv8(a.cfg)
        qa, qb = a.query(), b.query()
        oa, ob = qa.cuda(), qb.cuda()
        la, lb = (torch.empty(2, 8, dtype=torch.float32, device="cuda") for _ in range(2))
        da, db = oa.clone(), ob.clone()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(20):
            oscar.oscar_decode_kv8(a.ctx, a.cache, kind, da, oa, la, a.scratch, 2, stream=s1)
            oscar.oscar_decode_kv8(a.ctx, b.cache, kind, db, ob, lb, sb, 2, stream=s2)
        torch.cuda.synchronize()
        check_decode(a, qa, oa, la)
        check_decode(b, qb, ob, lb)
        ok(a)
    finally:
        a.close()
        b.close()


def test_rows_behind_the_batch_stay(kind=oscar.KV8_INT8):
    p = Pair(kind, 2, 2, 2, 12, seed=41, max_batch=4)
    try:
        p.cache["seq_lens"][2:] = 700
        p.cache["hist_lens"][2:] = 384
        p.weights[2:] = 3.0
        keep = {x: p.cache[x][2:].clone() for x in p.cache if x not in ("pool", "page_table")}
        mine = p.cache["page_table"][2:].reshape(-1).long()
        pages = p.cache["pool"].view(p.cfg.num_pages, -1)[mine].clone()
        for T in (600, 1, 300):
            p.append(T)
            q = p.query()
            out = torch.full((4, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.full((4, 4), 7.0, device="cuda")
            qd = torch.cat([q.cuda(), torch.zeros_like(q.cuda())])
            oscar.oscar_decode_kv8(p.ctx, p.cache, kind, qd, out, lse, p.scratch, 2, weights=p.weights)
            check_decode(p, q, out[:2], lse[:2], 1.0)
            assert bool((out[2:] == 7).all()) and bool((lse[2:] == 7).all())
        w = p.weights.cpu().numpy()
        oscar.oscar_evict_kv8(p.ctx, p.cache, p.weights, 100, p.scratch, 2)
        for b, r in enumerate(p.req):
            r.evict(100, w[b, :, 16:])
        p.check_state(weight_tol=1e-3)
        for x in keep:
            assert torch.equal(p.cache[x][2:].view(torch.uint8), keep[x].view(torch.uint8)), x
        assert bool((p.weights[2:] == 3).all())
        assert torch.equal(p.cache["pool"].view(p.cfg.num_pages, -1)[mine], pages)
        ok(p)
    finally:
        p.close()


def test_pinned_host_operands(kind=oscar.KV8_E4M3):
    p = Pair(kind, 2, 2, 2, 12, seed=51)
    try:
        for T in (400, 1, 300):
            k, v = p.draw(T)
            p.append(T, (k, v), call=lambda k, v: oscar.oscar_append_kv8(
                p.ctx, p.cache, kind, k.pin_memory(), v.pin_memory(), T, 2, weights=p.weights) or torch.cuda.synchronize())
        p.check_state()
        q = p.query()
        out, lse = torch.empty_like(q).pin_memory(), torch.empty(2, 4).pin_memory()
        oscar.oscar_decode_kv8(p.ctx, p.cache, kind, q.pin_memory(), out, lse, p.scratch, 2)
        torch.cuda.synchronize()
        check_decode(p, q, out, lse)
        ok(p)
    finally:
        p.close()


def test_batches_beyond_one_launch(kind=oscar.KV8_INT8):
    """1100 requests: two launches of at most 1024, one after the other over one scratch."""
    B = 1100
    p = Pair(kind, 1, 1, B, 2, seed=61)
    try:
        g = torch.Generator(device="cuda").manual_seed(1)
        for T in (340, 3):
            k, v = (torch.randn(B, T, 1, 128, device="cuda", generator=g).bfloat16() for _ in range(2))
            oscar.oscar_append_kv8(p.ctx, p.cache, kind, k, v, T, B, weights=p.weights)
        assert p.cache["seq_lens"].unique().tolist() == [343] and p.cache["hist_lens"].unique().tolist() == [32]
        before = p.weights.clone()
        q = p.query()
        out, lse = p.decode(q, 0.5)
        pick = [0, 1, 1022, 1023, 1024, 1025, B - 1]
        few = Pair.__new__(Pair)
        few.__dict__.update(p.__dict__)
        few.B = len(pick)
        few.cache = {x: p.cache[x][pick] if x != "pool" else p.cache[x] for x in p.cache}
        few.weights = p.weights[pick]
        check_decode_dense(few, q[pick], out[pick], lse[pick], before[pick], 0.5)
        oscar.oscar_evict_kv8(p.ctx, p.cache, p.weights, 0, p.scratch, B)  # 32 tokens of history: nothing to do
        assert p.cache["hist_lens"].unique().tolist() == [32]
        ok(p)
    finally:
        p.close()


def test_weights_of_a_batch_in_several_launches(kind=oscar.KV8_E4M3):
    """With weights the scratch is kept near 64 MB: long page tables split the batch."""
    lens = [700, 40, 3000, 500, 321, 1200, 0, 900, 2000]
    p = Pair(kind, 8, 8, len(lens), 6000, seed=71, num_pages=200)
    try:
        ids = torch.randperm(200, generator=p.g).int().cuda()
        at = 0
        for b, n in enumerate(lens):
            m = -(-max(n - 320 + 15, 0) // 64)
            p.cache["page_table"][b, :m] = ids[at:at + m]
            at += m
            if n:
                k, v = p.draw(n, B=1)
                row = {x: p.cache[x][b:b + 1] if x != "pool" else p.cache[x] for x in p.cache}
                oscar.oscar_append_kv8(p.ctx, row, kind, k.cuda(), v.cuda(), n, 1, weights=p.weights[b:b + 1])
        for decay in (1.0, 0.5):
            before = p.weights.clone()
            q = p.query()
            out, lse = p.decode(q, decay)
            check_decode_dense(p, q, out, lse, before, decay)
        ok(p)
    finally:
        p.close()


def test_pool_beyond_four_gigabytes(kind=oscar.KV8_INT8):
    p = Pair(kind, 8, 4, 1, 40, seed=81, num_pages=36000, dirty=False)
    try:
        assert p.cache["pool"].numel() > 1 << 32
        p.cache["page_table"][0] = torch.arange(36000 - 40, 36000).int().cuda()
        p.append(1500)
        q = p.query()
        out, lse = p.decode(q)
        check_decode(p, q, out, lse, 1.0)
        w = p.weights.cpu().numpy()
        oscar.oscar_evict_kv8(p.ctx, p.cache, p.weights, 500, p.scratch, 1)
        p.req[0].evict(500, w[0, :, 16:])
        p.check_state(weight_tol=1e-4)
        ok(p)
    finally:
        p.close()


def test_a_wait_that_runs_out_is_reported(kind=oscar.KV8_INT8):
    p = lengths_pair(kind, 2, 2, [5000, 300], seed=91)
    try:
        q = p.query()
        oscar.oscar_set_option(p.ctx, oscar.OPT_WAIT_POLLS, 0)
        p.decode(q, weights=False)
        assert oscar.oscar_get_error(p.ctx) == oscar.ERR_TIMEOUT
        oscar.oscar_set_option(p.ctx, oscar.OPT_WAIT_POLLS, oscar.WAIT_POLLS_DEFAULT)
        out, lse = p.decode(q, weights=False)
        check_decode(p, q, out, lse)
        ok(p)
    finally:
        p.close()


def test_refusals():
    p = Pair(oscar.KV8_INT8, 2, 2, 2, 4)
    try:
        k = torch.zeros(2, 1, 2, 128, dtype=torch.bfloat16, device="cuda")
        q = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
        out, lse, w, sc = torch.empty_like(q), torch.empty(2, 4, device="cuda"), p.weights, p.scratch
        bad = oscar.ERR_INVALID_ARG

        def refused(f, *a, status=bad, **kw):
            with pytest.raises(oscar.OscarError) as e:
                f(p.ctx, *a, **kw)
            assert e.value.status == status

        ap, de, ev = oscar.oscar_append_kv8, oscar.oscar_decode_kv8, oscar.oscar_evict_kv8
        c = p.cache
        odd = torch.zeros(2 * 2 * 128 + 8, dtype=torch.bfloat16, device="cuda")[1:]
        refused(ap, c, 2, k, k, 1, 2)                      # type
        refused(ap, c, -1, k, k, 1, 2)
        refused(ap, c, 1, None, k, 1, 2)
        refused(ap, c, 1, k, odd, 1, 2)                    # alignment
        refused(ap, c, 1, k, k, -1, 2)
        refused(ap, c, 1, k, k, (1 << 24) + 1, 2)
        refused(ap, c, 1, k, k, 1, 3)                      # batch
        refused(ap, c, 1, k, k, 1, -1)
        refused(ap, c, 1, k, k, 1, 2, weights=w.view(-1)[1:])
        refused(ap, {**c, "pool": None}, 1, k, k, 1, 2)
        refused(ap, {**c, "hist_lens": None}, 1, k, k, 1, 2)
        refused(de, c, 3, q, out, lse, sc, 2)
        refused(de, c, 1, None, out, lse, sc, 2)
        refused(de, c, 1, q, None, lse, sc, 2)
        refused(de, c, 1, q, out, lse, sc[256:512], 2)     # too small
        refused(de, c, 1, q, out, lse, sc[16:], 2)         # alignment
        refused(de, c, 1, q, out, lse, sc, 3)
        for decay in (-0.5, float("nan"), float("inf")):
            refused(de, c, 1, q, out, lse, sc, 2, weights=w, decay=decay)
        refused(ev, c, None, 0, sc, 2)
        refused(ev, c, w, -1, sc, 2)
        refused(ev, c, w, 0, sc[256:272], 2)
        refused(ev, c, w, 0, sc, 3)
        assert p.cache["seq_lens"].tolist() == [0, 0]
        ap(p.ctx, c, 1, k, k, 0, 2)                        # nothing to do is fine
        ap(p.ctx, c, 1, k, k, 1, 0)
        de(p.ctx, c, 1, q, out, None, sc, 0)
        ev(p.ctx, c, w, 0, sc, 0)
        de(p.ctx, c, 1, q, out, None, sc, 2)               # empty requests, no lse
        assert bool((out == 0).all())
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("fmt,budget", [("e4m3", None), ("int8", 320), ("int8", 0)])
def test_serving_loop(fmt, budget):
    """Requests admitted, stepped together, moved between slots, evicted and
    retired by the serving loop: every output within rounding of the oracle."""
    from bit_kv_cache_int2_gb300 import serving
    from oracle import kv8_oracle as K8

    Hkv, G, max_batch, pool_pages = 2, 2, 4, 40
    kind = serving.KV8_KINDS[fmt]
    rng = np.random.default_rng(3)
    reqs = [serving.Request(rid=i, prefix=int(rng.integers(0, 1300)), gen=int(rng.integers(20, 340))) for i in range(7)]
    need = lambda prefix, gen: serving.pages_needed_kv8(prefix, gen, budget=budget)  # noqa: E731
    mpr = max(need(r.prefix, r.gen) for r in reqs)
    cfg = oscar.make_config(1, Hkv * G, Hkv, max_batch=max_batch, max_pages_per_req=mpr, num_pages=pool_pages)
    ctx = oscar.oscar_create(cfg)
    cache = oscar.alloc_cache(cfg, kv8=True)
    streams, oracles, evictions = {}, {}, [0]

    def draw(req):
        g = torch.Generator().manual_seed(req.rid)
        n = req.prefix + req.gen
        K, V = (torch.randn(Hkv, n, 128, generator=g).bfloat16() for _ in range(2))
        Q = torch.randn(req.gen, Hkv * G, 128, generator=g).bfloat16()
        streams[req.rid] = (K.double().numpy(), V.double().numpy())
        o = oracles[req.rid] = K8.Request(Hkv, kind)
        for t in range(req.prefix):
            o.append(streams[req.rid][0][:, t], streams[req.rid][1][:, t])
        return K.cuda(), V.cuda(), Q.cuda()

    class View:  # what check_decode needs
        pass

    def on_step(active, q, out):
        v = View()
        v.B, v.Hkv, v.G, v.req = len(active), Hkv, G, [oracles[r.rid] for r in active]
        for r in active:
            t = r.prefix + r.done
            oracles[r.rid].append(streams[r.rid][0][:, t], streams[r.rid][1][:, t])
        if sched.steps % 9 == 0:
            lse = torch.zeros(len(active), Hkv * G)
            for b, r in enumerate(v.req):
                lse[b] = torch.from_numpy(r.attend(q[b].double().cpu().numpy().reshape(Hkv, G, 128))[1].reshape(-1)).float()
            check_decode(v, q.cpu(), out, lse)

    def on_evict(active):
        evictions[0] += 1
        w = backend.weights.cpu().numpy()
        for b, r in enumerate(active):
            oracles[r.rid].evict(budget, w[b, :, 16:])

    try:
        backend = serving.DeviceBackend(fmt, ctx, cfg, cache, draw, on_step=on_step, budget=budget, on_evict=on_evict)
        sched = serving.Scheduler(serving.PagePool(pool_pages), max_batch, backend, mpr, need)
        for r in reqs:
            sched.submit(r)
        done = sched.run()
        assert oscar.oscar_get_error(ctx) == 0
        assert sorted(r.rid for r in done) == list(range(len(reqs)))
        assert sched.pool.available == pool_pages and len(set(sched.pool._free)) == pool_pages
        assert (evictions[0] > 0) == (budget is not None)
        with pytest.raises(ValueError):
            serving.DeviceBackend("int2", ctx, cfg, cache, draw, budget=3)
    finally:
        oscar.oscar_destroy(ctx)
