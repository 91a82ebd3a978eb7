"""The prompt's side of the 8-bit-history cache on the GPU: attention of a chunk and reading
back, against the 64-bit oracle, and a layer's calls together."""
import numpy as np
import pytest
import torch

from bit_kv_cache_int2_gb300 import build as B
from bit_kv_cache_int2_gb300 import oscar

pytestmark = pytest.mark.gpu

from kv8_scenario import Pair, check_decode, dense  # noqa: E402
from oracle import kv8_oracle as K8  # noqa: E402
from oracle import rope_oracle as R  # noqa: E402

KINDS = [oscar.KV8_E4M3, oscar.KV8_INT8]


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    oscar.lib()


def ok(p):
    assert oscar.oscar_get_error(p.ctx) == 0


def scratch_of(p):
    s = oscar.alloc_scratch_kv8(p.cfg, prefill=True)
    s.fill_(0xFF)
    return s


def chunk_of(p, T, scale=1.0, B=None):
    B = B or p.B
    k, v = p.draw(T, scale, B)
    q = (torch.randn(B, T, p.Hkv * p.G, 128, generator=p.g) * scale).bfloat16()
    return q, k, v


def prefill(p, q, k, v, batch=None, scratch=None, cache=None):
    T = q.shape[1]
    qd = q.cuda()
    out = torch.full_like(qd, float("nan"))
    lse = torch.full(qd.shape[:3], float("nan"), dtype=torch.float32, device="cuda")
    oscar.oscar_prefill_kv8(p.ctx, cache or p.cache, p.kind, qd, k.cuda(), v.cuda(), T, out, lse,
                            scratch if scratch is not None else scratch_of(p), batch or q.shape[0])
    return out, lse


def limits(z_mag, p, V, is_hist, ref):
    """What rounding allows, from a row's [rows] largest logit magnitude, weights p [rows][n] and V [n][128]
    (numpy or torch, 64 bits).  A logit is an fp32 sum of 128 products, at most 128 roundings of 2^-23 of the
    sum of magnitudes (2^-16), with 2^-19 for scale, exponential and sums.  History weights go through FP16
    (2^-11, and 2^-33 of the largest p·|v| of the row where they are subnormal: they are scaled to 2^8 or
    more there), the others through BF16 (2^-8).  The products' sum has a rounding of 2^-23 for every 16
    tokens.  The output is rounded to BF16 (2^-8)."""
    ds = 2.0 ** -16 * z_mag + 2.0 ** -19
    dp = 2 * ds + 2.0 ** -19
    n = V.shape[0]
    a = abs(V)
    hist = p * is_hist
    amax = a.max(1) if isinstance(a, np.ndarray) else a.amax(1)
    top = (p * amax).max(1) if isinstance(a, np.ndarray) else (p * amax).amax(1)
    o = 2.0 ** -11 * (hist @ a) + 2.0 ** -8 * ((p - hist) @ a) + (dp[:, None] + n / 16 * 2.0 ** -23) * (p @ a)
    o = o + n * 2.0 ** -33 * top[:, None]
    return o + 2.0 ** -8 * (abs(ref) + o), ds + 2.0 ** -19


def check_chunk(p, q, k, v, out, lse, rows=None):
    T = q.shape[1]
    qn, kn, vn = (x.double().numpy() for x in (q, k, v))
    on = out.double().cpu().numpy().reshape(-1, T, p.Hkv, p.G, 128)
    ln = lse.double().cpu().numpy().reshape(-1, T, p.Hkv, p.G)
    for b in rows if rows is not None else range(q.shape[0]):
        r = p.req[b]
        qb = qn[b].reshape(T, p.Hkv, p.G, 128)
        ref, rl, ps = r.chunk(qb, kn[b], vn[b])
        for h in range(p.Hkv):
            K, V = r.tokens(h)
            K, V = np.concatenate([K, kn[b][:, h]]), np.concatenate([V, vn[b][:, h]])
            at = np.arange(len(K))
            is_hist = ((at >= 64) & (at < 64 + r.H)).astype(float)
            for t in range(T):
                n = r.L + t + 1
                mag = (np.abs(qb[t, h]) @ np.abs(K[:n]).T).max(1) / np.sqrt(128)
                lim, tl = limits(mag, ps[h, t, :, :n], V[:n], is_hist[:n], ref[t, h])
                err = np.abs(on[b, t, h] - ref[t, h])
                assert (err <= lim).all(), (b, h, t, r.L, T, float((err / lim).max()))
                assert (np.abs(ln[b, t, h] - rl[t, h]) <= tl + 2.0 ** -22 * np.abs(rl[t, h])).all(), (b, h, t, r.L, T)


def check_chunk_dense(p, q, k, v, out, lse, seen=None):
    """As check_chunk, from the device state: for long requests.  seen [n]: history tokens that count."""
    T = q.shape[1]
    for b in range(q.shape[0]):
        L, H = int(p.cache["seq_lens"][b]), int(p.cache["hist_lens"][b])
        for h in range(p.Hkv):
            K, V = dense(p, b, h)
            K, V = torch.cat([K, k[b, :, h].cuda().double()]), torch.cat([V, v[b, :, h].cuda().double()])
            at = torch.arange(L + T, device="cuda")
            is_hist = ((at >= 64) & (at < 64 + H)).double()
            for g in range(p.G):
                for t0 in range(0, T, 512):
                    t1 = min(T, t0 + 512)
                    x = q[b, t0:t1, h * p.G + g].cuda().double()
                    z = x @ K.T / 128 ** 0.5
                    hide = at[None] > L + torch.arange(t0, t1, device="cuda")[:, None]
                    if seen is not None:
                        hide |= ~seen[b][None]
                    z = z.masked_fill(hide, -float("inf"))
                    ps = torch.softmax(z, 1)
                    ref, rl = ps @ V, torch.logsumexp(z, 1)
                    mag = (x.abs() @ K.abs().T).amax(1) / 128 ** 0.5
                    lim, tl = limits(mag, ps, V, is_hist, ref)
                    err = (out[b, t0:t1, h * p.G + g].double() - ref).abs()
                    assert bool((err <= lim).all()), (b, h, g, t0, float((err / lim).max()))
                    dl = (lse[b, t0:t1, h * p.G + g].double() - rl).abs()
                    assert bool((dl <= tl + 2.0 ** -22 * rl.abs()).all()), (b, h, g, t0, float(dl.max()))


# -------------------------------------------------------------------- chunks
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 2), (2, 4), (1, 8), (3, 4)])
def test_chunk_matches_the_oracle(kind, Hkv, G):
    """Lengths around the borders of sink, block, window, page and tile; chunks around those of
    row tiles, from one token on."""
    p = Pair(kind, Hkv, G, 2, 12, seed=Hkv + G, weights=False)
    try:
        n = 0
        for L, Ts in ((0, (1, 2, 33, 130)), (1, (1, 64)), (63, (3, 65)), (64, (1, 17)), (65, (128,)), (193, (1, 9)), (320, (1, 66)),
                      (321, (1, 5, 31)), (337, (129,)), (384, (7,)), (385, (1, 4)), (449, (16,)), (700, (1, 63))):
            if L > n:
                p.append(L - n)
                n = L
            for T in Ts:
                q, k, v = chunk_of(p, T)
                out, lse = prefill(p, q, k, v)
                check_chunk(p, q, k, v, out, lse)
        ok(p)
    finally:
        p.close()


def fill(p, lens, keep_oracle=True):
    """Requests of these lengths, each appended alone."""
    for b, n in enumerate(lens):
        if n:
            k, v = p.draw(n, B=1)
            row = {x: p.cache[x][b:b + 1] if x != "pool" else p.cache[x] for x in p.cache}
            oscar.oscar_append_kv8(p.ctx, row, p.kind, k.cuda(), v.cuda(), n, 1)
            for t in range(n) if keep_oracle else ():
                p.req[b].append(k[0, t].double().numpy(), v[0, t].double().numpy())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 5, 40])
def test_chunk_of_requests_of_different_lengths(kind, T):
    p = Pair(kind, 2, 4, 7, 16, seed=T, weights=False)
    try:
        fill(p, [0, 1000, 1, 64, 320, 339, 700])
        q, k, v = chunk_of(p, T)
        out, lse = prefill(p, q, k, v)
        check_chunk(p, q, k, v, out, lse)
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("kind,Hkv,G,lens,T", [
    (oscar.KV8_E4M3, 2, 4, [20011], 64),
    (oscar.KV8_INT8, 8, 4, [9001, 301], 130),
    (oscar.KV8_INT8, 1, 8, [30000], 300),
    (oscar.KV8_E4M3, 8, 1, [5000, 100, 0, 12345], 257),
    (oscar.KV8_INT8, 2, 2, [0], 3001),
    (oscar.KV8_E4M3, 4, 8, [0, 700], 1111),
    (oscar.KV8_INT8, 1, 1, [100000], 4),
])
def test_long_chunks_and_long_requests(kind, Hkv, G, lens, T):
    p = Pair(kind, Hkv, G, len(lens), -(-max(lens) // 64) + 1, seed=T, weights=False)
    try:
        fill(p, lens, keep_oracle=False)
        q, k, v = chunk_of(p, T)
        out, lse = prefill(p, q, k, v)
        check_chunk_dense(p, q, k, v, out, lse)
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("kind", KINDS)
def test_many_requests_in_one_call(kind):
    """More (request, head) pieces than SMs, most of them shorter than a tile."""
    p = Pair(kind, 4, 2, 60, 8, seed=60, weights=False)
    try:
        lens = [(37 * b) % 500 for b in range(60)]
        fill(p, lens, keep_oracle=False)
        for T in (1, 6, 65):
            q, k, v = chunk_of(p, T)
            out, lse = prefill(p, q, k, v)
            check_chunk_dense(p, q, k, v, out, lse)
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes", [(2.0 ** -90, 1.0, 2.0 ** 40), (1.0, 2.0 ** -40, 2.0 ** -80), (2.0 ** 40, 2.0 ** 40, 2.0 ** -60),
                                   (0.0, 1.0, 1.0), (1.0, 0.0, 0.0)])
def test_values_of_sizes_far_apart(kind, sizes):
    """Values of the sink, the history (two halves) and the rest scaled far apart: each row within its own rounding.
    Some queries look at one region alone."""
    p = Pair(kind, 1, 4, 1, 16, seed=7, weights=False)
    try:
        n = 64 + 512 + 256
        k, v = p.draw(n)
        where = torch.zeros(n, 1, 1)
        where[:64], where[64:320], where[320:576], where[576:] = sizes[0], sizes[1], sizes[1] * 2.0 ** -30, sizes[2]
        v = (v.float() * where[None]).bfloat16()
        k[..., 0] = 0
        for i, (a, b) in enumerate(((0, 64), (64, 320), (320, 576), (576, n))):  # a channel of their own for each region
            k[:, :, :, i] = 0
            k[:, a:b, :, i] = 6.0
        p.append(n, (k, v))
        q, kc, vc = chunk_of(p, 70)
        for t in range(64):
            q[0, t, :, t % 5] = 60.0 if t % 5 < 4 else q[0, t, :, 4]
        vc = (vc.float() * sizes[2]).bfloat16()
        out, lse = prefill(p, q, kc, vc)
        check_chunk(p, q, kc, vc, out, lse)
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("L,T,at", [(0, 70, 3), (0, 300, 129), (400, 70, 69), (1000, 33, 0), (5, 513, 200)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_value_that_is_not_finite_is_seen_by_later_tokens_only(kind, L, T, at, bad):
    p = Pair(kind, 2, 2, 1, 20, seed=L + T, weights=False)
    try:
        if L:
            p.append(L, oracle=False)
        q, k, v = chunk_of(p, T)
        clean, clean_lse = prefill(p, q, k, v)
        v2 = v.clone()
        v2[0, at, 1, 77] = bad
        out, lse = prefill(p, q, k, v2)
        same = torch.ones_like(out, dtype=torch.bool)
        same[0, at:, 2:, 77] = False  # query heads 2 and 3 read kv head 1
        assert torch.equal(out[same], clean[same])
        assert not bool(torch.isfinite(out[~same]).any())
        assert torch.equal(lse, clean_lse)
        k2 = k.clone()
        k2[0, at, 0, 5] = float("nan")
        out, lse = prefill(p, q, k2, v)
        same = torch.ones_like(out, dtype=torch.bool)
        same[0, at:, :2] = False
        assert torch.equal(out[same], clean[same])
        assert bool(torch.isnan(out[~same]).all()) and bool(torch.isnan(lse[0, at:, :2]).all())
        assert torch.equal(lse[0, :, 2:], clean_lse[0, :, 2:]) and torch.equal(lse[0, :at], clean_lse[0, :at])
        q2 = q.clone()
        q2[0, at, 3, 100] = bad
        out, lse = prefill(p, q2, k, v)
        same = torch.ones_like(out, dtype=torch.bool)
        same[0, at, 3] = False
        assert torch.equal(out[same], clean[same]) and bool(torch.isnan(out[~same]).all())
        ok(p)
    finally:
        p.close()


def test_a_bad_block_shows_in_every_row(kind=oscar.KV8_INT8):
    p = Pair(kind, 2, 1, 1, 20, weights=False)
    try:
        k, v = p.draw(900)
        v[0, 70, 1, 3] = float("inf")  # in the history: the block's scale is NaN
        p.append(900, (k, v), oracle=False)
        q, kc, vc = chunk_of(p, 9)
        out, lse = prefill(p, q, kc, vc)
        assert bool(torch.isfinite(out[:, :, 0]).all()) and bool(torch.isnan(out[:, :, 1]).all())
        assert bool(torch.isfinite(lse).all())
        ok(p)
    finally:
        p.close()


def test_rows_that_see_only_logits_of_minus_infinity(kind=oscar.KV8_E4M3):
    """Keys of -inf: the first token's only logit is -inf (zeros, lse -inf); the next sees others."""
    p = Pair(kind, 1, 1, 1, 4, weights=False)
    try:
        q, k, v = chunk_of(p, 3)
        q[...] = 1.0
        k[0, 0, 0] = 0
        k[0, 0, 0, 0] = float("-inf")
        out, lse = prefill(p, q, k, v)
        assert bool((out[0, 0] == 0).all()) and bool(torch.isneginf(lse[0, 0]).all())
        assert torch.equal(out[0, 1, 0], v[0, 1, 0].cuda())
        assert bool(torch.isfinite(out).all())
        ok(p)
    finally:
        p.close()


def test_bad_pages_and_lengths(kind=oscar.KV8_E4M3):
    p = Pair(kind, 2, 2, 3, 20, seed=4, weights=False)
    try:
        fill(p, [1200, 900, 700], keep_oracle=False)
        q, k, v = chunk_of(p, 20)
        table = p.cache["page_table"].clone()
        for bad, code in ((-1, oscar.ERR_NO_PAGE), (10 ** 6, oscar.ERR_RANGE)):
            p.cache["page_table"][1, 3] = bad
            out, lse = prefill(p, q, k, v)
            assert oscar.oscar_get_error(p.ctx) == code
            p.cache["page_table"].copy_(table)
            seen = {b: torch.ones(int(p.cache["seq_lens"][b]) + 20, dtype=torch.bool, device="cuda") for b in range(3)}
            seen[1][64 + 192:64 + 256] = False
            check_chunk_dense(p, q, k, v, out, lse, seen)
        good = p.cache["seq_lens"].clone(), p.cache["hist_lens"].clone()
        for seq, hist in ((900, 592), (900, 100), (-5, 0), (10 ** 9, 0), (900, -16), (64 + 21 * 64 + 10, 21 * 64), (100, 640)):
            p.cache["seq_lens"][1], p.cache["hist_lens"][1] = seq, hist
            if (seq, hist) == (900, 592):
                p.cache["hist_lens"][1] = 560  # a window of 276 tokens
            out, lse = prefill(p, q, k, v)
            assert oscar.oscar_get_error(p.ctx) == oscar.ERR_STATE
            p.cache["seq_lens"][1], p.cache["hist_lens"][1] = 0, 0  # as an empty request
            check_chunk_dense(p, q, k, v, out, lse)
            p.cache["seq_lens"].copy_(good[0])
            p.cache["hist_lens"].copy_(good[1])
    finally:
        p.close()


def test_rows_behind_the_batch_stay_and_no_lse(kind=oscar.KV8_INT8):
    p = Pair(kind, 2, 2, 4, 12, seed=9, weights=False)
    try:
        fill(p, [500, 0, 330, 77])
        before = {x: p.cache[x].clone() for x in p.cache}
        q, k, v = chunk_of(p, 11)
        full, _ = prefill(p, q, k, v)
        qd = q.cuda()
        out = torch.full_like(qd, float("nan"))
        oscar.oscar_prefill_kv8(p.ctx, p.cache, kind, qd, k.cuda(), v.cuda(), 11, out, None, scratch_of(p), 3)
        check_chunk(p, q, k, v, full, prefill(p, q, k, v)[1])
        assert bool(torch.isnan(out[3]).all())
        check_chunk(p, q[:3], k[:3], v[:3], out[:3], prefill(p, q, k, v)[1][:3])
        for x in before:  # the cache is only read
            assert torch.equal(before[x].view(torch.uint8), p.cache[x].view(torch.uint8)), x
        ok(p)
    finally:
        p.close()


def test_batches_beyond_one_launch(kind=oscar.KV8_INT8):
    Bn = 1100
    p = Pair(kind, 1, 1, Bn, 1, seed=1, weights=False)
    try:
        k0, v0 = p.draw(30)
        p.append(30, (k0, v0), oracle=False)
        q, k, v = chunk_of(p, 2)
        out, lse = prefill(p, q, k, v)
        kk, vv = (torch.cat([a, b], 1).cuda().double()[:, :, 0] for a, b in ((k0, k), (v0, v)))
        z = q.cuda().double()[:, :, 0] @ kk.transpose(1, 2) / 128 ** 0.5
        z[:, 0, 31] = -float("inf")
        ref = torch.softmax(z, 2) @ vv
        lim = 2.0 ** -7 * (torch.softmax(z, 2) @ vv.abs()) + 2.0 ** -8 * ref.abs()
        assert bool(((out[:, :, 0].double() - ref).abs() <= lim).all())
        assert bool(((lse[:, :, 0].double() - torch.logsumexp(z, 2)).abs() <= 1e-4).all())
        K = torch.full((Bn, 32, 1, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        V = torch.full_like(K, float("nan"))
        oscar.oscar_read_kv8(p.ctx, p.cache, kind, 0, 32, K, V, Bn, oscar.ORDER_TOKENS)
        assert torch.equal(K[:, :30], k0.cuda()) and torch.equal(V[:, :30], v0.cuda()) and bool(torch.isnan(K[:, 30:]).all())
        ok(p)
    finally:
        p.close()


def test_captured_replayed_and_on_two_streams(kind=oscar.KV8_E4M3):
    """A captured chunk replays over a cache that has grown; two calls at once, each with its own scratch."""
    p = Pair(kind, 2, 4, 2, 30, seed=21, weights=False)
    try:
        p.append(600, oracle=False)
        T = 24
        q, k, v = chunk_of(p, T)
        qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
        out, lse, sc = torch.zeros_like(qd), torch.zeros(2, T, 8, device="cuda"), scratch_of(p)
        st = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            oscar.oscar_prefill_kv8(p.ctx, p.cache, kind, qd, kd, vd, T, out, lse, sc, 2)
            oscar.oscar_append_kv8(p.ctx, p.cache, kind, kd, vd, T, 2)
        for _ in range(4):
            want, want_lse = prefill(p, q, k, v)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert p.cache["seq_lens"].tolist() == [600 + 4 * T] * 2
        want, want_lse = prefill(p, q, k, v)
        q2, k2, v2 = chunk_of(p, 130)
        want2, want_lse2 = prefill(p, q2, k2, v2)
        torch.cuda.synchronize()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(a):
            got = [prefill(p, q, k, v) for _ in range(5)]
        with torch.cuda.stream(b):
            got2 = [prefill(p, q2, k2, v2) for _ in range(5)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) and torch.equal(y, want_lse) for x, y in got)
        assert all(torch.equal(x, want2) and torch.equal(y, want_lse2) for x, y in got2)
        ok(p)
    finally:
        p.close()


def test_two_graphs_at_once(kind=oscar.KV8_INT8):
    """Two captured passes over one cache (positions, attention, reading back), each with its own scratch,
    replayed together, equal the same calls alone."""
    p = Pair(kind, 2, 4, 2, 40, seed=22, weights=False)
    try:
        p.append(1700, oracle=False)
        table = oscar.make_rope(oscar.ROPE_INTERLEAVED, 64, 1e4)
        pos = torch.tensor([1700, 40], dtype=torch.int32, device="cuda")
        runs = []
        for T in (5, 90):
            x, sc = torch.randn(2, T, 12, 128, generator=p.g).bfloat16().cuda(), scratch_of(p)
            q, k, v, out = (torch.zeros(2, T, H, 128, dtype=torch.bfloat16, device="cuda") for H in (8, 2, 2, 8))
            lse = torch.zeros(2, T, 8, device="cuda")
            K, V = (torch.zeros(2, 2, 600, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))

            def run():
                oscar.oscar_rope(p.ctx, table, x, pos, T, q, k, v, 2)
                oscar.oscar_prefill_kv8(p.ctx, p.cache, kind, q, k, v, T, out, lse, sc, 2)
                oscar.oscar_read_kv8(p.ctx, p.cache, kind, 50, 600, K, V, 2)

            run()
            torch.cuda.synchronize()
            got = (q, k, v, out, lse, K, V)
            want = [y.clone() for y in got]
            st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                run()
            runs.append((st, graph, got, want, (x, sc)))  # a graph reads its input and writes its scratch: held with it
        for _ in range(6):
            for _, _, got, _, _ in runs:
                for y in got:
                    y.fill_(float("nan"))
            torch.cuda.synchronize()
            for st, graph, _, _, _ in runs:
                with torch.cuda.stream(st):
                    graph.replay()
            torch.cuda.synchronize()
            for _, _, got, want, _ in runs:
                assert all(torch.equal(y, z) for y, z in zip(got, want))
        ok(p)
    finally:
        p.close()


def test_calls_without_a_pause(kind=oscar.KV8_INT8):
    """Chunks, appends and decodes back to back equal the same calls one at a time."""
    runs = []
    for pause in (True, False):
        p = Pair(kind, 2, 4, 3, 60, seed=33, weights=False)
        try:
            sc, got = scratch_of(p), []
            steps = [(T, *(x.cuda() for x in chunk_of(p, T))) for T in (300, 1, 64, 7, 513, 1, 1, 130, 2, 64)]
            for T, q, k, v in steps:
                out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda")
                dec = torch.full_like(q[:, 0], float("nan"))
                got += [out, lse, dec]
                for call in (lambda: oscar.oscar_prefill_kv8(p.ctx, p.cache, kind, q, k, v, T, out, lse, sc, 3),
                             lambda: oscar.oscar_append_kv8(p.ctx, p.cache, kind, k, v, T, 3),
                             lambda: oscar.oscar_decode_kv8(p.ctx, p.cache, kind, q[:, -1].contiguous(), dec, None, p.scratch, 3)):
                    call()
                    if pause:
                        torch.cuda.synchronize()
            torch.cuda.synchronize()
            ok(p)
            runs.append([x.cpu() for x in got])
        finally:
            p.close()
    for x, y in zip(*runs):
        assert torch.equal(x, y) and bool(torch.isfinite(x).all())


def test_pool_beyond_four_gigabytes(kind=oscar.KV8_E4M3):
    p = Pair(kind, 8, 1, 1, 10, seed=2, num_pages=40000, weights=False)
    try:
        p.cache["page_table"][0] = torch.tensor([39999 - 7 * i for i in range(10)], dtype=torch.int32)
        p.append(900, oracle=False)
        q, k, v = chunk_of(p, 33)
        out, lse = prefill(p, q, k, v)
        check_chunk_dense(p, q, k, v, out, lse)
        K = torch.zeros(1, 8, 900, 128, dtype=torch.bfloat16, device="cuda")
        V = torch.zeros_like(K)
        oscar.oscar_read_kv8(p.ctx, p.cache, kind, 0, 900, K, V, 1)
        for h in range(8):
            k_, v_ = dense(p, 0, h)
            assert torch.equal(K[0, h], k_.float().bfloat16()) and torch.equal(V[0, h], v_.float().bfloat16())
        ok(p)
    finally:
        p.close()


# ---------------------------------------------------------------------- read
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("order", [oscar.ORDER_HEADS, oscar.ORDER_TOKENS])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_read_gives_the_cached_values(kind, order, Hkv):
    """Every region, ranges that begin and end anywhere; the scaled codes rounded to fp32 and then BF16."""
    lens = [0, 5, 64, 100, 320, 345, 777]
    p = Pair(kind, Hkv, 1, len(lens), 10, seed=Hkv, weights=False)
    try:
        fill(p, lens)
        for first, n in ((0, 800), (0, 1), (3, 17), (63, 2), (64, 16), (70, 300), (320, 99), (500, 277), (776, 1), (777, 5), (5000, 40)):
            shape = (len(lens), Hkv, n, 128) if order == oscar.ORDER_HEADS else (len(lens), n, Hkv, 128)
            store = torch.full((2, 8 + len(lens) * Hkv * n * 128 + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
            for shift in (0, 8):  # rows at 32 and at 16 bytes
                store.fill_(float("nan"))
                K, V = (x[shift:shift + len(lens) * Hkv * n * 128].view(shape) for x in store)
                oscar.oscar_read_kv8(p.ctx, p.cache, kind, first, n, K, V, len(lens), order)
                for side, got in enumerate((K, V)):
                    got = got.cpu() if order == oscar.ORDER_HEADS else got.cpu().transpose(1, 2)
                    for b, r in enumerate(p.req):
                        m = max(0, min(n, r.L - first))
                        assert bool(torch.isnan(got[b, :, m:]).all())
                        for h in range(Hkv):
                            want = torch.from_numpy(r.tokens(h)[side]).float().bfloat16()
                            assert torch.equal(got[b, h, :m], want[first:first + m]), (b, h, first, n)
                outside = torch.cat([store[:, :shift], store[:, shift + K.numel():]], 1)
                assert bool(torch.isnan(outside).all())
        ok(p)
    finally:
        p.close()


def test_read_of_bad_blocks_pages_and_lengths(kind=oscar.KV8_INT8):
    p = Pair(kind, 2, 1, 2, 10, seed=5, weights=False)
    try:
        k, v = p.draw(600)
        k[0, 80, 1, 3] = float("nan")
        p.append(600, (k, v))
        before = [[x.copy() for x in p.req[1].tokens(h)] for h in range(2)]

        def read():
            K = torch.full((2, 2, 600, 128), 7.0, dtype=torch.bfloat16, device="cuda")
            V = torch.full_like(K, 7.0)
            oscar.oscar_read_kv8(p.ctx, p.cache, kind, 0, 600, K, V, 2)
            torch.cuda.synchronize()
            return K.cpu(), V.cpu()

        K, V = read()
        assert bool(torch.isnan(K[0, 1, 80:96]).all()) and not bool(torch.isnan(K[0, 0]).any()) and not bool(torch.isnan(V).any())
        assert int(torch.isnan(K).sum()) == 16 * 128
        ok(p)
        for bad, code in ((-1, oscar.ERR_NO_PAGE), (20, oscar.ERR_RANGE)):
            keep = int(p.cache["page_table"][1, 2])
            p.cache["page_table"][1, 2] = bad
            K, V = read()
            assert oscar.oscar_get_error(p.ctx) == code
            assert bool((K[1, :, 192:256] == 7).all()) and bool((V[1, :, 192:256] == 7).all())
            assert torch.equal(K[1, 0, :192], torch.from_numpy(before[0][0][:192]).float().bfloat16())
            p.cache["page_table"][1, 2] = keep
        p.cache["hist_lens"][1] = 17
        K, V = read()
        assert oscar.oscar_get_error(p.ctx) == oscar.ERR_STATE
        assert bool((K[1] == 7).all()) and bool((V[1] == 7).all()) and not bool((K[0] == 7).all())
    finally:
        p.close()


# -------------------------------------------------------------------- together
@pytest.mark.parametrize("kind", KINDS)
def test_a_layers_calls_together(kind):
    """Prompt in chunks, then steps: positions, attention, append, decode; an eviction; the cache read back.
    Everything within rounding of the oracle, which is given the GPU's own turned queries and keys."""
    Hkv, G, Bn = 2, 4, 2
    p = Pair(kind, Hkv, G, Bn, 20, seed=3)
    try:
        table, w = oscar.make_rope(oscar.ROPE_HALF, 128, 1e4), R.speeds(128, 1e4)
        gam = [(1 + 0.2 * torch.randn(128, generator=p.g)).bfloat16().cuda() for _ in range(2)]
        sc, at = scratch_of(p), 0
        pos = torch.tensor([0, 1000], dtype=torch.int32, device="cuda")  # the second continues a text that is not cached
        for T in (333, 70, 1, 1, 200, 1, 5):
            x = torch.randn(Bn, T, Hkv * (G + 2), 128, generator=p.g).bfloat16()
            q, k, v = (torch.empty(Bn, T, H, 128, dtype=torch.bfloat16, device="cuda") for H in (Hkv * G, Hkv, Hkv))
            oscar.oscar_rope(p.ctx, table, x.cuda(), pos, T, q, k, v, Bn, *gam, eps=1e-6)
            for b in range(Bn):
                ref = R.rope(x[b, :, :Hkv * G].double().numpy(), int(pos[b]) + np.arange(T), w, False, gam[0].double().cpu().numpy(), 1e-6)
                assert np.abs(q[b].double().cpu().numpy() - ref).max() <= 2.0 ** -7 * np.abs(ref).max()
            if T > 1:
                out, lse = torch.empty_like(q), torch.empty(Bn, T, Hkv * G, device="cuda")
                oscar.oscar_prefill_kv8(p.ctx, p.cache, kind, q, k, v, T, out, lse, sc, Bn)
                check_chunk(p, q.cpu(), k.cpu(), v.cpu(), out, lse)
            p.append(T, (k.cpu(), v.cpu()))
            if T == 1:
                out, lse = p.decode(q[:, 0].cpu(), decay=0.9)
                check_decode(p, q[:, 0].cpu(), out, lse, 0.9)
            pos += T
            at += T
        wts = p.weights.cpu().numpy()
        oscar.oscar_evict_kv8(p.ctx, p.cache, p.weights, 16, p.scratch, Bn)
        for b, r in enumerate(p.req):
            r.evict(16, wts[b, :, 16:])
        n = p.req[0].L
        assert n == at - 256
        K = torch.zeros(Bn, Hkv, n, 128, dtype=torch.bfloat16, device="cuda")
        V = torch.zeros_like(K)
        oscar.oscar_read_kv8(p.ctx, p.cache, kind, 0, n, K, V, Bn)
        for b, r in enumerate(p.req):
            for h in range(Hkv):
                for got, want in zip((K, V), r.tokens(h)):
                    assert torch.equal(got[b, h].cpu(), torch.from_numpy(want).float().bfloat16())
        q, k, v = chunk_of(p, 40)
        out, lse = prefill(p, q, k, v)
        check_chunk(p, q, k, v, out, lse)
        ok(p)
    finally:
        p.close()


@pytest.mark.parametrize("fmt,budget,chunk", [("e4m3", None, 300), ("int8", 320, 77)])
def test_serving_from_projections(fmt, budget, chunk):
    """Prompts in chunks and steps from a layer's projections, with requests that move between slots and are
    evicted from: every output within rounding of the oracle, which is given the GPU's own turned queries and
    keys; a slot's cache moves to the INT2 format."""
    from bit_kv_cache_int2_gb300 import serving

    Hkv, G, max_batch, pool_pages = 2, 2, 3, 40
    kind = serving.KV8_KINDS[fmt]
    rng = np.random.default_rng(5)
    reqs = [serving.Request(rid=i, prefix=int(n), gen=int(g)) for i, (n, g) in
            enumerate(zip(rng.integers(0, 900, 5), rng.integers(5, 280, 5)))]
    reqs[1].prefix = 0

    def need(prefix, gen):
        return serving.pages_needed_kv8(prefix, gen, budget=budget)

    mpr = max(need(r.prefix, r.gen) for r in reqs)
    cfg = oscar.make_config(1, Hkv * G, Hkv, max_batch=max_batch, max_pages_per_req=mpr, num_pages=pool_pages)
    ctx = oscar.oscar_create(cfg)
    cache = oscar.alloc_cache(cfg, kv8=True)
    gam = [(1 + 0.2 * torch.randn(128, generator=torch.Generator().manual_seed(i))).bfloat16().cuda() for i in range(2)]
    table, w = oscar.make_rope(oscar.ROPE_HALF, 128, 1e4), R.speeds(128, 1e4)
    streams, held, seen = {}, {}, dict(chunks=0, steps=0, evictions=0, exports=0)

    class View:  # what check_chunk and check_decode look at
        def __init__(self, rids):
            self.Hkv, self.G, self.B, self.req = Hkv, G, len(rids), [held[i] for i in rids]

    def draw(req):
        n = req.prefix + req.gen
        x = torch.randn(1, n, Hkv * (G + 2), 128, generator=torch.Generator().manual_seed(req.rid)).bfloat16()
        q, k, v = (torch.empty(n, H, 128, dtype=torch.bfloat16, device="cuda") for H in (Hkv * G, Hkv, Hkv))
        oscar.oscar_rope(ctx, table, x.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), n, q, k, v, 1, *gam, eps=1e-6)
        ref = R.rope(x[0, :, :Hkv * G].double().numpy(), np.arange(n), w, False, gam[0].double().cpu().numpy(), 1e-6)
        assert np.abs(q.double().cpu().numpy() - ref).max() <= 2.0 ** -7 * np.abs(ref).max()
        streams[req.rid] = tuple(t.cpu() for t in (q, k, v))
        held[req.rid] = K8.Request(Hkv, kind)
        return x[0].cuda()

    def push(rid, t):
        held[rid].append(*(x[t].double().numpy() for x in streams[rid][1:]))

    def on_prompt(req, first, out):
        T = len(out)
        q, k, v = (x[None, first:first + T] for x in streams[req.rid])
        # the chunk's lse is not asked for here: the oracle's own stands in
        ref = held[req.rid].chunk(q[0].double().numpy().reshape(T, Hkv, G, 128), k[0].double().numpy(), v[0].double().numpy())
        check_chunk(View([req.rid]), q, k, v, out[None], torch.from_numpy(ref[1]))
        for t in range(T):
            push(req.rid, first + t)
        seen["chunks"] += 1

    def on_step(active, q, out):
        for r in active:
            push(r.rid, r.prefix + r.done)
        qs = torch.stack([streams[r.rid][0][r.prefix + r.done] for r in active])
        assert torch.equal(q.cpu(), qs)
        if seen["steps"] % 16 == 0 or budget is not None:
            view = View([r.rid for r in active])
            lse = np.stack([x.attend(y.double().numpy().reshape(Hkv, G, 128))[1] for x, y in zip(view.req, qs)])
            check_decode(view, qs, out, torch.from_numpy(lse))
        seen["steps"] += 1

    def on_evict(active):
        wts = backend.weights.cpu().numpy()
        for b, r in enumerate(active):
            held[r.rid].evict(budget, wts[b, :, 16:])
        seen["evictions"] += 1

    class Backend(serving.DeviceBackend):
        def step(self, active):
            super().step(active)
            if sched.steps % 100 == 2:  # a slot's cache as it is, and into an INT2 cache
                slot = len(active) - 1
                K, V = self.export(slot)
                r = held[active[slot].rid]
                assert K.shape == V.shape == (Hkv, r.L, 128)
                for h in range(Hkv):
                    for got, want in zip((K, V), r.tokens(h)):
                        assert torch.equal(got[h].cpu(), torch.from_numpy(want).float().bfloat16())
                pages = max(1, serving.pages_needed(r.L, 0))
                cfg2 = oscar.make_config(1, Hkv * G, Hkv, max_batch=1, max_pages_per_req=pages, num_pages=pages)
                ctx2 = oscar.oscar_create(cfg2)
                try:
                    c2 = oscar.alloc_cache(cfg2)
                    c2["page_table"][0] = torch.arange(pages, dtype=torch.int32)
                    oscar.oscar_import_tokens(ctx2, 0, c2, K[None], V[None], 1, r.L)
                    torch.cuda.synchronize()
                    assert oscar.oscar_get_error(ctx2) == 0 and int(c2["seq_lens"][0]) == r.L
                    assert torch.equal(c2["sink_k"][0, :, :min(64, r.L)], K[:, :64])
                finally:
                    oscar.oscar_destroy(ctx2)
                seen["exports"] += 1

    try:
        rope = dict(table=table, gamma_q=gam[0], gamma_k=gam[1], eps=1e-6)
        backend = Backend(fmt, ctx, cfg, cache, draw, on_step=on_step, budget=budget, on_evict=on_evict, rope=rope,
                          prompt_chunk=chunk, on_prompt=on_prompt, max_gen=8)
        sched = serving.Scheduler(serving.PagePool(pool_pages), max_batch, backend, mpr, need)
        for r in reqs:
            sched.submit(r)
        done = sched.run()
        assert oscar.oscar_get_error(ctx) == 0
        assert sorted(r.rid for r in done) == list(range(len(reqs))) and sched.pool.available == pool_pages
        assert seen["chunks"] > 4 and seen["exports"] > 0 and (budget is None or seen["evictions"] > 0)
        with pytest.raises(ValueError):
            serving.DeviceBackend("bf16", ctx, cfg, cache, draw, rope=rope)
        with pytest.raises(ValueError):
            serving.DeviceBackend(fmt, ctx, cfg, cache, draw, rope=rope, prompt_chunk=0)
    finally:
        torch.cuda.synchronize()
        oscar.oscar_destroy(ctx)


def test_refusals():
    p = Pair(oscar.KV8_INT8, 2, 2, 2, 4, weights=False)
    try:
        T, bad = 5, oscar.ERR_INVALID_ARG
        q = torch.zeros(2, T, 4, 128, dtype=torch.bfloat16, device="cuda")
        k = torch.zeros(2, T, 2, 128, dtype=torch.bfloat16, device="cuda")
        out, lse, sc = torch.full_like(q, 5.0), torch.zeros(2, T, 4, device="cuda"), scratch_of(p)
        odd = torch.zeros(q.numel() + 8, dtype=torch.bfloat16, device="cuda")[1:]
        c = p.cache

        def refused(f, *a, status=bad, **kw):
            with pytest.raises(oscar.OscarError) as e:
                f(p.ctx, *a, **kw)
            assert e.value.status == status

        pf, rd = oscar.oscar_prefill_kv8, oscar.oscar_read_kv8
        for kind in (-1, 2):
            refused(pf, c, kind, q, k, k, T, out, lse, sc, 2)
            refused(rd, c, kind, 0, T, k, k, 2)
        for i in range(3):
            for x in (None, odd):
                a = [q, k, k]
                a[i] = x
                refused(pf, c, 1, *a, T, out, lse, sc, 2)
        refused(pf, c, 1, q, k, k, T, None, lse, sc, 2)
        refused(pf, c, 1, q, k, k, T, odd, lse, sc, 2)
        refused(pf, c, 1, q, k, k, T, out, lse.view(torch.uint8).view(-1)[1:], sc, 2)
        refused(pf, c, 1, q, k, k, -1, out, lse, sc, 2)
        refused(pf, c, 1, q, k, k, (1 << 24) + 1, out, lse, sc, 2)
        refused(pf, c, 1, q, k, k, T, out, lse, sc, 3)
        refused(pf, c, 1, q, k, k, T, out, lse, sc, -1)
        refused(pf, c, 1, q, k, k, T, out, lse, sc[16:], 2)
        refused(pf, c, 1, q, k, k, T, out, lse, sc[:128], 2)
        refused(pf, {**c, "pool": None}, 1, q, k, k, T, out, lse, sc, 2)
        refused(pf, {**c, "ring_v": None}, 1, q, k, k, T, out, lse, sc, 2)
        refused(rd, c, 1, -1, T, k, k, 2)
        refused(rd, c, 1, 0, -1, k, k, 2)
        refused(rd, c, 1, 1 << 30, 1, k, k, 2)
        refused(rd, c, 1, 0, T, k, k, 2, order=2)
        refused(rd, c, 1, 0, T, None, k, 2)
        refused(rd, c, 1, 0, T, k, odd, 2)
        refused(rd, c, 1, 0, T, k, k, 3)
        refused(rd, {**c, "seq_lens": None}, 1, 0, T, k, k, 2)
        pf(p.ctx, c, 1, None, None, None, 0, None, None, sc, 2)  # nothing to do is fine
        pf(p.ctx, c, 1, None, None, None, T, None, None, sc, 0)
        rd(p.ctx, c, 1, 0, 0, None, None, 2)
        rd(p.ctx, c, 1, 5, 2, None, None, 0)
        assert bool((out == 5).all())
        ok(p)
    finally:
        p.close()
