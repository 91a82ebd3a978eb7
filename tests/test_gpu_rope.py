"""Rotary positions on the GPU against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from bit_kv_cache_int2_gb300 import build as B
from bit_kv_cache_int2_gb300 import oscar
from oracle import rope_oracle as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    oscar.lib()


def setup(Hkv, G, B, T, seed=0, pad=0, norm=False):
    g = torch.Generator().manual_seed(seed)
    heads = Hkv * (G + 2)
    x = torch.randn(B, T, heads * 128 + pad, generator=g) * torch.exp2(torch.randint(-6, 7, (B, T, 1), generator=g).float())
    gam = [(1 + 0.3 * torch.randn(128, generator=g)).bfloat16() for _ in range(2)] if norm else [None, None]
    ctx = oscar.oscar_create(oscar.make_config(1, Hkv * G, Hkv, max_batch=B, max_pages_per_req=1, num_pages=1))
    return ctx, x.bfloat16(), gam


def outputs(Hkv, G, B, T):
    return [torch.full((B, T, H, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for H in (Hkv * G, Hkv, Hkv)]


def cuda(x):
    return None if x is None else x.cuda()


def check(x, pos, gam, got, Hkv, G, w, m, interleaved, eps):
    """Rounding: the BF16 result's 2^-8 of itself; before it, each of the two products
    carries cosine and sine (angle within 2^-24 turns = 2^-21.3, two ulp of sincospi), the
    norm (sum of 128 squares, rsqrt, three products) and its own: below 2^-17 of |p| + |r|."""
    B, T = x.shape[:2]
    xs = x[..., :Hkv * (G + 2) * 128].double().numpy().reshape(B, T, Hkv * (G + 2), 128)
    assert torch.equal(got[2].cpu(), x[..., :Hkv * (G + 2) * 128].view(B, T, -1, 128)[:, :, Hkv * (G + 1):])
    for name, lo, hi, ga in (("q", 0, Hkv * G, gam[0]), ("k", Hkv * G, Hkv * (G + 1), gam[1])):
        y = got[0 if name == "q" else 1].double().cpu().numpy()
        for b in range(B):
            at = int(pos[b]) + np.arange(T)
            v = xs[b, :, lo:hi]
            gn = None if ga is None else ga.double().numpy()
            ref = R.rope(v, at, w, interleaved, gn, eps, m)
            n = len(w)
            i = np.arange(n)
            p, r = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            mag = np.abs(R.rope(v, at, w[:0], interleaved, gn, eps))
            both = mag.copy()
            both[..., p] = both[..., r] = (mag[..., p] + mag[..., r]) * abs(m)
            lim = 2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * both
            err = np.abs(y[b] - ref)
            assert (err <= lim).all(), (name, b, float((err / np.maximum(lim, 1e-300)).max()))


SCALED = [(R.PLAIN, {}), (R.LINEAR, dict(factor=4.0)), (R.NTK, dict(factor=8.0)), (R.BANDS, dict(factor=8.0, trained=8192.0)),
          (R.YARN, dict(factor=4.0, trained=32768.0)), (R.YARN, dict(factor=0.5, trained=300.0, low=2.0, high=16.0)),
          (R.BANDS, dict(factor=3.0, trained=100.0, low=0.5, high=9.0))]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("Hkv,G,B,T,dims", [(8, 4, 1, 1, 128), (1, 1, 3, 7, 128), (2, 8, 2, 5, 64), (3, 2, 2, 33, 16),
                                           (1, 4, 1, 600, 112), (5, 1, 4, 3, 48), (2, 4, 5, 1, 96)])
def test_rope_matches_the_oracle(Hkv, G, B, T, dims, norm, interleaved):
    for k, (scaling, kw) in enumerate(SCALED):
        ctx, x, gam = setup(Hkv, G, B, T, seed=k, norm=norm)
        try:
            pos = torch.tensor([[0, 100_000, 1 << 22, 2_000_000_000, -5][(b + k) % 5] for b in range(B)], dtype=torch.int32)
            theta = [1e4, 1e6, 5e5][k % 3]
            table = oscar.make_rope(oscar.ROPE_INTERLEAVED if interleaved else oscar.ROPE_HALF, dims, theta, scaling, **kw)
            got = outputs(Hkv, G, B, T)
            eps = 1e-6 if k % 2 else 0.01
            oscar.oscar_rope(ctx, table, x.cuda().view(B, T, -1, 128), pos.cuda(), T, *got, B, cuda(gam[0]), cuda(gam[1]), eps)
            check(x, pos, gam, got, Hkv, G, R.speeds(dims, theta, scaling, **kw), R.size(scaling, kw.get("factor", 1.0)),
                  interleaved, eps)
        finally:
            oscar.oscar_destroy(ctx)


def test_rows_apart_and_a_given_size():
    Hkv, G, B, T = 2, 2, 3, 9
    ctx, x, gam = setup(Hkv, G, B, T, pad=136, norm=True)
    try:
        table = oscar.make_rope(oscar.ROPE_HALF, 128, 1e4, oscar.ROPE_YARN, factor=2.0, trained=4096.0, size=1.75)
        pos = torch.tensor([3, 70_000, 12], dtype=torch.int32)
        for view in (x.cuda(), x.cuda()[..., :Hkv * (G + 2) * 128].unflatten(-1, (-1, 128))):  # rows with a gap
            got = outputs(Hkv, G, B, T)
            oscar.oscar_rope(ctx, table, view, pos.cuda(), T, *got, B, cuda(gam[0]), cuda(gam[1]), 1e-5)
            check(x, pos, gam, got, Hkv, G, R.speeds(128, 1e4, R.YARN, 2.0, 4096.0), 1.75, False, 1e-5)
        one = x[:, 4:5].cuda()  # one token of each request, a whole request apart
        got = outputs(Hkv, G, B, 1)
        oscar.oscar_rope(ctx, table, one, pos.cuda(), 1, *got, B, cuda(gam[0]), cuda(gam[1]), 1e-5)
        check(x[:, 4:5], pos, gam, got, Hkv, G, R.speeds(128, 1e4, R.YARN, 2.0, 4096.0), 1.75, False, 1e-5)
    finally:
        oscar.oscar_destroy(ctx)


@pytest.mark.parametrize("layout", [oscar.ROPE_HALF, oscar.ROPE_INTERLEAVED])
def test_values_that_are_not_finite_stay_in_their_pair(layout):
    Hkv, G, T = 1, 2, 4
    ctx, x, _ = setup(Hkv, G, 1, T)
    try:
        table = oscar.make_rope(layout, 64, 1e4)
        pos = torch.tensor([11], dtype=torch.int32)
        clean, bad = outputs(Hkv, G, 1, T), outputs(Hkv, G, 1, T)
        oscar.oscar_rope(ctx, table, x.cuda(), pos.cuda(), T, *clean, 1)
        y = x.view(1, T, 4, 128).clone()
        y[0, 1, 0, 5], y[0, 2, 2, 100], y[0, 0, 3, 7] = float("inf"), float("nan"), float("-inf")
        oscar.oscar_rope(ctx, table, y.cuda(), pos.cuda(), T, *bad, 1)
        pair = [5, 37] if layout == oscar.ROPE_HALF else [4, 5]
        for a, b, at in ((clean[0], bad[0], [(1, 0, c) for c in pair]), (clean[1], bad[1], [(2, 0, 100)]), (clean[2], bad[2], [(0, 0, 7)])):
            differ = set(map(tuple, (a[0] != b[0]).nonzero().tolist()))
            assert differ == set(at)
            assert not any(bool(torch.isfinite(b[0][i])) for i in at)
    finally:
        oscar.oscar_destroy(ctx)


def test_rows_behind_the_batch_stay_and_large_batches():
    Hkv, G, T = 1, 1, 2
    ctx, x, _ = setup(Hkv, G, 1500, T, seed=3)
    try:
        table = oscar.make_rope()
        pos = torch.arange(1500, dtype=torch.int32) * 7
        got = outputs(Hkv, G, 1500, T)
        oscar.oscar_rope(ctx, table, x.cuda(), pos.cuda(), T, *got, 1400)
        for y in got:
            assert bool(torch.isnan(y[1400:]).all())
        check(x[:1400], pos[:1400], [None, None], [y[:1400] for y in got], Hkv, G, R.speeds(128, 1e6), 1.0, False, 0.0)
    finally:
        oscar.oscar_destroy(ctx)


def test_captured_and_replayed_with_other_positions():
    Hkv, G, B, T = 2, 4, 2, 3
    ctx, x, gam = setup(Hkv, G, B, T, norm=True)
    try:
        table = oscar.make_rope()
        xd, pos, got = x.cuda(), torch.tensor([5, 6], dtype=torch.int32, device="cuda"), outputs(Hkv, G, B, T)
        gd = [y.cuda() for y in gam]
        st = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            oscar.oscar_rope(ctx, table, xd, pos, T, *got, B, *gd, 1e-6)
        for at in ([5, 6], [400_000, 0]):
            pos.copy_(torch.tensor(at, dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
            check(x, at, gam, got, Hkv, G, R.speeds(128, 1e6), 1.0, False, 1e-6)
    finally:
        oscar.oscar_destroy(ctx)


def test_refusals():
    ctx, x, gam = setup(2, 2, 2, 3, norm=True)
    try:
        table, xd, pos = oscar.make_rope(), x.cuda(), torch.zeros(2, dtype=torch.int32, device="cuda")
        q, k, v = outputs(2, 2, 2, 3)
        ga = gam[0].cuda()

        def refused(*a, status=oscar.ERR_INVALID_ARG, **kw):
            with pytest.raises(oscar.OscarError) as e:
                oscar.oscar_rope(ctx, *a, **kw)
            assert e.value.status == status

        odd = torch.zeros(3 * 4 * 128 * 8, dtype=torch.bfloat16, device="cuda")[1:]
        refused(table, None, pos, 3, q, k, v, 2, row=1024)
        refused(table, xd, None, 3, q, k, v, 2)
        refused(table, xd, pos, 3, None, k, v, 2)
        refused(table, xd, pos, 3, q, odd, v, 2)
        refused(table, xd, pos, -1, q, k, v, 2, row=1024)
        refused(table, xd, pos, (1 << 24) + 1, q, k, v, 2, row=1024)
        refused(table, xd, pos, 3, q, k, v, 3)
        refused(table, xd, pos, 3, q, k, v, -1)
        refused(table, xd, pos, 3, q, k, v, 2, row=1016)      # shorter than a row
        refused(table, xd, pos, 3, q, k, v, 2, row=1028)      # not whole 16-byte pieces
        refused(table, xd, pos, 3, q, k, v, 2, gamma_q=ga)    # one gamma alone
        refused(table, xd, pos, 3, q, k, v, 2, gamma_q=ga, gamma_k=ga, eps=-1.0)
        refused(table, xd, pos, 3, q, k, v, 2, gamma_q=ga, gamma_k=ga, eps=float("nan"))
        refused(oscar.oscar_rope_table(), xd, pos, 3, q, k, v, 2)
        with pytest.raises(ValueError):
            oscar.oscar_rope(ctx, table, xd[:, :2], pos, 2, q, k, v, 2)  # rows not evenly apart
        oscar.oscar_rope(ctx, table, None, None, 0, None, None, None, 2, row=1024)
        oscar.oscar_rope(ctx, table, None, None, 3, None, None, None, 0, row=1024)
        assert all(bool(torch.isnan(y).all()) for y in (q, k, v))
    finally:
        oscar.oscar_destroy(ctx)
