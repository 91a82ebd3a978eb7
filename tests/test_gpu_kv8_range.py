"""Attention over 8-bit history where logits and values differ in size between
the regions: values of any size, tokens that lead by many nats and have small
values (an attention sink), against the definition in 64 bits on the device's
own state.

Every CTA holds whole requests here (152 pairs of request and KV head, 6000
tokens each), so a warp's softmax state sees window tokens and pages.

What rounding allows, relative to S = sum p |v| of a channel:
  2^-11   the weights of history tokens go through fp16
  dp      a logit is an fp32 sum of 128 products (at most 128 roundings of 2^-23
          of the sum of magnitudes: 2^-16 of it), and a weight has two of them
  2^-16   the exponentials' arguments: s, log2 of the scale and the maximum, up to
          2^7 in base 2 (2^-17 for a rounding), 2^-22 for ex2 and lg2 themselves
  n 2^-22 a warp adds up every eighth page, four products of 16 tokens each, and
          some window tiles: n = L / 128 + 40 fp32 additions on the tensor cores
and, absolute, a floor where weights are fp16 subnormals: tokens 2^29 below the
largest p A lose bits, half a step is 2^-40 of it and the codes reach at most
twice A / scale (A: the largest magnitude in a history token's block, in a window
token's own row):  L 2^-39 max(p A).  The output is then rounded to BF16 (2^-8).
"""
import pytest
import torch

from bit_kv_cache_int2_gb300 import build as B
from bit_kv_cache_int2_gb300 import oscar

pytestmark = pytest.mark.gpu

from kv8_scenario import Pair, dense  # noqa: E402

HKV, G, N = 8, 4, 6000
KINDS = [oscar.KV8_E4M3, oscar.KV8_INT8]


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    oscar.lib()


def fill(kind, batch, n, size, lead, at, small, seed):
    """A pair whose n tokens have values of about `size`; token `at` (if any) has a
    logit `lead` nats above the others for every query head and `small` times the
    values of the others.  (pair, queries)"""
    p = Pair(kind, HKV, G, batch, -(-n // 64), seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    base = rand(batch, 1, HKV, 128)
    q = (base.view(batch, HKV, 1, 128) + 0.05 * rand(batch, HKV, G, 128)).bfloat16()
    k, v = 0.3 * rand(batch, n, HKV, 128), size * rand(batch, n, HKV, 128)
    if at is not None:
        k[:, at:at + 1] = base * (lead * 128 ** 0.5 / base.square().sum(-1, keepdim=True))
        v[:, at] *= small
    oscar.oscar_append_kv8(p.ctx, p.cache, kind, k.bfloat16(), v.bfloat16(), n, batch, weights=p.weights)
    return p, q.view(batch, HKV * G, 128)


def check(p, q, out, lse):
    qd, od = q.double().view(p.B, HKV, G, 128), out.double().view(p.B, HKV, G, 128)
    ld = lse.double().view(p.B, HKV, G)
    for b in range(0, p.B, 4):
        L, H = int(p.cache["seq_lens"][b]), int(p.cache["hist_lens"][b])
        for h in range(HKV):
            K, V = dense(p, b, h)
            z = qd[b, h] @ K.T / 128 ** 0.5
            w = torch.softmax(z, 1)
            ref, rl = w @ V, torch.logsumexp(z, 1)
            ds = 2.0 ** -16 * (qd[b, h].abs() @ K.abs().T).amax(1, keepdim=True) / 128 ** 0.5 + 2.0 ** -19
            rel = 2.0 ** -11 + 2 * ds + 2.0 ** -16 + (L / 128 + 40) * 2.0 ** -22
            A = V.abs().amax(1)
            A[64:64 + H] = A[64:64 + H].view(-1, 16).amax(1).repeat_interleave(16)
            lim = rel * (w @ V.abs()) + L * 2.0 ** -39 * (w * A).amax(1, keepdim=True)
            lim = lim + 2.0 ** -8 * (ref.abs() + lim)
            worst = float(((od[b, h] - ref).abs() / lim).max())
            assert worst <= 1, (b, h, worst)
            assert bool(((ld[b, h] - rl).abs() <= ds[:, 0] + 2.0 ** -18 + 2.0 ** -22 * rl.abs()).all()), (b, h)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [2.0 ** 40, 1.0, 2.0 ** -6, 2.0 ** -10, 2.0 ** -17, 2.0 ** -30, 2.0 ** -90])
def test_decode_follows_values_of_any_size(kind, size):
    p, q = fill(kind, 19, N, size, 0, None, 1, seed=1)
    try:
        check(p, q, *p.decode(q))
        assert oscar.oscar_get_error(p.ctx) == 0
    finally:
        p.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size,lead,small", [(1.0, 14, 0.0), (1.0, 14, 2.0 ** -7), (0.05, 8, 0.01), (0.02, 10, 0.01),
                                             (2.0 ** -17, 6, 1.0), (1.0, 24, 0.0)])
@pytest.mark.parametrize("at", [0, 40, 1000, N - 200, N - 1])
def test_decode_with_a_token_that_leads(kind, size, lead, small, at):
    """In the sink, the history, the window; the last token; 24 nats are 2^35."""
    p, q = fill(kind, 19, N, size, lead, at, small, seed=at + lead)
    try:
        check(p, q, *p.decode(q))
        assert oscar.oscar_get_error(p.ctx) == 0
    finally:
        p.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("where", [slice(0, 64), slice(N - 240, N)])
def test_decode_with_a_region_of_other_size(kind, where):
    """The sink's or the window's values 2^20 times and 2^-20 times the history's, and their logits higher."""
    for size in (2.0 ** -20, 2.0 ** 20):
        p, q = fill(kind, 19, N, 1.0, 0, None, 1, seed=7)
        try:
            g = torch.Generator(device="cuda").manual_seed(9)
            n = where.stop - where.start
            k = 0.3 * torch.randn(19, HKV, n, 128, device="cuda", generator=g) + 0.4 * q.view(19, HKV, G, 128)[:, :, :1]
            v = size * torch.randn(19, HKV, n, 128, device="cuda", generator=g)
            if where.start == 0:
                p.cache["sink_k"].copy_(k)
                p.cache["sink_v"].copy_(v)
            else:
                slots = (torch.arange(where.start, where.stop, device="cuda") - 64) % 256
                p.cache["ring_k"][:, :, slots] = k.bfloat16()
                p.cache["ring_v"][:, :, slots] = v.bfloat16()
            check(p, q, *p.decode(q))
            assert oscar.oscar_get_error(p.ctx) == 0
        finally:
            p.close()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -60, 2.0 ** 60])
@pytest.mark.parametrize("at", [3, N - 30])
def test_decode_shows_a_bad_value_in_its_own_channel(bad, size, at, kind=oscar.KV8_INT8):
    """One infinity or NaN among the values of the sink or window: the other channels
    are as without, whatever the values' size."""
    p, q = fill(kind, 19, N, size, 0, None, 1, seed=11)
    try:
        region, row = ("sink_v", at) if at < 64 else ("ring_v", (at - 64) % 256)
        was = p.cache[region][:, :, row, 5].clone()
        p.cache[region][:, :, row, 5] = bad
        out, lse = p.decode(q)
        assert not bool(torch.isfinite(out[..., 5]).any())
        p.cache[region][:, :, row, 5] = was
        out[..., 5] = p.decode(q)[0][..., 5]
        check(p, q, out, lse)
        assert oscar.oscar_get_error(p.ctx) == 0
    finally:
        p.close()
