"""Host side of the prompt's calls on the 8-bit-history cache: refusals (nothing is launched), the
scratch size, the oracle's chunk, and the serving loop's prompt in chunks with a fake device."""
import ctypes

import numpy as np
import pytest

from bit_kv_cache_int2_gb300 import build as B
from bit_kv_cache_int2_gb300 import oscar
from oracle import kv8_oracle as K8


@pytest.fixture(scope="module")
def lib():
    B.build()
    return oscar.lib()


def test_null_arguments_are_refused(lib):
    cs, fake, bad = oscar.oscar_cache(), ctypes.c_void_p(256), oscar.ERR_INVALID_ARG
    assert lib.oscar_prefill_kv8(None, ctypes.byref(cs), 0, fake, fake, fake, 1, fake, None, fake, 1 << 30, 1, None) == bad
    assert lib.oscar_read_kv8(None, ctypes.byref(cs), 0, 0, 1, 0, fake, fake, 1, None) == bad


def test_scratch_size(lib):
    def size(**kw):
        cfg = oscar.make_config(1, 32, 8, **{**dict(max_batch=4, max_pages_per_req=100, num_pages=400), **kw})
        return lib.oscar_prefill_kv8_scratch_bytes(ctypes.byref(cfg))

    # two records of 256 rows of 132 floats for each CTA, whatever the batch and the lengths
    assert size() == size(max_batch=4096) == size(max_pages_per_req=6250)
    assert 2 * 256 * 130 * 4 < size() < 64 << 20
    assert lib.oscar_prefill_kv8_scratch_bytes(None) == 0
    cfg = oscar.make_config(1, 32, 8, max_batch=4, max_pages_per_req=100, num_pages=400)
    cfg.head_dim = 64
    assert lib.oscar_prefill_kv8_scratch_bytes(ctypes.byref(cfg)) == 0
    with pytest.raises(oscar.OscarError):
        oscar.alloc_scratch_kv8(cfg, "cpu", prefill=True)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("L", [0, 40, 700])
def test_the_oracles_chunk_is_its_attention_token_by_token(kind, L):
    """While the window has room the chunk's tokens stay BF16, so appending them one by one and attending gives
    the same."""
    rng = np.random.default_rng(L)
    one, many = K8.Request(2, kind), K8.Request(2, kind)
    for _ in range(L):
        kv = rng.normal(size=(2, 2, 128))
        one.append(*kv)
        many.append(*kv)
    T = (256 - len(one.window)) if len(one.sink) == 64 else 12
    q, k, v = rng.normal(size=(T, 2, 3, 128)), rng.normal(size=(T, 2, 128)), rng.normal(size=(T, 2, 128))
    out, lse, ps = many.chunk(q, k, v)
    assert T > 0
    for t in range(T):
        one.append(k[t], v[t])
        o, l, p = one.attend(q[t])
        np.testing.assert_allclose(out[t], o, rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(lse[t], l, rtol=1e-12)
        np.testing.assert_allclose(ps[:, t, :, :L + t + 1], p, rtol=1e-12, atol=1e-15)
        assert not ps[:, t, :, L + t + 1:].any()


@pytest.mark.parametrize("prefix,chunk", [(0, 8), (1, 8), (8, 8), (29, 8), (5, 100)])
def test_a_prompt_is_taken_in_chunks(monkeypatch, prefix, chunk):
    """The order and the sizes of the calls for a prompt and a step: positions, attention before the append."""
    torch = pytest.importorskip("torch")
    from bit_kv_cache_int2_gb300 import serving

    calls = []
    cfg = oscar.make_config(1, 4, 2, max_batch=2, max_pages_per_req=4, num_pages=8)
    cache = dict(page_table=torch.zeros(2, 4, dtype=torch.int32), seq_lens=torch.zeros(2, dtype=torch.int32),
                 hist_lens=torch.zeros(2, dtype=torch.int32), **{x: torch.zeros(2, 1) for x in ("sink_k", "sink_v", "ring_k", "ring_v")})

    def rope(ctx, table, rows, place, T, q, k, v, batch, gq, gk, eps):
        assert rows.shape == (batch, T, 8, 128) and q.shape == (batch, T, 4, 128) and k.shape == v.shape == (batch, T, 2, 128)
        calls.append(("turn", place.tolist(), T, batch, float(rows[0, 0, 0, 0])))

    monkeypatch.setattr(oscar, "oscar_rope", rope)
    monkeypatch.setattr(oscar, "oscar_prefill_kv8", lambda ctx, c, kind, q, k, v, T, out, lse, sc, b: calls.append(("attend", T)))
    monkeypatch.setattr(oscar, "oscar_append_kv8", lambda ctx, c, kind, k, v, T, b, weights=None: calls.append(("append", T)))
    monkeypatch.setattr(oscar, "alloc_scratch_kv8", lambda cfg, dev, prefill=False: None)
    monkeypatch.setattr(oscar, "bind_step_kv8", lambda *a: lambda k, v, q, n: calls.append(("step", n)))

    def draw(req):
        return torch.arange(req.prefix + req.gen).bfloat16()[:, None, None].expand(-1, 8, 128)

    be = serving.DeviceBackend("int8", None, cfg, cache, draw, rope=dict(table=None), prompt_chunk=chunk,
                               on_prompt=lambda req, at, out: calls.append(("seen", at, len(out))))
    req = serving.Request(rid=0, prefix=prefix, gen=3, pages=[1])
    be.admit(0, req)
    want = []
    for at in range(0, prefix, chunk):
        T = min(chunk, prefix - at)
        want += [("turn", [at], T, 1, float(at)), ("attend", T), ("seen", at, T), ("append", T)]
    assert calls == want and be.place.tolist() == [prefix, 0]
    be.admit(1, serving.Request(rid=1, prefix=0, gen=2, pages=[2]))
    del calls[:]
    be.step([req, serving.Request(rid=1, prefix=0, gen=2, pages=[2])])
    assert calls == [("turn", [prefix, 0], 1, 2, float(prefix)), ("step", 2)] and be.place.tolist() == [prefix + 1, 1]
    be.move(1, 0)
    assert be.place.tolist() == [1, 1] and float(be.rows[0, 1, 0, 0]) == 1.0
    with pytest.raises(ValueError):
        serving.DeviceBackend("int2", None, cfg, cache, draw, rope=dict(table=None))
