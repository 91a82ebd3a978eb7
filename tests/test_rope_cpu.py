"""The host side of the rotary positions: the table against the oracle's speeds, and refusals."""
import ctypes

import numpy as np
import pytest

from bit_kv_cache_int2_gb300 import build as B
from bit_kv_cache_int2_gb300 import oscar
from oracle import rope_oracle as R


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return oscar.lib()


@pytest.mark.parametrize("dims", [16, 64, 96, 128])
@pytest.mark.parametrize("scaling,kw", [(R.PLAIN, {}), (R.LINEAR, dict(factor=4.0)), (R.NTK, dict(factor=8.0)),
                                        (R.BANDS, dict(factor=8.0, trained=8192.0)), (R.YARN, dict(factor=4.0, trained=32768.0)),
                                        (R.YARN, dict(factor=1.0, trained=10.0, low=3.0, high=5.0)),
                                        (R.LINEAR, dict(factor=0.001))])
def test_table_is_the_oracles(dims, scaling, kw):
    for theta in (1.5, 1e4, 1e6):
        t = oscar.make_rope(oscar.ROPE_HALF, dims, theta, scaling, **kw)
        w = R.speeds(dims, theta, scaling, **kw)
        got = np.array([t.turn[i] for i in range(64)], dtype=np.float64) / 2.0 ** 64
        turns = w / (2 * np.pi)
        # a pow, a log or two and a few operations in 64 bits: 2^-44 of the speed
        d = np.abs(got[:dims // 2] - turns % 1)
        assert (np.minimum(d, 1 - d) <= 2.0 ** -44 * np.maximum(turns, 2.0 ** -20)).all()
        assert not got[dims // 2:].any()
        assert abs(t.size - R.size(scaling, kw.get("factor", 1.0))) < 1e-7 and (t.dims, t.layout) == (dims, oscar.ROPE_HALF)


def test_oracle_against_plain_formulas():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 2, 128))
    for inter in (False, True):
        y = R.rope(x, [0, 5, 9], R.speeds(128, 1e4), inter)
        np.testing.assert_array_equal(y[0], x[0])
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
        i = np.arange(64)
        z = x[..., 2 * i] + 1j * x[..., 2 * i + 1] if inter else x[..., :64] + 1j * x[..., 64:]
        z = z * np.exp(1j * np.array([0, 5, 9])[:, None, None] * 1e4 ** (-i / 64))
        got = y[..., 2 * i] + 1j * y[..., 2 * i + 1] if inter else y[..., :64] + 1j * y[..., 64:]
        np.testing.assert_allclose(got, z, atol=1e-12)


def test_refusals(lib):
    def status(*a, **kw):
        with pytest.raises(oscar.OscarError) as e:
            oscar.make_rope(*a, **kw)
        return e.value.status

    bad = oscar.ERR_INVALID_ARG
    assert status(2) == bad and status(-1) == bad
    for dims in (0, 8, 24, 130, 144, -16):
        assert status(0, dims) == oscar.ERR_UNSUPPORTED
    for theta in (1.0, 0.0, -3.0, float("nan"), float("inf")):
        assert status(0, 128, theta) == bad
    assert status(0, 128, 1e4, 5) == bad and status(0, 128, 1e4, -1) == bad
    for f in (0.0, -1.0, float("nan"), float("inf")):
        assert status(0, 128, 1e4, oscar.ROPE_LINEAR, factor=f) == bad
    for kw in (dict(trained=0.0), dict(trained=float("nan")), dict(trained=100.0, low=2.0, high=2.0), dict(trained=1.0, low=-1.0, high=2.0),
               dict(trained=1.0, low=0.0, high=2.0), dict(trained=1.0, low=1.0, high=float("inf"))):
        assert status(0, 128, 1e4, oscar.ROPE_YARN, factor=2.0, **kw) == bad
    assert status(size=float("nan")) == bad
    t = oscar.oscar_rope_table()
    assert lib.oscar_make_rope(None, ctypes.byref(t)) == bad
    fake = ctypes.c_void_p(256)
    assert lib.oscar_rope(None, ctypes.byref(t), fake, 1024, fake, None, None, 0.0, 1, fake, fake, fake, 1, None) == bad
