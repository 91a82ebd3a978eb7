"""YaRN's speeds where the ramp ends behind the last pair, against numbers worked out by hand.

The ramp's ends are clamped to 0 and dims - 1 while the pairs are numbered 0 .. dims / 2 - 1.  With theta 1e4 and dims 128
pair i has w = 10^(-i / 16) and i(t) = 128 ln(trained / 2 pi t) / 18.420681 = 6.948711 ln(trained / 2 pi t):
  trained 131072: i(32) = 6.948711 ln 651.90 = 45.03, i(1) = 6.948711 ln 20860.8 = 69.11, so the ramp goes from 45 to 70.
  trained  65536: i(32) = 40.21, i(1) = 64.29: from 40 to 65.
and with dims 16, w = 10^(-i / 2) and i(t) = 0.868589 ln(trained / 2 pi t):
  trained  32768: i(32) = 4.42, i(1) = 7.43: from 4 to 8.
A pair keeps c = 1 - (i - a) / (b - a) of its speed and 1 / factor of the rest."""
import math

import pytest

from bit_kv_cache_int2_gb300 import build as B
from bit_kv_cache_int2_gb300 import oscar
from oracle import rope_oracle as R


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return oscar.lib()


CASES = [
    (128, 131072.0, 4.0, {44: 1.77827941e-3, 45: 1.53992653e-3, 57: 1.75258857e-4, 63: 5.31199713e-5}),  # 1, 1, 0.64, 0.46
    (128, 65536.0, 8.0, {40: 3.16227766e-3, 63: 2.25182487e-5}),                                           # 1, 0.195
    (16, 32768.0, 2.0, {4: 1.0e-2, 5: 2.76699295e-3, 7: 1.97642354e-4}),                                    # 1, 0.875, 0.625
]


@pytest.mark.parametrize("dims,trained,factor,speeds", CASES)
def test_ramp_that_ends_behind_the_last_pair(dims, trained, factor, speeds):
    t = oscar.make_rope(oscar.ROPE_HALF, dims, 1e4, oscar.ROPE_YARN, factor=factor, trained=trained)
    w = R.speeds(dims, 1e4, R.YARN, factor, trained)
    for i, want in speeds.items():
        assert abs(t.turn[i] / 2.0 ** 64 * 2 * math.pi / want - 1) < 1e-8, i
        assert abs(w[i] / want - 1) < 1e-8, i


@pytest.mark.parametrize("theta,trained", [(1e4, 131072.0), (1e4, 65536.0), (5e5, 4194304.0), (1e6, 32768.0), (1e4, 8192.0), (1.5, 100.0)])
@pytest.mark.parametrize("dims", [16, 64, 112, 128])
def test_table_is_the_oracles(dims, theta, trained):
    t = oscar.make_rope(oscar.ROPE_HALF, dims, theta, oscar.ROPE_YARN, factor=4.0, trained=trained)
    for i, w in enumerate(R.speeds(dims, theta, R.YARN, 4.0, trained)):
        assert abs(t.turn[i] / 2.0 ** 64 - w / (2 * math.pi)) <= 2.0 ** -44 * max(w / (2 * math.pi), 2.0 ** -20), i


@pytest.mark.parametrize("size", [1e39, -1e300, 3.5e38])
def test_a_size_that_32_bits_do_not_hold_is_refused(size):
    with pytest.raises(oscar.OscarError) as e:
        oscar.make_rope(size=size)
    assert e.value.status == oscar.ERR_INVALID_ARG
    assert oscar.make_rope(size=3e38).size == pytest.approx(3e38, rel=1e-6)
