"""Host side of the 8-bit-history calls: layout, refusals (nothing is launched),
and the oracle's own pins."""
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


def test_layout(lib):
    cfg = oscar.make_config(1, 32, 8, max_batch=4, max_pages_per_req=100, num_pages=400)
    info = oscar.oscar_layout_kv8(cfg)
    assert (info.head_bytes, info.page_bytes, info.off_scales) == (16416, 8 * 16416, 16384)
    assert info.weights_floats == 16 + 400
    # partial records of 4 x 132 floats, and 20 bytes per (page, query head) for the weights
    assert info.scratch_bytes >= 4 * 8 * (4 * 132 * 4 + 108 * 4 * 20)
    big = oscar.oscar_layout_kv8(oscar.make_config(1, 64, 8, max_batch=4096, max_pages_per_req=6250, num_pages=9))
    assert big.scratch_bytes < 256 << 20  # long batches run in several launches over one scratch
    cfg.head_dim = 64
    with pytest.raises(oscar.OscarError) as e:
        oscar.oscar_layout_kv8(cfg)
    assert e.value.status == oscar.ERR_UNSUPPORTED
    assert lib.oscar_layout_kv8(None, ctypes.byref(info)) == oscar.ERR_INVALID_ARG


def test_null_arguments_are_refused(lib):
    cs = oscar.oscar_cache()
    fake = ctypes.c_void_p(256)
    assert lib.oscar_append_kv8(None, ctypes.byref(cs), 0, fake, fake, 1, None, 1, None) == oscar.ERR_INVALID_ARG
    assert lib.oscar_decode_kv8(None, ctypes.byref(cs), 0, fake, fake, None, None, 1.0, fake, 1 << 20, 1,
                                None) == oscar.ERR_INVALID_ARG
    assert lib.oscar_evict_kv8(None, ctypes.byref(cs), fake, 0, fake, 1 << 20, 1, None) == oscar.ERR_INVALID_ARG


def test_kernel_names_cover_the_profile_ids():
    assert sorted(oscar.KERNEL_NAMES) == list(range(13))


def test_oracle_e4m3_is_the_format():
    t = K8.E4M3
    assert t[0x7E] == 448 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[0x38] == 1 and t[0xB8] == -1
    torch = pytest.importorskip("torch")
    b = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(b.view(torch.float8_e4m3fn).double().numpy(), t)


def test_oracle_encode_rounds_to_the_nearest_code():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(0, 0.02, 4000), K8.E4M3[:126],
                        (K8.E4M3[:126] + K8.E4M3[1:127]) / 2, [-0.0, 448.0, -448.0]])
    want = torch.from_numpy(y).float().to(torch.float8_e4m3fn)
    ok = y == y.astype(np.float32)  # the others are rounded twice by torch
    got = K8.E4M3[K8.encode(y, 0)]
    np.testing.assert_array_equal(got[ok], want.double().numpy()[ok])
    err = np.abs(got - y)
    assert (err <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10)).all()
    z = np.array([0.5, 1.5, -2.5, 126.5, -127.0])
    np.testing.assert_array_equal(K8.encode(z, 1).view(np.int8), [0, 2, -2, 126, -127])


def test_oracle_block_order_is_a_permutation():
    x = np.random.default_rng(1).integers(0, 256, (16, 128)).astype(np.uint8)
    for side in (0, 1):
        assert sorted(K8.PLACE[side]) == list(range(2048))
        np.testing.assert_array_equal(K8.unpack(K8.pack(x, side), side), x)
    # by hand: K byte 512c + 16(4g + q) + 8s + 4h + 2r + l at (c, g, q, s, h, r, l) = (2, 5, 3, 1, 0, 1, 1)
    i = 512 * 2 + 16 * (4 * 5 + 3) + 8 + 2 + 1
    assert K8.PLACE[0][i] == (8 + 5) * 128 + 64 + 24 + 4 + 1
    assert K8.PLACE[1][i] == (2 * 3 + 1) * 128 + 80 + 8 + 2 + 1


def test_oracle_window_holds_241_to_256_tokens_once_full():
    r = K8.Request(1, 1)
    z = np.zeros((1, 128))
    for n in range(1, 700):
        r.append(z, z)
        assert r.L == n and r.H % 16 == 0
        assert r.H == max(0, -(-(n - 320) // 16) * 16)
        assert len(r.window) <= 256


def test_serving_page_account_covers_every_step():
    """pages_needed_kv8 is the largest page count along the way, with and
    without a budget, by playing the rule step by step."""
    import random

    from bit_kv_cache_int2_gb300.serving import kv8_history, pages_needed_kv8

    rng = random.Random(0)
    for _ in range(300):
        prefix, gen = rng.randint(0, 3000), rng.randint(1, 1500)
        budget = rng.choice([None, 0, rng.randint(0, 2500)])
        L, H = prefix, kv8_history(prefix)
        peak = H
        for _ in range(gen):
            L += 1
            H = max(H, kv8_history(L))
            peak = max(peak, H)
            if budget is not None and H - budget >= 256:
                gone = (H - budget) // 256 * 256
                L, H = L - gone, H - gone
        want = pages_needed_kv8(prefix, gen, budget=budget)
        assert -(-peak // 64) <= want, (prefix, gen, budget)
        if budget is None:
            assert want == -(-peak // 64)


def test_scheduler_returns_pages_a_backend_no_longer_needs():
    from bit_kv_cache_int2_gb300.serving import PagePool, Request, Scheduler

    class Shrinking:
        def __init__(self):
            self.left = {}

        def admit(self, slot, req):
            self.left[slot] = len(req.pages)

        def move(self, src, dst):
            self.left[dst] = self.left.pop(src)

        def step(self, active):
            for slot in range(len(active)):
                self.left[slot] = max(1, self.left[slot] - 1)

        def kept_pages(self, slot):
            return self.left[slot]

    pool = PagePool(12)
    sched = Scheduler(pool, 2, Shrinking(), 16, need=lambda prefix, gen: 6)
    for i in range(5):
        sched.submit(Request(rid=i, prefix=0, gen=4 + i))
    done = sched.run()
    assert sorted(r.rid for r in done) == list(range(5))
    assert pool.available == 12 and len(set(pool._free)) == 12
