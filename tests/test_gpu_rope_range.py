"""Head norms of heads whose squares leave the range of 32 bits, against the 64-bit oracle with the ordinary
heads' limits (test_gpu_rope.check; they are relative to the result)."""
import pytest
import torch

from bit_kv_cache_int2_gb300 import build as B
from bit_kv_cache_int2_gb300 import oscar
from oracle import rope_oracle as R

pytestmark = pytest.mark.gpu

from test_gpu_rope import check, outputs, setup  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()
    oscar.lib()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hkv,G,T", [(2, 4, 5), (1, 1, 3), (3, 2, 40)])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-20, 1e-6, 1e6])
def test_heads_of_any_size(interleaved, Hkv, G, T, eps):
    """Heads of 2^-100 to 2^120 beside ordinary ones, whose results stay as they are."""
    ctx, _, gam = setup(Hkv, G, 2, T, norm=True)
    try:
        g, heads = torch.Generator().manual_seed(T), Hkv * (G + 2)
        table = oscar.make_rope(oscar.ROPE_INTERLEAVED if interleaved else oscar.ROPE_HALF, 128, 1e4)
        pos, gd = torch.tensor([3, 70_000], dtype=torch.int32), [y.cuda() for y in gam]
        x = torch.randn(2, T, heads, 128, generator=g)
        size = torch.tensor([0, 70, -80, 120, 0, -40, 62, -62, 100, -100, 0])[torch.arange(2 * T * heads) % 11].view(2, T, heads, 1)
        y = (x.double() * 2.0 ** size.double()).bfloat16()
        plain, got = outputs(Hkv, G, 2, T), outputs(Hkv, G, 2, T)
        oscar.oscar_rope(ctx, table, x.bfloat16().cuda(), pos.cuda(), T, *plain, 2, *gd, eps)
        oscar.oscar_rope(ctx, table, y.cuda(), pos.cuda(), T, *got, 2, *gd, eps)
        same = (size[..., 0] == 0).cuda()
        for a, b, at in ((got[0], plain[0], same[:, :, :Hkv * G]), (got[1], plain[1], same[:, :, Hkv * G:Hkv * (G + 1)])):
            assert torch.equal(a[at], b[at])
        check(y.view(2, T, -1), pos, gam, got, Hkv, G, R.speeds(128, 1e4), 1.0, interleaved, eps)
    finally:
        oscar.oscar_destroy(ctx)


def test_heads_of_zeros_and_with_values_that_are_not_finite():
    """Zeros stay zeros with an eps; without one, and with an infinity or NaN, what the formula gives; other heads stay."""
    ctx, _, _ = setup(1, 2, 1, 4)
    try:
        x = torch.randn(1, 4, 4, 128, generator=torch.Generator().manual_seed(0))
        one, pos, table = torch.ones(128, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), oscar.make_rope()
        for eps in (0.0, 1e-6):
            clean, got = outputs(1, 2, 1, 4), outputs(1, 2, 1, 4)
            oscar.oscar_rope(ctx, table, x.bfloat16().cuda(), pos, 4, *clean, 1, one, one, eps)
            y = x.clone()
            y[0, 0, 0], y[0, 1, 1], y[0, 2, 2, 9], y[0, 3, 0, 77] = 0, 2.0 ** -130, float("inf"), float("nan")
            oscar.oscar_rope(ctx, table, y.bfloat16().cuda(), pos, 4, *got, 1, one, one, eps)
            if eps:
                assert bool((got[0][0, 0, 0] == 0).all()) and bool((got[0][0, 1, 1].abs() < 2.0 ** -119).all())
            else:
                assert bool(torch.isnan(got[0][0, 0, 0]).all())
                norm = got[0][0, 1, 1].double().square().sum()  # turning keeps it: 128
                assert abs(float(norm) / 128 - 1) < 2.0 ** -6
            assert bool(torch.isnan(got[1][0, 2, 0, [9, 73]]).all()) and bool(torch.isnan(got[0][0, 3, 0]).all())
            rest = torch.ones(4, 2, dtype=torch.bool)
            rest[0, 0] = rest[1, 1] = rest[3, 0] = False
            assert torch.equal(got[0][0][rest], clean[0][0][rest]) and torch.equal(got[1][0, [0, 1, 3]], clean[1][0, [0, 1, 3]])
    finally:
        oscar.oscar_destroy(ctx)
