"""8-bit products whose two scales (or whose scale and routing weight) multiply
to something that float32 does not hold well, while every value does."""
import numpy as np
import pytest
import torch

from lowbit_util import U, half_step, make_routing
from mixture_experts_projections_b200 import rom
from test_q8_proj import acc_err, products
from test_q8_whole_tiles import gated

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
gpu = pytest.mark.gpu

# Powers of two of the rows' scale, the features', the codes of both and the
# routing weight. Each partial product of value = ((acc * row) * feature) * weight
# is in float32's range; acc is a sum of K = 256 products of codes.
RANGES = {
    "subnormal product of the scales": (-90, -50, 7, 7, 0),
    "product of the scales beyond float32's range": (70, 58, -8, -8, 0),
    "weight times row scale below float32's range": (-90, 80, 6, 0, -70),
    "small row scale, large feature scale": (-110, 60, 6, 0, 0),
}


def rows(shape, exponent, gen):
    """e4m3 codes of magnitude 2^exponent, one in eight of the rows zero."""
    v = torch.randn(shape, generator=gen).clamp(-3, 3) * 2.0 ** exponent
    v[..., 0::8, :] = 0
    return v.to(E4M3)


def scales(shape, exponent, gen):
    """No powers of two: a subnormal product would keep those exact."""
    return (1 + torch.rand(shape, generator=gen)) * 2.0 ** exponent


@gpu
@pytest.mark.parametrize("what", RANGES)
@pytest.mark.parametrize("T,E,k", [(100, 4, 1), (300, 3, 1), (60, 4, 2), (300, 3, 2)])
def test_the_value_is_as_good_as_its_factors(T, E, k, what):
    K, N = 256, 128
    row_e, feature_e, a_e, w_e, weight_e = RANGES[what]
    gen = torch.Generator().manual_seed(T + k)
    idx, w, order, off = make_routing(T, E, k, T)
    w = w * np.float32(2.0 ** weight_e)
    R = T * k
    a, sa = rows((R, K), a_e, gen), scales((R,), row_e, gen)
    ws = [(rows((E, N, K), w_e, gen), scales((E, N), feature_e, gen)) for _ in range(2)]
    offd, slotd, wd = (torch.from_numpy(t).cuda() for t in (off, order, w))
    da = [a.cuda(), sa.cuda()]
    d0, d1 = ([t.cuda() for t in p] for p in ws)
    slots = torch.from_numpy(order.astype(np.int64))
    r = torch.from_numpy(w).double().flatten()[slots][:, None]
    (u, mu), (z, mz) = (products(a, sa, *p, off, E) for p in ws)
    eu, ez = acc_err(K, mu), acc_err(K, mz)
    assert u.abs().max() < 2.0 ** 126 and mu[mu > 0].min() > 2.0 ** -125

    uz = torch.full((2, R, N), float("nan"), device="cuda")
    rom.rom_expert_proj_q8(rom.ROM_PROJ_CONV_GATE_SLOTS, *da, *d0, *d1, k, offd, slotd, wd, uz)
    got = uz.cpu().double()
    assert ((got[0][slots] - u).abs() <= eu).all() and ((got[1][slots] - z).abs() <= ez).all()
    one = torch.full((R, N), float("nan"), device="cuda")
    rom.rom_expert_proj_q8(rom.ROM_PROJ_SLOTS, *da, *d0, None, None, k, offd, slotd, wd, one)
    tol = r * (eu + 2 * U * u.abs()) + 2.0 ** -149
    assert ((one.cpu().double()[slots] - r * u).abs() <= tol).all()
    if k == 1:
        h16 = half_step(BF16)
        o = torch.full((T, N), float("nan"), dtype=BF16, device="cuda")
        rom.rom_expert_proj_q8(rom.ROM_PROJ_OUT, *da, *d0, None, None, 1, offd, slotd, wd, o)
        # below 2^-126 bf16 (7 bits behind the point) goes in steps of 2^-133: half of one
        err = tol * (1 + h16) + h16 * (r * u).abs() + 2.0 ** -134
        assert ((o.cpu().double()[slots] - r * u).abs() <= err).all()
        if u.abs().max() < 2.0 ** 60:  # (u * z is in range)
            h = torch.full((R, N), float("nan"), dtype=BF16, device="cuda")
            rom.rom_expert_proj_q8(rom.ROM_PROJ_CONV_GATE, *da, *d0, *d1, 1, offd, slotd, wd, h)
            ref, err = gated(u, z, eu, ez)
            # (products below float32's normal range: a step of the subnormals, in bf16)
            assert ((h.cpu().double() - ref).abs() <= err + 2.0 ** -126).all()
    torch.cuda.synchronize()
    assert rom.rom_get_status() == 0
