"""The 8-bit products over several tiles per SM pair: whole 256-column tiles,
half tiles behind whole waves, the next tile's scales fetched during the stores,
both accumulators in turn and the ring over tile boundaries. (The cases of
test_q8_proj.py have one half tile per pair.)"""
import numpy as np
import pytest
import torch

from lowbit_util import U, half_step, make_routing
from mixture_experts_projections_b200 import rom
from test_q8_proj import acc_err, codes, products

BF16 = torch.bfloat16
gpu = pytest.mark.gpu

# T, K, cols (column tiles), cut (128 columns of the last one missing), E, k, pin, waves:
# tiles over the 74 pairs as (whole waves, how the last, partial one runs).
CASES = [
    (1500, 160, 7, False, 4, 1, None, (0, "whole")),    # 56 tiles: more than half a wave
    (1900, 48, 11, False, 4, 1, None, (1, "halves")),   # one K block: the ring spans tiles
    (1900, 1040, 11, True, 4, 1, None, (1, "halves")),  # nine K blocks: it goes round in a tile
    (1300, 272, 13, False, 8, 2, 3, (2, "halves")),     # uneven, top-2, 169 tiles
    (1300, 144, 15, True, 8, 2, 3, (2, "whole")),       # 195 tiles
    (2300, 144, 20, False, 5, 1, 1, (2, "halves")),     # every row on one expert, the others empty
]


def waves(off, cols):
    """(whole waves, form of the partial one) of 256-row tiles on 74 SM pairs."""
    tiles = cols * sum(-(-int(n) // 256) for n in np.diff(off))
    full, rest = divmod(tiles, 74)
    return full, "none" if not rest else "halves" if rest <= 37 else "whole"


def case(T, K, N, E, k, pin, m):
    """Routing, codes of the sorted rows and of m matrices, on CPU and GPU."""
    gen = torch.Generator().manual_seed(T + K)
    idx, w, order, off = make_routing(T, E, k, T, pin)
    a, sa = codes((T * k, K), gen)
    ws = [t for _ in range(m) for t in codes((E, N, K), gen)]
    dev = [t.cuda() for t in (a, sa, *ws)]
    return w, order, off, (a, sa, ws), dev, [torch.from_numpy(t).cuda() for t in (off, order, w)]


@pytest.mark.parametrize("T,K,cols,cut,E,k,pin,expect", CASES)
def test_cases_have_these_waves(T, K, cols, cut, E, k, pin, expect):
    _, _, _, off = make_routing(T, E, k, T, pin)
    assert waves(off, cols) == expect
    assert T * k > 64 * E  # the pair kernel's, not the few rows'


@gpu
@pytest.mark.parametrize("T,K,cols,cut,E,k,pin,expect", CASES)
def test_one_matrix(T, K, cols, cut, E, k, pin, expect):
    N = 256 * cols - (128 if cut else 0)
    w, order, off, (a, sa, ws), d, (offd, slotd, wd) = case(T, K, N, E, k, pin, 1)
    v, m = products(a, sa, *ws, off, E)
    e = acc_err(K, m)
    R = T * k
    slots = torch.from_numpy(order.astype(np.int64))
    r = torch.from_numpy(w).double().flatten()[slots][:, None]
    h16 = half_step(BF16)
    out = torch.full((R, N), float("nan"), device="cuda")
    rom.rom_expert_proj_q8(rom.ROM_PROJ_SLOTS, *d, None, None, k, offd, slotd, None, out)
    assert ((out.cpu().double()[slots] - v).abs() <= e).all()
    weighted = r * (e + 2 * U * v.abs())
    if k > 1:
        out.fill_(float("nan"))
        rom.rom_expert_proj_q8(rom.ROM_PROJ_OUT, *d, None, None, k, offd, slotd, wd, out)
        assert ((out.cpu().double()[slots] - r * v).abs() <= weighted).all()
    else:
        o = torch.full((T, N), float("nan"), dtype=BF16, device="cuda")
        rom.rom_expert_proj_q8(rom.ROM_PROJ_OUT, *d, None, None, k, offd, slotd, wd, o)
        assert ((o.cpu().double()[slots] - r * v).abs() <= weighted * (1 + h16) + h16 * (r * v).abs()).all()
    torch.cuda.synchronize()
    assert rom.rom_get_status() == 0


def gated(u, z, eu, ez):
    """float64 u * SiLU(z) and how far the kernels' may be from it, for every z.
    The fast exponential is off by 2 + 1.173 |z| steps of 2^-23 (105 of them at
    the largest |z| that matters), the quotient and the two products by 4 more:
    109 * 2^-23 < 2^-16. Where e^-z overflows or its reciprocal is no normal
    number the quotient is 0, and |u SiLU(z)| below 2^-126 |u z| < 1e-30 |u z|."""
    sig = torch.sigmoid(z)
    ref = u * z * sig
    e = eu * (z * sig).abs() + 1.1 * ez * (u.abs() + eu) + 2.0 ** -16 * ref.abs()
    h16 = half_step(BF16)
    return ref, e * (1 + h16) + h16 * ref.abs() + 1e-30 * (u * z).abs()


@gpu
@pytest.mark.parametrize("T,K,cols,cut,E,k,pin,expect", CASES)
def test_two_matrices(T, K, cols, cut, E, k, pin, expect):
    N = 128 * cols
    _, order, off, (a, sa, ws), d, (offd, slotd, wd) = case(T, K, N, E, k, pin, 2)
    u, mu = products(a, sa, *ws[:2], off, E)
    z, mz = products(a, sa, *ws[2:], off, E)
    eu, ez = acc_err(K, mu), acc_err(K, mz)
    R = T * k
    slots = torch.from_numpy(order.astype(np.int64))
    uz = torch.full((2, R, N), float("nan"), device="cuda")
    rom.rom_expert_proj_q8(rom.ROM_PROJ_CONV_GATE_SLOTS, *d, k, offd, slotd, wd, uz)
    got = uz.cpu().double()
    assert ((got[0][slots] - u).abs() <= eu).all() and ((got[1][slots] - z).abs() <= ez).all()
    if k == 1:
        h = torch.full((R, N), float("nan"), dtype=BF16, device="cuda")
        rom.rom_expert_proj_q8(rom.ROM_PROJ_CONV_GATE, *d, k, offd, slotd, wd, h)
        ref, err = gated(u, z, eu, ez)
        assert ((h.cpu().double() - ref).abs() <= err).all()
        assert (z < -90).any() and (z > 90).any()  # (both ends of the exponential's range are met)
    torch.cuda.synchronize()
    assert rom.rom_get_status() == 0


@gpu
@pytest.mark.parametrize("T,K,N,E", [(200, 256, 128, 4), (300, 1008, 384, 5), (1500, 256, 128, 8)])
def test_gate_of_few_rows_and_of_half_tiles_at_every_z(T, K, N, E):
    """As above for the few rows' kernel (the first two) and for half tiles."""
    _, order, off, (a, sa, ws), d, (offd, slotd, wd) = case(T, K, N, E, 1, None, 2)
    u, mu = products(a, sa, *ws[:2], off, E)
    z, mz = products(a, sa, *ws[2:], off, E)
    h = torch.full((T, N), float("nan"), dtype=BF16, device="cuda")
    rom.rom_expert_proj_q8(rom.ROM_PROJ_CONV_GATE, *d, 1, offd, slotd, wd, h)
    ref, err = gated(u, z, acc_err(K, mu), acc_err(K, mz))
    assert ((h.cpu().double() - ref).abs() <= err).all()
    assert (z < -90).any() and (z > 90).any()
