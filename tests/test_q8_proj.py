"""The expert projections on 8-bit rows and weights, their dispatch, and the
block that runs on them."""
import ctypes

import numpy as np
import pytest
import torch

from lowbit_util import U, half_step, make_routing, rows_to_8bit
from mixture_experts_projections_b200 import rom
from mixture_experts_projections_b200.inputs import make_block_inputs
from oracle import rom_oracle as orc
from parity_util import assert_routing_matches, block_to_dev

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
FAKE = ctypes.c_void_p(1 << 20)
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_projections_b200.build import build
    build()
    return rom.load_library()


@pytest.mark.parametrize("kw,code", [
    (dict(proj=5), 1), (dict(proj=-1), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(k=2, R=7), 1),
    (dict(E=65), 1), (dict(k=9, E=16), 1), (dict(R=-1), 1), (dict(w1=None), 1), (dict(w1_scale=None), 1),
    (dict(w0_scale=None), 1), (dict(a_scale=None), 1), (dict(a_sorted=None), 1), (dict(out=None), 1),
    (dict(offsets=None), 1), (dict(proj=1, topk_w=None), 1), (dict(proj=4, sorted_slot=None), 1),
    (dict(proj=3, offsets=None, sorted_slot=None), 1), (dict(proj=3, offsets=None), 1),
    (dict(N=200), 2), (dict(K=24), 2), (dict(R=1 << 31), 2),
    (dict(out=ctypes.c_void_p((1 << 20) + 8)), 2), (dict(w0_scale=ctypes.c_void_p((1 << 20) + 4)), 2),
    (dict(w1_scale=ctypes.c_void_p((1 << 20) + 4)), 2),
])
def test_expert_proj_q8_rejects_bad_arguments(lib, kw, code):
    a = dict(proj=0, a_sorted=FAKE, a_scale=FAKE, R=256, K=64, w0=FAKE, w0_scale=FAKE, w1=FAKE,
             w1_scale=FAKE, N=256, E=8, k=1, offsets=FAKE, sorted_slot=FAKE, topk_w=FAKE, out=FAKE,
             stream=None)
    a.update(kw)
    assert lib.rom_expert_proj_q8(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), 1), (dict(k=3, E=2), 1), (dict(offsets=None), 1), (dict(x8_sorted=None), 1),
    (dict(x_scale=None), 1), (dict(scale_sorted=None), 1), (dict(ws_bytes=0), 3), (dict(Dm=24), 2),
    (dict(x8=ctypes.c_void_p((1 << 20) + 8)), 2),
])
def test_dispatch_q8_rejects_bad_arguments(lib, kw, code):
    a = dict(x8=FAKE, x_scale=FAKE, T=300, Dm=64, E=8, k=1, topk_idx=FAKE, ws=FAKE, ws_bytes=1 << 20,
             offsets=FAKE, sorted_slot=FAKE, slot_pos=FAKE, x8_sorted=FAKE, scale_sorted=FAKE, stream=None)
    a.update(kw)
    assert lib.rom_dispatch_q8(*a.values()) == code


# ------------------------------------------------------------------ numerics


def codes(shape, gen):
    """Random rows in 8 bits, with scales of several magnitudes."""
    v = torch.randn(shape, generator=gen) * 2.0 ** torch.randint(-6, 6, shape[:-1] + (1,), generator=gen)
    q, s = rows_to_8bit(v.reshape(-1, shape[-1]))
    return q.view(shape), s.view(shape[:-1])


def products(a, sa, w, sw, off, E):
    """float64 (values, sums of magnitudes) of the sorted rows."""
    A = a.double() * sa.double()[:, None]
    W = w.double() * sw.double()[..., None]
    v = torch.zeros(a.shape[0], w.shape[1], dtype=torch.float64)
    m = torch.zeros_like(v)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        v[r] = A[r] @ W[e].t()
        m[r] = A[r].abs() @ W[e].abs().t()
    return v, m


def acc_err(K, m):
    """K products of e4m3 codes are exact; their float32 sum, in any order and
    with roundings of up to a whole unit each (2 U), and the scales' products."""
    return (K + 4) * 2 * U * m


CASES = [
    # T, K, N, E, k, pin
    (1, 64, 128, 4, 1, None), (300, 128, 256, 8, 1, None), (77, 1008, 384, 5, 1, None),
    (64, 400, 128, 64, 8, None), (1500, 256, 128, 8, 1, None), (700, 272, 384, 33, 2, None),
    # both sides of the 64 rows per expert at which the kernels change
    (256, 144, 128, 4, 1, None), (257, 144, 128, 4, 1, None), (33, 96, 128, 2, 2, 1),
    (1300, 160, 256, 4, 1, 2), (2, 16, 128, 1, 1, None), (300, 2048, 640, 3, 2, None),
    (250, 144, 384, 4, 1, 3),  # few rows, several token tiles of one expert
]


@gpu
@pytest.mark.parametrize("T,K,N,E,k,pin", CASES)
def test_expert_proj_q8_matches_the_products(T, K, N, E, k, pin):
    gen = torch.Generator().manual_seed(T + K)
    idx, w, order, off = make_routing(T, E, k, T, pin)
    R = T * k
    a, sa = codes((R, K), gen)
    w0, s0 = codes((E, N, K), gen)
    w1, s1 = codes((E, N, K), gen)
    d = [t.cuda() for t in (a, sa, w0, s0, w1, s1)]
    offd, slotd, wd = (torch.from_numpy(t).cuda() for t in (off, order, w))
    u, mu = products(a, sa, w0, s0, off, E)
    z, mz = products(a, sa, w1, s1, off, E)
    eu, ez = acc_err(K, mu), acc_err(K, mz)
    slots = torch.from_numpy(order.astype(np.int64))
    h16 = half_step(BF16)

    # u and z in slot order
    uz = torch.full((2, R, N), float("nan"), device="cuda")
    rom.rom_expert_proj_q8(rom.ROM_PROJ_CONV_GATE_SLOTS, *d, k, offd, slotd, wd, uz)
    got = uz.cpu().double()
    assert ((got[0][slots] - u).abs() <= eu).all() and ((got[1][slots] - z).abs() <= ez).all()

    # one projection, unweighted and weighted
    out = torch.full((R, N), float("nan"), device="cuda")
    rom.rom_expert_proj_q8(rom.ROM_PROJ_SLOTS, *d[:4], None, None, k, offd, slotd, None, out)
    assert ((out.cpu().double()[slots] - u).abs() <= eu).all()
    r = torch.from_numpy(w).double().flatten()[slots][:, None]
    if k > 1:
        rom.rom_expert_proj_q8(rom.ROM_PROJ_OUT, *d[:4], None, None, k, offd, slotd, wd, out)
        assert ((out.cpu().double()[slots] - r * u).abs() <= r * (eu + 2 * U * u.abs())).all()
    else:
        o = torch.full((T, N), float("nan"), dtype=BF16, device="cuda")
        for proj in (rom.ROM_PROJ_OUT, rom.ROM_PROJ_INPROJ):
            rom.rom_expert_proj_q8(proj, *d[:4], None, None, k, offd, slotd, wd, o)
            e = r * (eu + 2 * U * u.abs())
            assert ((o.cpu().double()[slots] - r * u).abs() <= e * (1 + h16) + h16 * (r * u).abs()).all()
        h = torch.full((R, N), float("nan"), dtype=BF16, device="cuda")
        rom.rom_expert_proj_q8(rom.ROM_PROJ_CONV_GATE, *d, k, offd, slotd, wd, h)
        sig = torch.sigmoid(z)
        ref = u * z * sig
        # |d silu| <= 1.1; the fast exponential and quotient: 2^-20 (|z| <= 88
        # bounds the exponential's own relative error by 88 * 2^-23 + 2^-21)
        e = eu * (z * sig).abs() + 1.1 * ez * (u.abs() + eu) + 2.0 ** -16 * ref.abs()
        big = z < -80  # there 1 + e^-z overflows to a quotient of 0: |u z| e^-80 is below any bf16 step kept here
        ok = (h.cpu().double() - ref).abs() <= e * (1 + h16) + h16 * ref.abs() + 1e-30 * (u * z).abs()
        assert (ok | big).all()
    torch.cuda.synchronize()
    assert rom.rom_get_status() == 0


@gpu
def test_expert_proj_q8_dense_projection_and_no_rows():
    gen = torch.Generator().manual_seed(0)
    a, sa = codes((1100, 144), gen)
    w, sw = codes((1, 256, 144), gen)
    for R in (1100, 50):
        out = torch.empty(R, 256, device="cuda")
        rom.rom_expert_proj_q8(rom.ROM_PROJ_SLOTS, a[:R].cuda(), sa[:R].cuda(), w.cuda(), sw.cuda(), None,
                               None, 1, None, None, None, out)
        v, m = products(a[:R], sa[:R], w, sw, [0, R], 1)
        assert ((out.cpu().double() - v).abs() <= acc_err(144, m)).all()
    rom.rom_expert_proj_q8(rom.ROM_PROJ_SLOTS, a[:0].cuda(), sa[:0].cuda(), w.cuda(), sw.cuda(), None, None, 1,
                           None, None, None, torch.empty(0, 256, device="cuda"))


@gpu
def test_expert_proj_q8_nan_rows_stay_in_their_rows():
    """A row that has no 8-bit form (NaN codes and scale) gives NaN outputs for
    itself and leaves every other row as it is."""
    for T in (200, 1200):  # the two kernels
        x = torch.randn(T, 256, generator=torch.Generator().manual_seed(1))
        gen = torch.Generator().manual_seed(2)
        w, sw = codes((4, 128, 256), gen)
        idx, r, order, off = make_routing(T, 4, 1, 5)
        args = [torch.from_numpy(t).cuda() for t in (off, order, r)]
        outs = []
        for bad in (False, True):
            if bad:
                x[7, 100] = float("inf")
            q, s = rom.quant_rows(x.cuda()[torch.from_numpy(order).long().cuda()])
            o = torch.empty(T, 128, dtype=BF16, device="cuda")
            rom.rom_expert_proj_q8(rom.ROM_PROJ_OUT, q, s, w.cuda(), sw.cuda(), None, None, 1, *args, o)
            outs.append(o.cpu())
        keep = torch.arange(T) != 7
        assert outs[1][7].isnan().all() and torch.equal(outs[0][keep], outs[1][keep])


@gpu
@pytest.mark.parametrize("T,Dm,E,k", [(1, 64, 4, 1), (300, 2048, 8, 2), (1000, 144, 64, 8)])
def test_dispatch_q8_moves_what_dispatch_moves(T, Dm, E, k):
    inp = make_block_inputs(T, Dm, 128, E, seed=T)
    d = block_to_dev(inp, "bf16")
    ref = rom.route_and_dispatch(d["x"], d["w_r"], None, E, k, False)
    x8, sc = rom.quant_rows(d["x"])
    b = rom.RoutingBuffers(T, Dm, E, k, E4M3, "cuda")
    ss = torch.empty(T * k, device="cuda")
    rom.rom_dispatch_q8(x8, sc, E, k, ref.topk_idx, ref.ws, b.offsets, b.sorted_slot, b.slot_pos, b.x_sorted, ss)
    for n in ("offsets", "sorted_slot", "slot_pos"):
        assert torch.equal(getattr(b, n), getattr(ref, n)), n
    tok = ref.sorted_slot.long() // k
    assert torch.equal(b.x_sorted.view(torch.uint8), x8.view(torch.uint8)[tok]) and torch.equal(ss, sc[tok])


@gpu
def test_dispatch_q8_refuses_inconsistent_routing():
    T, Dm, E = 300, 64, 8
    inp = make_block_inputs(T, Dm, 128, E, seed=1)
    d = block_to_dev(inp, "bf16")
    ref = rom.route_and_dispatch(d["x"], d["w_r"], None, E, 1, False)
    x8, sc = rom.quant_rows(d["x"])
    b = rom.RoutingBuffers(T, Dm, E, 1, E4M3, "cuda")
    ss = torch.full((T,), 7.0, device="cuda")
    idx = ref.topk_idx.clone()
    idx[5] = E + 3
    rom.rom_dispatch_q8(x8, sc, E, 1, idx, ref.ws, b.offsets, b.sorted_slot, b.slot_pos, b.x_sorted, ss)
    torch.cuda.synchronize()
    assert rom.rom_get_status() == rom.ROM_ERR_ROUTING
    assert 0 <= int(b.sorted_slot.min()) and int(b.sorted_slot.max()) < T and ss.isfinite().all()


# ------------------------------------------------------------------ the block


def weights(inp):
    """Q8Weights of a block on the GPU, and their float64 values [E, N, K]."""
    d = block_to_dev(inp, "bf16")
    q = [rom.Q8Weights.quantize(d[n]) for n in ("w_conv", "w_gate", "w_out")]
    return d, q, [w.q.double().cpu() * w.scale.double().cpu()[..., None] for w in q]


@gpu
@pytest.mark.parametrize("T,Dm,De,E,k,renorm", [(300, 256, 384, 8, 1, False), (1, 128, 128, 4, 2, True),
                                                (1100, 128, 256, 5, 2, True), (1300, 384, 128, 8, 1, False)])
def test_norm_and_block_in_8_bits(T, Dm, De, E, k, renorm):
    """The norm, the router, the dispatch and both projections as a user chains
    them, each stage against the formula on what the stage before it stored."""
    inp = make_block_inputs(T, Dm, De, E, seed=T, router_std=0.1)
    d, qw, w64 = weights(inp)
    nw = (1 + 0.1 * torch.randn(Dm, generator=torch.Generator().manual_seed(1))).cuda()
    res = torch.randn(T, Dm, generator=torch.Generator().manual_seed(2)).cuda()
    f = rom.residual_block_forward(d["x"], res, nw, d["w_r"], None, *qw, k, renorm)
    torch.cuda.synchronize()
    assert rom.rom_get_status() == 0
    b, n = f.block, f.norm
    rb = b.routing
    y = n.y.float().cpu().numpy()
    rt = orc.route(y, inp["w_r"], k=k, renorm=renorm)
    assert_routing_matches(rb.topk_idx.cpu().numpy(), rb.topk_w.cpu().numpy().astype(np.float64), rt, x=y, w_r=inp["w_r"])
    R = T * k
    slot = rb.sorted_slot.cpu().long()
    off = rb.offsets.cpu().tolist()
    one = torch.ones(E, De)
    A, sa = n.y8.cpu()[slot // k], n.y_scale.cpu()[slot // k]
    assert torch.equal(A.view(torch.uint8), rb.x_sorted.cpu()[:R].view(torch.uint8))
    u, mu = products(A, sa, w64[0], one, off, E)
    z, mz = products(A, sa, w64[1], one, off, E)
    eu, ez = acc_err(Dm, mu), acc_err(Dm, mz)
    tok = slot // k
    per = lambda v: torch.zeros(T, De, dtype=torch.float64).index_add_(0, tok, v)[tok]  # noqa: E731
    U_, Z_, eU, eZ = per(u), per(z), per(eu), per(ez)
    sig = torch.sigmoid(Z_)
    ref = U_ * Z_ * sig
    h16 = half_step(BF16)
    # the projections' errors through the gate; the sums over the slots and the
    # gate's own operations (fast exponential: 2^-16)
    e = eU * (Z_ * sig).abs() + 1.1 * eZ * (U_.abs() + eU) + 2.0 ** -16 * ref.abs() + 2 * k * U * (per(u.abs()) * (Z_ * sig).abs() + 1.1 * per(z.abs()) * U_.abs())
    hs = b.h_sorted.cpu()
    assert ((hs.double() - ref).abs() <= e * (1 + h16) + h16 * ref.abs() + 1e-30).all()
    h8, hsc = rows_to_8bit(hs)
    assert torch.equal(b.h8.cpu().view(torch.uint8), h8.view(torch.uint8)) and torch.equal(b.h_scale.cpu(), hsc)
    v, m = products(h8, hsc, w64[2], torch.ones(E, Dm), off, E)
    r = rb.topk_w.cpu().double().flatten()[slot][:, None]
    o = torch.zeros(T, Dm, dtype=torch.float64).index_add_(0, tok, r * v)
    eo = torch.zeros_like(o).index_add_(0, tok, r * (acc_err(De, m) + 4 * U * v.abs())) + 2 * k * U * torch.zeros_like(o).index_add_(0, tok, (r * v).abs())
    assert ((f.out.cpu().double() - o).abs() <= eo * (1 + h16) + h16 * o.abs()).all()
    # the residual stream goes on to the next norm
    again = rom.add_rmsnorm(f.out, f.residual, nw)
    assert torch.equal(again.residual.cpu(), f.out.float().cpu() + f.residual.cpu())


@gpu
def test_block_q8_quantises_x_itself_and_replays_in_a_graph():
    T, Dm, De, E = 400, 256, 256, 8
    inp = make_block_inputs(T, Dm, De, E, seed=3)
    d, qw, _ = weights(inp)
    x8, sc = rom.quant_rows(d["x"])
    a = rom.block_forward_q8(d["x"], d["w_r"], None, *qw, 1)
    b = rom.block_forward_q8(d["x"], d["w_r"], None, *qw, 1, x8=x8, x_scale=sc)
    assert torch.equal(a.out, b.out)
    ref = a.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rom.block_forward_q8(d["x"], d["w_r"], None, *qw, 1, bufs=a)
    a.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, ref)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c = rom.block_forward_q8(d["x"], d["w_r"], None, *qw, 1, stream=st)
    st.synchronize()
    assert torch.equal(c.out, ref) and rom.rom_get_status() == 0


@gpu
def test_block_q8_empty_batch_and_refusals():
    inp = make_block_inputs(4, 128, 128, 4, seed=3)
    d, qw, _ = weights(inp)
    for k in (1, 2):
        b = rom.block_forward_q8(d["x"][:0], d["w_r"], None, *qw, k)
        assert b.out.shape == (0, 128) and (b.routing.offsets.cpu() == 0).all()
    # d_model 144: no whole 128-column tiles of the Out projection
    i2 = make_block_inputs(1300, 144, 128, 8, seed=1300, router_std=0.1)
    d2, qw2, _ = weights(i2)
    with pytest.raises(rom.RomError, match="multiples of 128"):
        rom.block_forward_q8(d2["x"], d2["w_r"], None, *qw2, 1)
    with pytest.raises(rom.RomError, match="fit together"):
        rom.block_forward_q8(d["x"], d["w_r"], None, qw[0], qw[1], qw2[2], 1)
    with pytest.raises(rom.RomError, match="x must be"):
        rom.block_forward_q8(d["x"].float(), d["w_r"], None, *qw, 1)
    with pytest.raises(rom.RomError, match="come together"):
        rom.block_forward_q8(d["x"], d["w_r"], None, *qw, 1, x8=torch.empty(4, 128, dtype=E4M3, device="cuda"))
    o = torch.empty(4, 128, device="cuda")
    with pytest.raises(rom.RomError, match="out must be"):
        rom.rom_expert_proj_q8(rom.ROM_PROJ_OUT, qw[0].q[0, :4], qw[0].scale[0, :4], qw[2].q, qw[2].scale, None, None, 1,
                               torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"),
                               torch.zeros(4, 1, device="cuda"), o)
    with pytest.raises(rom.RomError, match="need w1"):
        rom.rom_expert_proj_q8(rom.ROM_PROJ_CONV_GATE, qw[0].q[0, :4], qw[0].scale[0, :4], qw[2].q, qw[2].scale, None, None, 1,
                               torch.zeros(5, dtype=torch.int32, device="cuda"), None, None, o.to(BF16))


@gpu
def test_norm_and_block_train_together():
    """residual_block_forward / _backward on bf16 weights: the norm's output and
    gradients around the block's own, checked against those calls made one by
    one, and the norm's part against the formula."""
    T, Dm, De, E = 200, 256, 256, 4
    inp = make_block_inputs(T, Dm, De, E, seed=5, with_dout=True)
    d = block_to_dev(inp, "bf16")
    nw = (1 + 0.1 * torch.randn(Dm, generator=torch.Generator().manual_seed(1))).cuda()
    res = torch.randn(T, Dm, generator=torch.Generator().manual_seed(2)).cuda()
    dres = torch.randn(T, Dm, generator=torch.Generator().manual_seed(3)).cuda()
    dout = torch.from_numpy(inp["dout"]).to(BF16).cuda()
    ws = (d["w_conv"], d["w_gate"], d["w_out"])
    f = rom.residual_block_forward(d["x"], res, nw, d["w_r"], None, *ws, 2, True)
    bwd, g = rom.residual_block_backward(f, dout, nw, d["w_r"], *ws, True, dresidual=dres)
    blk = rom.block_forward(f.norm.y, d["w_r"], None, *ws, k=2, renorm=True)
    assert torch.equal(blk.out, f.out)
    b2 = rom.block_backward(blk, dout, d["w_r"], *ws, renorm=True, x=f.norm.y)
    assert torch.equal(b2.dx, bwd.dx) and torch.equal(b2.dw_out, bwd.dw_out) and torch.equal(b2.dw_r, bwd.dw_r)
    from test_norm_quant import bwd_reference
    ds, err, dw, dw_err = bwd_reference(bwd.dx.cpu(), dres.cpu(), f.residual.cpu(), nw.cpu(), f.norm.rstd.cpu())
    h = half_step(BF16)
    assert ((g.dx.cpu().double() - ds).abs() <= err * (1 + h) + h * ds.abs()).all()
    assert ((g.dresidual.cpu().double() - ds).abs() <= err + U * ds.abs()).all()
    assert ((g.dw.cpu().double() - dw).abs() <= dw_err).all()


def test_residual_block_backward_refuses_other_blocks_and_weights_modes():
    class Norm:
        residual = None

    class Fake:
        out = None

    plain = rom.BlockBuffers.__new__(rom.BlockBuffers)
    plain.out = None
    with pytest.raises(rom.RomError, match="no backward"):
        rom.residual_block_backward(rom.ResidualBlock(Norm(), Fake(), True), *[None] * 6)
    for ran, asked in ((True, False), (False, True)):
        with pytest.raises(rom.RomError, match="renorm="):
            rom.residual_block_backward(rom.ResidualBlock(Norm(), plain, ran), *[None] * 6, renorm=asked)


@gpu
@pytest.mark.parametrize("renorm", [True, False])
def test_residual_block_backward_takes_the_forwards_weights_mode(renorm):
    T, Dm, De, E = 70, 256, 256, 4  # (the backward takes multiples of 256)
    inp = make_block_inputs(T, Dm, De, E, seed=6, with_dout=True)
    d = block_to_dev(inp, "bf16")
    nw = torch.ones(Dm, device="cuda")
    dout = torch.from_numpy(inp["dout"]).to(BF16).cuda()
    ws = (d["w_conv"], d["w_gate"], d["w_out"])
    f = rom.residual_block_forward(d["x"], None, nw, d["w_r"], None, *ws, 2, renorm)
    bwd, _ = rom.residual_block_backward(f, dout, nw, d["w_r"], *ws)
    ref = rom.block_backward(f.block, dout, d["w_r"], *ws, renorm=renorm, x=f.norm.y)
    assert torch.equal(ref.dx, bwd.dx) and torch.equal(ref.dlogits, bwd.dlogits)
