"""The routed projection on 4-bit weights, its quantiser and the decode paths
that call it."""
import ctypes

import numpy as np
import pytest
import torch

from lowbit_util import U, half_step, make_routing, w4_decode, w4_position
from mixture_experts_projections_b200 import rom
from mixture_experts_projections_b200.inputs import make_block_inputs
from oracle import rom_oracle as orc
from parity_util import assert_routing_matches, block_to_dev

BF16, F32 = torch.bfloat16, torch.float32
FAKE = ctypes.c_void_p(1 << 20)
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_projections_b200.build import build
    build()
    return rom.load_library()


@pytest.mark.parametrize("kw,code", [
    (dict(proj=0), 1), (dict(proj=5), 1), (dict(T=-1), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(E=65), 1),
    (dict(k=3, E=2), 1), (dict(k=9, E=16), 1), (dict(group=16), 1), (dict(group=0), 1), (dict(x=None), 1),
    (dict(q0=None), 1), (dict(s0=None), 1), (dict(topk_idx=None), 1), (dict(topk_w=None), 1), (dict(out=None), 1),
    (dict(q1=FAKE), 1), (dict(proj=4, q1=FAKE), 1), (dict(proj=4), 1),
    (dict(T=65), 2), (dict(K=60), 2), (dict(K=1500), 2), (dict(x=ctypes.c_void_p((1 << 20) + 8)), 2),
    (dict(s0=ctypes.c_void_p((1 << 20) + 2)), 2), (dict(out=ctypes.c_void_p((1 << 20) + 1)), 2),
    (dict(k=2, out=ctypes.c_void_p((1 << 20) + 2)), 2),
])
def test_expert_proj_w4_rejects_bad_arguments(lib, kw, code):
    a = dict(proj=2, x=FAKE, T=8, K=64, q0=FAKE, s0=FAKE, q1=None, s1=None, N=100, E=8, k=1, group=64,
             topk_idx=FAKE, topk_w=FAKE, out=FAKE, stream=None)
    a.update(kw)
    assert lib.rom_expert_proj_w4(*a.values()) == code


def far(i):
    return ctypes.c_void_p((1 << 20) + i * (1 << 32))


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 1), (dict(E=0), 1), (dict(N=0), 1), (dict(K=-8), 1), (dict(group=96), 1), (dict(w=None), 1),
    (dict(q=None), 1), (dict(s=None), 1), (dict(K=12), 2), (dict(q=ctypes.c_void_p((1 << 32) + 8)), 2),
    (dict(q=far(0)), 1), (dict(s=far(1)), 1),
])
def test_quant_w4_rejects_bad_arguments(lib, kw, code):
    a = dict(dtype=1, w=far(0), E=2, N=20, K=64, group=32, q=far(1), s=far(2), stream=None)
    a.update(kw)
    assert lib.rom_quant_expert_weights_w4(*a.values()) == code


def test_w4_sizes(lib):
    assert lib.rom_w4_code_bytes(2, 16, 128) == 2 * 1024
    assert lib.rom_w4_code_bytes(1, 17, 129) == 4 * 1024
    assert lib.rom_w4_code_bytes(0, 16, 128) == 0
    assert lib.rom_w4_scale_bytes(1, 16, 128, 32) == 16 * 4 * 2
    assert lib.rom_w4_scale_bytes(3, 17, 129, 128) == 3 * 4 * 16 * 2
    assert lib.rom_w4_scale_bytes(1, 16, 128, 48) == 0


def test_w4_positions_are_a_bijection():
    byte, shift = w4_position(32, 256)
    at = (byte * 2 + shift // 4).reshape(-1)
    assert np.array_equal(np.sort(at), np.arange(32 * 256))


def random_w4(E, N, K, group, seed):
    """Any codes 0 .. 15 and scales of several magnitudes, in the storage (random
    bytes: the padding holds the codes and scales that it has to)."""
    g = torch.Generator().manual_seed(seed)
    nt, kb = -(-N // 16), -(-K // 128)
    q = torch.full((E, nt, kb, 2, 8, 4, 16), 0x88, dtype=torch.uint8)
    byte, shift = w4_position(N, K)
    flat = q.view(E, -1).numpy()
    code = torch.randint(0, 16, (E, N, K), generator=g).numpy().astype(np.uint8)
    flat[:] = 0
    pad = np.full((E, flat.shape[1] * 2), 8, np.uint8)
    pad[:, (byte * 2 + shift // 4)] = code
    flat[:] = pad[:, 0::2] | (pad[:, 1::2] << 4)
    s = (torch.rand(E, nt, kb, 16, 128 // group, generator=g) * 2.0 ** torch.randint(-6, 0, (E, nt, kb, 16, 128 // group), generator=g)).to(BF16)
    n = (np.arange(nt * 16) >= N).reshape(nt, 16)
    for a in range(nt):
        for r in range(16):
            if n[a, r]:
                s[:, a, :, r] = 0
    kpad = (np.arange(kb * (128 // group)) * group >= K).reshape(kb, -1)
    s[:, :, torch.from_numpy(kpad).nonzero()[:, 0], :, torch.from_numpy(kpad).nonzero()[:, 1]] = 0
    return q, s


def slot_products(x, w64, idx, k):
    """float64 (values, sums of magnitudes) per slot."""
    T = x.shape[0]
    X = x.double().numpy()
    v = np.einsum("sk,snk->sn", np.repeat(X, k, 0), w64[idx.reshape(-1)]) if T else np.zeros((0, w64.shape[1]))
    m = np.einsum("sk,snk->sn", np.abs(np.repeat(X, k, 0)), np.abs(w64[idx.reshape(-1)]))
    return torch.from_numpy(v), torch.from_numpy(m)


def acc_err(K, m):
    """Codes and bf16 activations multiply exactly; sums in float32 in any order
    with up to a whole unit (2 U) each, one product per group, up to 8 parts of
    the columns."""
    return (K + K // 32 + 16) * 2 * U * m


CASES = [
    # T, K, N, E, k, group, pin
    (1, 64, 16, 1, 1, 128, None), (1, 4096, 130, 4, 1, 128, None), (5, 1000, 37, 4, 2, 32, None),
    (8, 128, 128, 8, 1, 64, None), (9, 2056, 300, 3, 3, 64, None), (16, 520, 1, 16, 2, 32, None),
    (17, 384, 260, 5, 1, 128, None), (64, 256, 144, 4, 1, 32, None), (64, 640, 50, 64, 8, 64, None),
    # columns shared by a cluster, once over the tokens and (all 64 on one expert) several times
    (3, 8192, 16, 1, 1, 64, None), (64, 4096, 130, 4, 1, 128, 2), (40, 2048, 20, 16, 2, 32, 3),
    (64, 768, 140, 4, 1, 128, 2), (33, 8, 8, 2, 2, 32, None), (40, 1160, 129, 2, 1, 128, 0),
    # an expert's passes shared by CTAs, with and without shared columns; fewer blocks of columns than CTAs of a cluster
    (60, 1504, 200, 1, 1, 64, None), (64, 264, 70, 2, 2, 32, None), (41, 72, 2500, 1, 1, 128, None),
    (20, 640, 20, 4, 1, 64, None),
    # more CTAs of one token block than two per SM
    (6, 256, 9000, 16, 2, 32, None), (7, 264, 8200, 16, 2, 64, None), (5, 136, 9100, 16, 3, 128, None),
]


@gpu
@pytest.mark.parametrize("T,K,N,E,k,group,pin", CASES)
def test_expert_proj_w4_matches_the_products(T, K, N, E, k, group, pin):
    q0, s0 = random_w4(E, N, K, group, seed=T)
    q1, s1 = random_w4(E, N, K, group, seed=T + 1)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(2)).to(BF16)
    idx, r, _, _ = make_routing(T, E, k, T, pin)
    if pin is not None:
        idx = np.minimum(idx, E - 1)
    d = [t.cuda() for t in (x, q0, s0, q1, s1)]
    idxd, rd = torch.from_numpy(idx).cuda(), torch.from_numpy(r).cuda()
    v0, m0 = slot_products(x, w4_decode(q0, s0, N, K)[0], idx, k)
    v1, m1 = slot_products(x, w4_decode(q1, s1, N, K)[0], idx, k)
    R = T * k
    # guard rows behind the output: they stay as they are
    uz = torch.full((2 * R + 1, N), 7.0, device="cuda")
    rom.rom_expert_proj_w4(rom.ROM_PROJ_CONV_GATE_SLOTS, *d, N, k, idxd, None, uz[:2 * R].view(2, R, N))
    got = uz.cpu().double()
    assert ((got[:R] - v0).abs() <= acc_err(K, m0)).all() and ((got[R:2 * R] - v1).abs() <= acc_err(K, m1)).all()
    assert (got[2 * R] == 7).all()
    out = torch.full((R + 1, N), 7.0, device="cuda")
    rom.rom_expert_proj_w4(rom.ROM_PROJ_SLOTS, d[0], d[3], d[4], None, None, N, k, idxd, None, out[:R])
    # (not bit for bit: how the columns are shared out goes by the whole call)
    assert ((out[:R].cpu().double() - v1).abs() <= acc_err(K, m1)).all() and (out[R] == 7).all()
    rr = torch.from_numpy(r).double().view(-1, 1)
    e = rr * (acc_err(K, m0) + U * v0.abs())
    if k == 1:
        o = torch.full((T + 1, N), 7.0, dtype=BF16, device="cuda")
        h = half_step(BF16)
        for proj in (rom.ROM_PROJ_INPROJ, rom.ROM_PROJ_OUT):
            rom.rom_expert_proj_w4(proj, *d[:3], None, None, N, k, idxd, rd, o[:T])
            assert ((o[:T].cpu().double() - rr * v0).abs() <= e * (1 + h) + h * (rr * v0).abs()).all()
        assert (o[T].float() == 7).all()
    else:
        rom.rom_expert_proj_w4(rom.ROM_PROJ_OUT, *d[:3], None, None, N, k, idxd, rd, out[:R])
        assert ((out[:R].cpu().double() - rr * v0).abs() <= e).all()
    torch.cuda.synchronize()
    assert rom.rom_get_status() == 0


@gpu
def test_expert_proj_w4_repeated_and_invalid_experts():
    """A token that names one expert in several slots gets the same product in
    each, also when that gives an expert more than 64 slots; a slot with an index
    outside [0, E) is left as it was and reported."""
    T, K, N, E, k = 40, 256, 48, 3, 3
    q, s = random_w4(E, N, K, 64, seed=1)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(2)).to(BF16)
    idx = np.full((T, k), 1, np.int32)
    idx[3] = (0, 2, 0)
    v, m = slot_products(x, w4_decode(q, s, N, K)[0], idx, k)
    out = torch.full((T * k, N), 7.0, device="cuda")
    args = (rom.ROM_PROJ_SLOTS, x.cuda(), q.cuda(), s.cuda(), None, None, N, k)
    rom.rom_expert_proj_w4(*args, torch.from_numpy(idx).cuda(), None, out)
    assert ((out.cpu().double() - v).abs() <= acc_err(K, m)).all()
    assert rom.rom_get_status() == 0
    bad = idx.copy()
    bad[0, 1], bad[7, 0] = -1, E
    out2 = torch.full((T * k, N), 7.0, device="cuda")
    rom.rom_expert_proj_w4(*args, torch.from_numpy(bad).cuda(), None, out2)
    torch.cuda.synchronize()
    assert rom.rom_get_status() == rom.ROM_ERR_ROUTING
    left = torch.zeros(T * k, dtype=torch.bool)
    left[[1, 21]] = True
    assert (out2[left.cuda()] == 7).all()
    assert ((out2.cpu().double() - v).abs() <= acc_err(K, m))[~left].all()


@gpu
def test_expert_proj_w4_special_values_stay_in_their_rows():
    T, K, N = 20, 520, 40
    q, s = random_w4(1, N, K, 128, seed=3)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(2)).to(BF16)
    idx, r = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda")
    o = [torch.empty(T, N, dtype=BF16, device="cuda") for _ in range(2)]
    rom.rom_expert_proj_w4(rom.ROM_PROJ_OUT, x.cuda(), q.cuda(), s.cuda(), None, None, N, 1, idx, r, o[0])
    x[4, 519] = float("nan")
    s[0, 1, 0, 5, 0] = float("nan")  # row 21
    rom.rom_expert_proj_w4(rom.ROM_PROJ_OUT, x.cuda(), q.cuda(), s.cuda(), None, None, N, 1, idx, r, o[1])
    assert o[1][4].isnan().all() and o[1][:, 21].isnan().all()
    keep = torch.ones(T, N, dtype=torch.bool)
    keep[4], keep[:, 21] = False, False
    assert torch.equal(o[0].cpu()[keep], o[1].cpu()[keep])


@gpu
@pytest.mark.parametrize("E,N,K,group", [(1, 16, 128, 128), (3, 37, 1000, 32), (2, 130, 264, 64), (1, 5, 8, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantiser_gives_the_definitions_codes(E, N, K, group, dtype):
    w = (torch.randn(E, N, K, generator=torch.Generator().manual_seed(N)) / K ** 0.5).to(dtype)
    w[0, 0, :] = 0
    w[0, 1 % N, 0] = 0 if N == 1 else 3.0
    p = rom.W4Weights.quantize(w.cuda(), group)
    val, codes, scale = w4_decode(p.q, p.s, N, K)
    gw = torch.nn.functional.pad(w.float(), (0, -K % group)).view(E, N, -1, group)
    s = (gw.abs().amax(-1) / torch.tensor(7.0)).to(BF16).float()
    q = torch.where(s[..., None] > 0, torch.round(gw / s[..., None]), torch.zeros(())).clamp(-8, 7) + 8
    q = q.reshape(E, N, -1)[..., :K].numpy()
    s = s.repeat_interleave(group, -1)[..., :K].numpy()
    assert np.array_equal(codes, q) and np.array_equal(scale, s)
    assert np.array_equal(p.dequantize().cpu().numpy(), (val).astype(np.float32))
    # padding: codes 8, scales 0
    byte, shift = w4_position(-(-N // 16) * 16, -(-K // 128) * 128)
    allc = (p.q.cpu().numpy().reshape(E, -1)[:, byte] >> shift) & 15
    assert (allc[:, N:] == 8).all() and (allc[:, :, K:] == 8).all()
    assert (p.s.cpu().float()[:, -1, :, N % 16 or 16:] == 0).all()
    # half a step of the group's scale from the weights (the largest may clamp by the scale's rounding)
    assert (np.abs(val - w.double().numpy()) <= s * (0.5 + 7 * 2.0 ** -8)).all()


@gpu
def test_quantiser_marks_groups_without_a_scale():
    w = torch.randn(1, 16, 256, generator=torch.Generator().manual_seed(0))
    w[0, 2, 40], w[0, 3, 200] = float("inf"), float("nan")
    p = rom.W4Weights.quantize(w.cuda(), 64)
    s = p.s.float().cpu()[0, 0].permute(1, 0, 2).reshape(16, 4)
    want = torch.zeros(16, 4, dtype=torch.bool)
    want[2, 0] = want[3, 3] = True
    assert torch.equal(s.isnan(), want)


# ------------------------------------------------------------------ decode paths


@gpu
@pytest.mark.parametrize("T,k,renorm", [(1, 1, False), (64, 1, False), (30, 2, True), (150, 2, True), (130, 1, False)])
def test_inproj_forward_on_4_bit_weights(T, k, renorm):
    Dm, N, E = 512, 200, 8
    inp = make_block_inputs(T, Dm, 208, E, seed=T)
    d = block_to_dev(inp, "bf16")
    w = d["w_conv"][:, :N].contiguous()
    p = rom.W4Weights.quantize(w, 64)
    out, bufs = rom.inproj_forward(d["x"], d["w_r"], None, k, renorm, w_q4=p)
    torch.cuda.synchronize()
    assert rom.rom_get_status() == 0
    rt = orc.route(inp["x"], inp["w_r"], k=k, renorm=renorm)
    idx, r = bufs.topk_idx.cpu().numpy(), bufs.topk_w.cpu()
    assert_routing_matches(idx, r.numpy().astype(np.float64), rt, x=inp["x"], w_r=inp["w_r"])
    v, m = slot_products(d["x"].cpu(), w4_decode(p.q, p.s, N, Dm)[0], idx, k)
    rr = r.double().view(-1, 1)
    ref = (rr * v).view(T, k, N).sum(1)
    e = (rr * (acc_err(Dm, m) + (k + 1) * U * v.abs())).view(T, k, N).sum(1)
    h = half_step(BF16)
    assert ((out.cpu().double() - ref).abs() <= e * (1 + h) + h * ref.abs()).all()


@gpu
@pytest.mark.parametrize("T,k,renorm", [(1, 1, False), (37, 2, True), (64, 1, False), (100, 2, True)])
def test_norm_and_block_on_4_bit_weights(T, k, renorm):
    """The norm, the router and the three projections of a decode step as a user
    chains them, each stage against the formula on what the stage before stored."""
    Dm, De, E = 264, 392, 4
    inp = make_block_inputs(T, Dm, De, E, seed=T, router_std=0.1)
    d = block_to_dev(inp, "bf16")
    p = [rom.W4Weights.quantize(d[n], g) for n, g in (("w_conv", 32), ("w_gate", 32), ("w_out", 128))]
    nw = torch.ones(Dm, device="cuda")
    f = rom.residual_block_forward(d["x"], None, nw, d["w_r"], None, *p, k, renorm)
    torch.cuda.synchronize()
    assert rom.rom_get_status() == 0
    b = f.block
    y = f.norm.y.cpu()
    idx, r = b.topk_idx.cpu().numpy(), b.topk_w.cpu()
    rt = orc.route(y.float().numpy(), inp["w_r"], k=k, renorm=renorm)
    assert_routing_matches(idx, r.numpy().astype(np.float64), rt, x=y.float().numpy(), w_r=inp["w_r"])
    uz = b.uz.cpu().double()
    for i in range(2):
        v, m = slot_products(y, w4_decode(p[i].q, p[i].s, De, Dm)[0], idx, k)
        assert ((uz[i] - v).abs() <= acc_err(Dm, m)).all()
    u, z = (t.view(T, k, De).sum(1) for t in uz)
    mu, mz = (t.abs().view(T, k, De).sum(1) for t in uz)
    ref = u * z * torch.sigmoid(z)
    h = half_step(BF16)
    # the slots' sums (k roundings of their magnitudes) and expf, 1 + ., / and *
    e = k * U * (mu * (z * torch.sigmoid(z)).abs() + 1.1 * mz * u.abs()) + 16 * U * ref.abs() * (1 + z.abs())
    hs = b.h.cpu()
    assert ((hs.double() - ref).abs() <= e * (1 + h) + h * ref.abs()).all()
    v, m = slot_products(hs, w4_decode(p[2].q, p[2].s, Dm, De)[0], idx, k)
    rr = r.double().view(-1, 1)
    o = (rr * v).view(T, k, Dm).sum(1)
    e = (rr * (acc_err(De, m) + (k + 1) * U * v.abs())).view(T, k, Dm).sum(1)
    assert ((f.out.cpu().double() - o).abs() <= e * (1 + h) + h * o.abs()).all()


@gpu
def test_w4_block_replays_in_a_graph_and_on_another_stream():
    T, Dm, De, E = 16, 256, 256, 4
    inp = make_block_inputs(T, Dm, De, E, seed=3)
    d = block_to_dev(inp, "bf16")
    p = [rom.W4Weights.quantize(d[n]) for n in ("w_conv", "w_gate", "w_out")]
    a = rom.block_forward_w4(d["x"], d["w_r"], None, *p, 1)
    ref = a.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rom.block_forward_w4(d["x"], d["w_r"], None, *p, 1, bufs=a)
    for _ in range(3):
        a.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, ref)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c = rom.block_forward_w4(d["x"], d["w_r"], None, *p, 1, stream=st)
    st.synchronize()
    assert torch.equal(c.out, ref)
    assert rom.block_forward_w4(d["x"][:0], d["w_r"], None, *p, 1).out.shape == (0, Dm)
    assert rom.inproj_forward(d["x"][:0], d["w_r"], None, 2, True, w_q4=p[0])[0].shape == (0, De)


@gpu
def test_w4_binding_refuses_wrong_tensors():
    q, s = (t.cuda() for t in random_w4(2, 40, 256, 64, seed=0))
    x = torch.zeros(4, 256, dtype=BF16, device="cuda")
    idx, r = torch.zeros(4, 1, dtype=torch.int32, device="cuda"), torch.ones(4, 1, device="cuda")
    o = torch.empty(4, 40, dtype=BF16, device="cuda")
    ok = dict(proj=rom.ROM_PROJ_OUT, x=x, q0=q, s0=s, q1=None, s1=None, N=40, k=1, topk_idx=idx, topk_w=r, out=o)
    rom.rom_expert_proj_w4(**ok)
    for bad, match in ((dict(x=x.float()), "x must be"), (dict(N=64), "does not hold"), (dict(x=x[:, :128].contiguous()), "does not hold"),
                       (dict(s0=s[:1]), "s0 must be"), (dict(out=o.float()), "out must be"), (dict(topk_idx=idx.long()), "topk_idx must be"),
                       (dict(topk_w=None), "INVALID"), (dict(q1=q), "go with"), (dict(x=torch.zeros(65, 256, dtype=BF16, device="cuda"), topk_idx=torch.zeros(65, 1, dtype=torch.int32, device="cuda"), topk_w=torch.ones(65, 1, device="cuda"), out=torch.empty(65, 40, dtype=BF16, device="cuda")), "UNSUPPORTED")):
        with pytest.raises(rom.RomError, match=match):
            rom.rom_expert_proj_w4(**{**ok, **bad})
    with pytest.raises(rom.RomError, match="group must be"):
        rom.W4Weights.quantize(torch.zeros(1, 16, 64, device="cuda"), 16)


@gpu
def test_w4_calls_on_two_streams_at_once():
    q, s = (t.cuda() for t in random_w4(4, 1000, 2048, 64, seed=0))
    x = torch.randn(32, 2048, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    idx, r, _, _ = make_routing(32, 4, 2, 3)
    idx, r = torch.from_numpy(idx).cuda(), torch.from_numpy(r).cuda()
    outs = [torch.empty(64, 1000, device="cuda") for _ in range(9)]
    args = (rom.ROM_PROJ_OUT, x, q, s, None, None, 1000, 2, idx, r)
    rom.rom_expert_proj_w4(*args, outs[8])
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    for i in range(8):
        rom.rom_expert_proj_w4(*args, outs[i], stream=st[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[8]) for o in outs[:8]) and rom.rom_get_status() == 0
